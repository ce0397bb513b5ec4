// blocks.cuh -- rows of fp32, bf16 or fp16 as a thread's columns, and e4m3 with a
// scale per block, for the experts' row kernels (moe.cu) and the quantisation
// (quant.cu).
//
// A block of values x with the largest magnitude a stands for scale q:
//   a' = max(a, 2^-100),  scale = a' / 448,  q = e4m3(x (448 / a'))
// (448: the type's largest value; both divisions rounded in fp32, q to nearest even).
// 2^-100 keeps scale and 448 / a' normal numbers, so a block of zeros needs no case of
// its own.  a is the largest of the bit patterns without their signs, so a NaN wins over
// an infinity and that over every number: a block that holds either has a scale that is
// not finite, and each of its values stands for a NaN.
#pragma once

#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "act.cuh"
#include "vlmce.h"

namespace vlmce {
namespace blocks {

constexpr int kBlock = 128;
constexpr uint32_t kTinyBits = (127u - 100u) << 23;  // 2^-100
constexpr float kE4m3Max = 448.f;

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The scale of a block whose largest magnitude has these bits, and what its values are
// multiplied by.
__device__ __forceinline__ float scale_of(uint32_t amax, float &inv) {
    const float a = __uint_as_float(max(amax, kTinyBits));
    inv = kE4m3Max / a;
    return a / kE4m3Max;
}

__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}
template <int DT>
constexpr int elt_bytes = DT == VLMCE_F32 ? 4 : 2;

template <int DT>
__device__ __forceinline__ float load1(const unsigned char *row, int64_t c) {
    if constexpr (DT == VLMCE_F32)
        return reinterpret_cast<const float *>(row)[c];
    else
        return act::from16(reinterpret_cast<const uint16_t *>(row)[c], DT == VLMCE_F16);
}
// W words that start `off` (of 16, a multiple of their elements' size) bytes into these.
template <int W, bool HALVES>
__device__ __forceinline__ void move_into_place(uint32_t (&w)[W + 4], uint32_t off) {
#pragma unroll
    for (int k = 0; k < W + 2; ++k) w[k] = off & 8 ? w[k + 2] : w[k];
#pragma unroll
    for (int k = 0; k < W + 1; ++k) w[k] = off & 4 ? w[k + 1] : w[k];
    if constexpr (HALVES) {
#pragma unroll
        for (int k = 0; k < W; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], (off & 2) * 8);
    }
}

// A thread's eight columns of a row, of the 256 that its warp takes from `base`, in accesses
// of U bytes (16, 4, or 2 of 16-bit values) that divide the row's length and addresses: a
// warp's access covers 32 U consecutive bytes.
template <int DT, int U>
struct Cols {
    static constexpr int kElt = elt_bytes<DT>, P = U / kElt;  // columns of an access
    static constexpr int N = 8, kWarp = 32 * N;
    static constexpr bool kF16 = DT == VLMCE_F16;
    int64_t c;
    __device__ __forceinline__ Cols(int64_t base, int lane) : c(base + P * lane) {}
    __device__ __forceinline__ bool in(int i, int64_t H) const { return c + i / P * (32 * P) < H; }
    __device__ __forceinline__ int64_t at(int i) const { return (c + i / P * (32 * P)) * kElt; }

    // The values as they are in memory, to have many on their way in few registers.
    struct Raw {
        uint32_t u[U > 2 ? N * kElt / 4 : N];
    };
    __device__ __forceinline__ void fetch(const unsigned char *row, int64_t H, Raw &r) const {
#pragma unroll
        for (int i = 0; i < N; i += P) {
            if constexpr (U == 16) {
                uint32_t *to = r.u + i * kElt / 4;
                if (in(i, H)) {
                    const uint4 q = *reinterpret_cast<const uint4 *>(row + at(i));
                    to[0] = q.x, to[1] = q.y, to[2] = q.z, to[3] = q.w;
                } else {
                    to[0] = to[1] = to[2] = to[3] = 0;
                }
            } else if constexpr (U == 4) {
                r.u[i * kElt / 4] = in(i, H) ? *reinterpret_cast<const uint32_t *>(row + at(i)) : 0;
            } else {
                r.u[i] = in(i, H) ? *reinterpret_cast<const uint16_t *>(row + at(i)) : 0;
            }
        }
    }
    // Value i of them.
    static __device__ __forceinline__ float value(const Raw &r, int i) {
        if constexpr (DT == VLMCE_F32) {
            return __uint_as_float(r.u[i]);
        } else if constexpr (U > 2) {
            float a, b;
            act::unpack16x2(r.u[i / 2], a, b, kF16);
            return i & 1 ? b : a;
        } else {
            return act::from16(static_cast<uint16_t>(r.u[i]), kF16);
        }
    }
    __device__ __forceinline__ void store(unsigned char *row, int64_t H, const float (&v)[N]) const {
#pragma unroll
        for (int i = 0; i < N; i += P) {
            if (!in(i, H)) continue;
            uint32_t w[U > 4 ? U / 4 : 1];
            if constexpr (DT == VLMCE_F32) {
#pragma unroll
                for (int k = 0; k < P; ++k) w[k] = __float_as_uint(v[i + k]);
            } else if constexpr (U > 2) {
#pragma unroll
                for (int k = 0; k < P; k += 2) w[k / 2] = act::pack16x2(v[i + k], v[i + k + 1], kF16);
            } else {
                w[0] = act::to16(v[i], kF16);
            }
            if constexpr (U == 16)
                *reinterpret_cast<uint4 *>(row + at(i)) = make_uint4(w[0], w[1], w[2], w[3]);
            else if constexpr (U == 4)
                *reinterpret_cast<uint32_t *>(row + at(i)) = w[0];
            else
                *reinterpret_cast<uint16_t *>(row + at(i)) = static_cast<uint16_t>(w[0]);
        }
    }
};

}  // namespace blocks
}  // namespace vlmce
