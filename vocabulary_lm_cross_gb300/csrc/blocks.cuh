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
__device__ __forceinline__ uint8_t to_e4m3(float a) {
    return __nv_cvt_float_to_fp8(a, __NV_SATFINITE, __NV_E4M3);
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
template <int DT>
__device__ __forceinline__ void store1(unsigned char *row, int64_t c, float v) {
    if constexpr (DT == VLMCE_F32)
        reinterpret_cast<float *>(row)[c] = v;
    else
        reinterpret_cast<uint16_t *>(row)[c] = act::to16(v, DT == VLMCE_F16);
}
// Eight consecutive values, 16-byte aligned.
template <int DT>
__device__ __forceinline__ void load8(const unsigned char *row, int64_t c, float (&v)[8]) {
    if constexpr (DT == VLMCE_F32) {
        const float4 *p = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(row) + c);
        const float4 a = p[0], b = p[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 u =
            *reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(row) + c);
        act::unpack16x2(u.x, v[0], v[1], DT == VLMCE_F16);
        act::unpack16x2(u.y, v[2], v[3], DT == VLMCE_F16);
        act::unpack16x2(u.z, v[4], v[5], DT == VLMCE_F16);
        act::unpack16x2(u.w, v[6], v[7], DT == VLMCE_F16);
    }
}
template <int DT>
__device__ __forceinline__ void store8(unsigned char *row, int64_t c, const float (&v)[8]) {
    if constexpr (DT == VLMCE_F32) {
        float4 *p = reinterpret_cast<float4 *>(reinterpret_cast<float *>(row) + c);
        p[0] = make_float4(v[0], v[1], v[2], v[3]);
        p[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        constexpr bool f16 = DT == VLMCE_F16;
        *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(row) + c) =
            make_uint4(act::pack16x2(v[0], v[1], f16), act::pack16x2(v[2], v[3], f16),
                       act::pack16x2(v[4], v[5], f16), act::pack16x2(v[6], v[7], f16));
    }
}

// A thread's columns of a row, of the 256 (VEC) or 128 that its warp takes from `base`:
// eight in a row, in 16-byte accesses; or four that are 32 apart, at any alignment (a
// warp's accesses cover consecutive elements).
template <bool VEC>
struct Cols {
    static constexpr int N = VEC ? 8 : 4;
    static constexpr int kWarp = 32 * N;
    int64_t c;
    __device__ __forceinline__ Cols(int64_t base, int lane) : c(base + (VEC ? 8 * lane : lane)) {}
    __device__ __forceinline__ bool in(int i, int64_t H) const { return VEC ? c < H : c + 32 * i < H; }

    // The values as they are in memory, to have many on their way in few registers.
    template <int DT>
    struct Raw {
        static constexpr int kWords = VEC ? 2 * elt_bytes<DT> : 4;
        uint32_t u[kWords];
    };
    template <int DT>
    __device__ __forceinline__ void fetch(const unsigned char *row, int64_t H, Raw<DT> &r) const {
        if constexpr (VEC) {
            if (c < H) {
                const uint4 *p = reinterpret_cast<const uint4 *>(row + c * elt_bytes<DT>);
#pragma unroll
                for (int i = 0; i < elt_bytes<DT> / 2; ++i) {
                    const uint4 q = p[i];
                    r.u[4 * i] = q.x, r.u[4 * i + 1] = q.y, r.u[4 * i + 2] = q.z, r.u[4 * i + 3] = q.w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < Raw<DT>::kWords; ++i) r.u[i] = 0;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (DT == VLMCE_F32)
                    r.u[i] = in(i, H) ? reinterpret_cast<const uint32_t *>(row)[c + 32 * i] : 0;
                else
                    r.u[i] = in(i, H) ? reinterpret_cast<const uint16_t *>(row)[c + 32 * i] : 0;
            }
        }
    }
    // Value i of them.
    template <int DT>
    static __device__ __forceinline__ float value(const Raw<DT> &r, int i) {
        if constexpr (DT == VLMCE_F32) {
            return __uint_as_float(r.u[i]);
        } else if constexpr (VEC) {
            float a, b;
            act::unpack16x2(r.u[i / 2], a, b, DT == VLMCE_F16);
            return i & 1 ? b : a;
        } else {
            return act::from16(static_cast<uint16_t>(r.u[i]), DT == VLMCE_F16);
        }
    }

    // values outside the row are 0
    template <int DT>
    __device__ __forceinline__ void load(const unsigned char *row, int64_t H, float (&v)[N]) const {
        if constexpr (VEC) {
            if (c < H) {
                load8<DT>(row, c, v);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = 0.f;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = in(i, H) ? load1<DT>(row, c + 32 * i) : 0.f;
        }
    }
    template <int DT>
    __device__ __forceinline__ void store(unsigned char *row, int64_t H, const float (&v)[N]) const {
        if constexpr (VEC) {
            if (c < H) store8<DT>(row, c, v);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (in(i, H)) store1<DT>(row, c + 32 * i, v[i]);
        }
    }
};

}  // namespace blocks
}  // namespace vlmce
