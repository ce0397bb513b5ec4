// act.cuh -- the activations of the linear and gated layers and their
// derivatives in fp32, and 16-bit element access (bf16 or fp16 at run time).
//
//   silu       a s(a)                       s(a) = 1 / (1 + e^-a)
//   gelu       a P(a)                       P(a) = erfc(-a / sqrt 2) / 2, the normal CDF
//   gelu_tanh  a s(2 c0 (a + c1 a^3))       (1 + tanh v) / 2 = s(2 v); c0 = sqrt(2/pi), c1 = 0.044715
//   relu       max(a, 0), NaN kept
//
// erfc keeps the relative accuracy of P for negative a, where 1 + erf cancels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "ptx.cuh"
#include "vlmce.h"

namespace vlmce {
namespace act {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kC0x2 = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kC1 = 0.044715f;

__device__ __forceinline__ float sigmoid(float a) {
    return ptx::rcp(1.f + ptx::ex2(-a * kLog2e));
}
__device__ __forceinline__ float cdf(float a) { return 0.5f * erfcf(-0.70710678f * a); }

template <int ACT>
__device__ __forceinline__ float fwd(float a) {
    if constexpr (ACT == VLMCE_ACT_SILU) return a * sigmoid(a);
    if constexpr (ACT == VLMCE_ACT_GELU) return a * cdf(a);
    if constexpr (ACT == VLMCE_ACT_GELU_TANH)
        return a * sigmoid(kC0x2 * fmaf(kC1 * a * a, a, a));
    if constexpr (ACT == VLMCE_ACT_RELU) return a < 0.f ? 0.f : a;
    return a;
}

// f = act(a), d = act'(a).  The polynomial factors are evaluated on a clamped
// to +-30, beyond which every derivative is 0 or 1 in fp32, so that an
// overflowing a^2 never meets a factor of 0.
template <int ACT>
__device__ __forceinline__ void fwd_bwd(float a, float &f, float &d) {
    const float c = fminf(fmaxf(a, -30.f), 30.f);
    if constexpr (ACT == VLMCE_ACT_SILU) {
        const float s = sigmoid(a);
        f = a * s;
        d = fmaf(c * s, 1.f - s, s);
    } else if constexpr (ACT == VLMCE_ACT_GELU) {
        const float p = cdf(a);
        f = a * p;
        d = fmaf(c, 0.3989422804f * ptx::ex2(-0.5f * kLog2e * c * c), p);
    } else if constexpr (ACT == VLMCE_ACT_GELU_TANH) {
        const float s = sigmoid(kC0x2 * fmaf(kC1 * a * a, a, a));
        f = a * s;
        d = fmaf(c * s * (1.f - s), kC0x2 * fmaf(3.f * kC1 * c, c, 1.f), s);
    } else if constexpr (ACT == VLMCE_ACT_RELU) {
        f = a < 0.f ? 0.f : a;
        d = a > 0.f ? 1.f : 0.f;
    } else {
        f = a;
        d = 1.f;
    }
}

// act(a) with the activation chosen at run time (uniform over the grid).
__device__ __forceinline__ float apply(float a, int kind) {
    switch (kind) {
        case VLMCE_ACT_SILU: return fwd<VLMCE_ACT_SILU>(a);
        case VLMCE_ACT_GELU: return fwd<VLMCE_ACT_GELU>(a);
        case VLMCE_ACT_GELU_TANH: return fwd<VLMCE_ACT_GELU_TANH>(a);
        case VLMCE_ACT_RELU: return fwd<VLMCE_ACT_RELU>(a);
        default: return a;
    }
}
template <int N>
__device__ __forceinline__ void apply_n(float (&v)[N], int kind) {
    switch (kind) {
#define VLMCE_ACT_CASE(A)                                  \
    case A: {                                              \
        _Pragma("unroll") for (int j = 0; j < N; ++j) v[j] = fwd<A>(v[j]); \
        break;                                             \
    }
        VLMCE_ACT_CASE(VLMCE_ACT_SILU)
        VLMCE_ACT_CASE(VLMCE_ACT_GELU)
        VLMCE_ACT_CASE(VLMCE_ACT_GELU_TANH)
        VLMCE_ACT_CASE(VLMCE_ACT_RELU)
#undef VLMCE_ACT_CASE
        default: break;
    }
}

// ------------------------------------------------------------ 16-bit elements
__device__ __forceinline__ float from16(uint16_t u, bool f16) {
    return f16 ? __half2float(__ushort_as_half(u))
               : __uint_as_float(static_cast<uint32_t>(u) << 16);
}
__device__ __forceinline__ uint16_t to16(float a, bool f16) {
    return f16 ? __half_as_ushort(__float2half_rn(a))
               : __bfloat16_as_ushort(__float2bfloat16_rn(a));
}
__device__ __forceinline__ uint32_t pack16x2(float a, float b, bool f16) {
    uint32_t u;
    if (f16) {
        const __half2 v = __floats2half2_rn(a, b);
        memcpy(&u, &v, 4);
    } else {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        memcpy(&u, &v, 4);
    }
    return u;
}
__device__ __forceinline__ void unpack16x2(uint32_t u, float &a, float &b, bool f16) {
    if (f16) {
        __half2 h;
        memcpy(&h, &u, 4);
        const float2 f = __half22float2(h);
        a = f.x;
        b = f.y;
    } else {
        a = __uint_as_float(u << 16);
        b = __uint_as_float(u & 0xffff0000u);
    }
}

}  // namespace act
}  // namespace vlmce
