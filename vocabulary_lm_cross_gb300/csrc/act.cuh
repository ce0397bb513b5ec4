// act.cuh -- the activations of the linear and gated layers and their
// derivatives in fp32, and 16-bit element access (bf16 or fp16 at run time).
//
//   silu       a s(a)                       s(a) = 1 / (1 + e^-a)
//   gelu       a P(a)                       P: the normal CDF
//   gelu_tanh  a s(2 c0 (a + c1 a^3))       (1 + tanh v) / 2 = s(2 v); c0 = sqrt(2/pi), c1 = 0.044715
//   relu       max(a, 0), NaN kept
//
// P(-x) = e^(-x^2/2) R(x) / 2 for x >= 0, with the scaled complementary error
// function R(x) = e^(x^2/2) erfc(x / sqrt 2) as t p(t), t = 1 / (1 + 0.3 x / sqrt 2)
// and p of degree 8: a least-squares fit, reweighted towards the smallest largest
// relative error (6e-8 with the coefficients below, for x <= 13.4, beyond which
// e^(-x^2/2) is 0 in fp32).  So the relative accuracy holds for negative a too (1 + erf
// would cancel; 9e-7 for a > -4, 8e-6 for a > -13 in fp32), one exponential serves P and
// its derivative, and there is no branch (T 1007, K 1000, N 777 in the small kernel with
// erfcf 15.1 us, so 13.9).
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
// P(a) and e^(-a^2/2).
__device__ __forceinline__ float cdf(float a, float &e) {
    e = ptx::ex2(-0.5f * kLog2e * a * a);
    const float t = ptx::rcp(fmaf(0.3f * 0.70710678f, fabsf(a), 1.f));
    float p = -0.12943436f;
    p = fmaf(p, t, 0.48509780f);
    p = fmaf(p, t, -0.51122928f);
    p = fmaf(p, t, 0.54639840f);
    p = fmaf(p, t, -0.09363360f);
    p = fmaf(p, t, 0.21443731f);
    p = fmaf(p, t, 0.14848216f);
    p = fmaf(p, t, 0.17069197f);
    p = fmaf(p, t, 0.16918962f);
    const float q = 0.5f * t * p * e;
    return a < 0.f ? q : 1.f - q;
}

template <int ACT>
__device__ __forceinline__ float fwd(float a) {
    if constexpr (ACT == VLMCE_ACT_SILU) return a * sigmoid(a);
    if constexpr (ACT == VLMCE_ACT_GELU) {
        float e;
        return a * cdf(a, e);
    }
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
        float e;
        const float p = cdf(a, e);
        f = a * p;
        d = fmaf(c, 0.3989422804f * e, p);
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

// act(v) with the activation chosen at run time (uniform over the grid).
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
