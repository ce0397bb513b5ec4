// mm_types.h -- launch parameters of the matrix-product kernels of the linear
// and gated layers (mm_large.cuh: CTA pairs on 256 x 256 tiles; mm_small.cuh:
// single CTAs on 128 weight rows x few tokens) and their host entry points.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "vlmce.h"

namespace vlmce {
namespace mm {

// What a forward epilogue does with an accumulator acc[t, n]:
//   z = acc xs[t] ws[n] + bias[n];  preact[t, n] = z;
//   y[t, n] = act(z) + residual[t, n]                        (linear)
//   g, u = the two accumulators of column n, scaled likewise;
//   preact[t, n], preact[t, n_out + n] = g, u;  y[t, n] = act(g) u   (gated)
// in fp32, each output rounded once to 16 bits.  Null pointers leave a step out.
struct Epi {
    uint16_t *y;
    int64_t y_ld;
    uint16_t *preact;
    int64_t preact_ld;
    const uint16_t *bias;
    const uint16_t *residual;
    int64_t residual_ld;
    const float *xs, *ws;
    int act, f16;
    // vec_of() of the tensors
    int y_vec, preact_vec, preact_up_vec;
};

// One forward product: x [T, K], weight [N, K] (gated: [2N, K]).
struct Fwd {
    const void *x, *w;
    int64_t x_ld, w_ld;
    int64_t T, N, K;
    int gated;
    int w_mn;       // the weight is stored [K, N] (small kernel, 16 bits, not gated)
    int32_t dtype;  // VLMCE_BF16, VLMCE_F16 or VLMCE_E4M3
    Epi e;
    int *err;       // null: the device's own word
};

// Enqueue it (T, N, K >= 1); the kernel is chosen by the sizes.
cudaError_t forward(const Fwd &f, cudaStream_t s);

// The gradient products from dz [T, rows] (dz_ld a multiple of 8 elements, 16-bit
// type of x and w, 16-byte aligned): dx [T, K] = dz W and dw [rows, K] = dz^T x,
// either may be null.
struct Bwd {
    const void *dz, *x, *w;
    int64_t dz_ld, x_ld, w_ld;
    int64_t T, rows, K;
    int f16;
    void *dx;
    int64_t dx_ld;
    void *dw;              // [rows, K] contiguous
    int dw_f32, accumulate;
    int *err;              // null: the device's own word
};
cudaError_t backward(const Bwd &b, cudaStream_t s);

// The launches that forward() and backward() (dx and dw) would make for these sizes
// and types, in the words of vlmce_linear_describe_plan.
cudaError_t describe(const Fwd &f, int32_t *out);
cudaError_t describe(const Bwd &b, int32_t *out);

// Bytes (16 or 2) an access to 32 consecutive 16-bit columns of a row may use; 16
// also means that a tensor map can describe the rows (their whole granules of 16 bytes).
inline int vec_of(const void *p, int64_t ld, int64_t cols) {
    const uint64_t a = reinterpret_cast<uint64_t>(p) | static_cast<uint64_t>(2 * ld);
    return a % 16 == 0 && ld < (int64_t{1} << 39) && cols >= 8 ? 16 : 2;
}

}  // namespace mm
}  // namespace vlmce
