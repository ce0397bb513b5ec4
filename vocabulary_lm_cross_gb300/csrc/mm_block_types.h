// mm_block_types.h -- the products of e4m3 operands with one scale per block of 128 of K:
// what their host side (mm_block.cu) takes and their kernels' parameters.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "vlmce.h"

namespace vlmce {
namespace mmb {

// y [T, N] = x W^T (+ residual).  x [T, K], weight [groups * N, K]; scales of x [T, K / 128]
// and of the weight [groups * ceil(N / block), K / 128].  offsets: null (one group), or
// [groups + 1], the groups' rows of x.
struct Fwd {
    const void *x, *w;
    int64_t x_ld, w_ld;
    const float *xs, *ws;
    int64_t xs_ld, ws_ld;
    int block;  // 128: a scale for 128 rows of the weight, 1: for each
    const int *offsets;
    int64_t groups, T, N, K;
    const uint16_t *residual;
    int64_t residual_ld;
    uint16_t *y;
    int64_t y_ld;
    int f16;
    int *err;   // null: the device's own word
};
cudaError_t forward(const Fwd &f, cudaStream_t s);

// dw [groups, N, K] = sum over a group's rows of dyt[n, r] xt[k, r]; dyt [N, R] and xt
// [K, R] with scales [N, R / 128] and [K, R / 128].
struct Dw {
    const void *dyt, *xt;
    int64_t dyt_ld, xt_ld;
    const float *dyts, *xts;
    int64_t dyts_ld, xts_ld;
    const int *offsets;
    int64_t groups, R, N, K;
    void *dw;
    int32_t dtype;  // VLMCE_F32, VLMCE_BF16 or VLMCE_F16
    int accumulate;
    int *err;
};
cudaError_t dweight(const Dw &d, cudaStream_t s);

// What forward() would run: vlmce_block_linear_describe_plan.
cudaError_t describe(const Fwd &f, int32_t *out);

struct SmallParams {
    const int *offsets;
    const float *xs, *ws;
    int64_t xs_ld, ws_ld;
    const uint16_t *residual;
    int64_t residual_ld;
    uint16_t *y;
    int64_t y_ld;
    int T, N, groups;
    int block, scale_rows;  // rows of the weight for a scale; scales of a group
    int nt;                 // tiles of 128 weight rows
    int chunks;             // K in blocks
    int split;              // CTAs of a cluster that share a tile's K
    int stages, per_stage;
    int part_offset, factor_offset, table_offset, bar_offset;
    int f16;
    int *err;
};

struct PairParams {
    const int *offsets;
    const float *as, *bs;   // scales of operand A (its rows) and B
    int64_t as_ld, bs_ld;
    const uint16_t *residual;
    int64_t residual_ld;
    void *y;
    int64_t y_ld;
    int T, N, groups;       // forward: rows of x, outputs; dweight: contracted rows, rows of dw
    int K;                  // dweight: columns of dw
    int scale_rows;         // forward: scales of a group's weight
    int nt, mt;             // forward: tiles of 256 outputs; dweight: tiles across and down a dw
    int chunks;             // forward: K in blocks
    int out;                // VLMCE_BF16, VLMCE_F16 or VLMCE_F32
    int add;                // dweight: added to y
    int vec;                // y's rows take TMA stores
    int *err;
};

}  // namespace mmb
}  // namespace vlmce
