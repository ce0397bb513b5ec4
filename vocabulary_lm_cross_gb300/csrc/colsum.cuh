// colsum.cuh -- out[j] (+)= sum over q of part[q][j], in a fixed order: the last
// step of the weight and bias gradients, whose CTAs each leave one row of partial
// sums.  Latency-bound: 32 warps per 32 columns, each with its share of the rows
// in flight at once.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace vlmce {
namespace colsum {

constexpr int kWarps = 32;

struct Params {
    const float *part;  // [rows][cols]
    float *out;         // [cols]
    int64_t cols;
    int rows, accumulate;
};

template <int WARPS>
__global__ void __launch_bounds__(32 * WARPS) kernel(const Params p) {
    __shared__ float sh[WARPS][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t j = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    float a = 0.f;
    if (j < p.cols) {
#pragma unroll 8
        for (int q = warp; q < p.rows; q += WARPS) a += p.part[q * p.cols + j];
    }
    sh[warp][lane] = a;
    __syncthreads();
    if (warp == 0 && j < p.cols) {
        a = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) a += sh[w][lane];
        p.out[j] = p.accumulate ? p.out[j] + a : a;
    }
}

inline unsigned blocks(int64_t cols) { return static_cast<unsigned>((cols + 31) / 32); }

}  // namespace colsum
}  // namespace vlmce
