// mm_block.cuh -- what the products of operands with one scale per block of 128 share
// (mm_block_small.cuh, mm_block_pair.cuh): their sizes, the experts' tiles, and the
// factors of an accumulator.
//
//   y[t, n] = sum_b xs[t, b] ws[n, b] sum_{k in block b} x[t, k] w[n, k]
//
// The factors change with every 128 of K, so the tensor core's sum over a block (four
// tcgen05.mma of K = 32) is taken out of TMEM, and the sum over the blocks is kept in
// registers: acc += (xs ws) d in fp32, while the tensor core works on the next block in
// another TMEM buffer.
//
// With experts, rows offsets[e] .. offsets[e + 1] of x meet weight e (`groups` of them;
// without, one group of all rows).  How many tiles there are is known on the device only:
// every CTA sums them over the experts, and finds a tile's expert by bisection.
#pragma once

#include <cuda.h>

#include "mbar_wait.cuh"
#include "mm_block_types.h"
#include "ptx_async.cuh"
#include "tcgen05.cuh"

namespace vlmce {
namespace mmb {

// ------------------------------------------------------------ the groups' tiles
// In shared memory: for each group its rows and the tiles of `step` rows before it.
struct Table {
    int *tile0;  // [groups + 1]
    int *row0, *row1;
};
constexpr int table_bytes(int groups) { return 4 * (3 * groups + 1); }
__device__ __forceinline__ Table table_at(unsigned char *p, int groups) {
    Table t;
    t.tile0 = reinterpret_cast<int *>(p);
    t.row0 = t.tile0 + groups + 1;
    t.row1 = t.row0 + groups;
    return t;
}
// All threads.  Offsets outside [0, rows] or descending, or (`whole` > 1) not its multiples
// but for `rows` itself, are reported, and every group is empty then.
__device__ __forceinline__ void table_fill(const Table &t, const int *offsets, int groups, int rows,
                                           int step, int whole, int *err) {
    if (!offsets) {
        if (threadIdx.x == 0) {
            t.row0[0] = 0;
            t.row1[0] = rows;
            t.tile0[0] = 0;
            t.tile0[1] = (rows + step - 1) / step;
        }
        __syncthreads();
        return;
    }
    bool bad = false;
    for (int e = threadIdx.x; e < groups; e += blockDim.x) {
        const int a = offsets[e], b = offsets[e + 1];
        bad |= a < 0 || b < a || b > rows || a % whole != 0 || (b % whole != 0 && b != rows);
        t.row0[e] = a;
        t.row1[e] = b;
    }
    if (__syncthreads_or(bad)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(err, VLMCE_DEVERR_OFFSETS);
        for (int e = threadIdx.x; e < groups; e += blockDim.x) t.row0[e] = t.row1[e] = 0;
        __syncthreads();
    }
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int before = 0;
        for (int e0 = 0; e0 < groups; e0 += 32) {
            const int e = e0 + lane;
            const int n = e < groups ? (t.row1[e] - t.row0[e] + step - 1) / step : 0;
            int sum = n;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int v = __shfl_up_sync(0xffffffffu, sum, d);
                if (lane >= d) sum += v;
            }
            if (e < groups) t.tile0[e] = before + sum - n;
            before += __shfl_sync(0xffffffffu, sum, 31);
        }
        if (lane == 0) t.tile0[groups] = before;
    }
    __syncthreads();
}
// The group that the `at`-th tile of rows belongs to (tile0[g] <= at < tile0[g + 1]).
__device__ __forceinline__ int group_of(const Table &t, int groups, int at) {
    int lo = 0, hi = groups;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (t.tile0[mid] <= at)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

}  // namespace mmb
}  // namespace vlmce
