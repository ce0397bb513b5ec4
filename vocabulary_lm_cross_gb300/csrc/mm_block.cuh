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

#include "f32x2.cuh"
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
    int *row;    // [groups + 1]: a group's rows end where the next one's start
};
constexpr int table_bytes(int groups) { return 8 * (groups + 1); }
__device__ __forceinline__ Table table_at(unsigned char *p, int groups) {
    Table t;
    t.tile0 = reinterpret_cast<int *>(p);
    t.row = t.tile0 + groups + 1;
    return t;
}
// All threads.  Offsets outside [0, rows] or descending, or (`whole` > 1) not its multiples
// but for `rows` itself, are reported, and every group is empty then.
__device__ __forceinline__ void table_fill(const Table &t, const int *offsets, int groups, int rows,
                                           int step, int whole, int *err) {
    if (!offsets) {
        if (threadIdx.x == 0) {
            t.row[0] = 0;
            t.row[1] = rows;
            t.tile0[0] = 0;
            t.tile0[1] = (rows + step - 1) / step;
        }
        __syncthreads();
        return;
    }
    bool bad = false;
    for (int e = threadIdx.x; e <= groups; e += blockDim.x) {
        const int b = offsets[e], a = e > 0 ? offsets[e - 1] : 0;
        bad |= a < 0 || b < a || b > rows || (b % whole != 0 && b != rows);
        t.row[e] = b;
    }
    if (__syncthreads_or(bad)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(err, VLMCE_DEVERR_OFFSETS);
        for (int e = threadIdx.x; e <= groups; e += blockDim.x) t.row[e] = 0;
        __syncthreads();
    }
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int before = 0;
        for (int e0 = 0; e0 < groups; e0 += 32) {
            const int e = e0 + lane;
            const int n = e < groups ? (t.row[e + 1] - t.row[e] + step - 1) / step : 0;
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

// ------------------------------------------------------------ factors
// A warp of its own brings the factors into shared memory, four blocks at a time and up to
// eight ahead: behind the operands' copies an answer takes thousands of clocks (fetched into
// registers two blocks ahead, T 4096, K 4096, N 4096 took 151 us).  Its lanes take four
// blocks of eight rows, so that an access covers eight lines of memory (with 32 rows of one
// block, 32 lines kept the load unit busy for 60 clocks), and rows of the ring are 8 words
// apart from a multiple of 32, so that they write to 32 banks.
constexpr int kFactorBatch = 4;
constexpr int kFactorSlots = 3;  // batches
constexpr int kFactorBarBytes = 16 * kFactorSlots;
// Words of a block's factors: n of them.
constexpr int factor_words(int n) { return (n + 31) / 32 * 32 + 8; }

struct Factors {
    uint32_t slots, bars;  // shared-memory addresses
    int words;             // of a block
    __device__ __forceinline__ uint32_t full(int s) const { return bars + 8u * s; }
    __device__ __forceinline__ uint32_t empty(int s) const { return bars + 8u * (kFactorSlots + s); }
    __device__ __forceinline__ uint32_t at(int s) const {
        return slots + static_cast<uint32_t>(4 * kFactorBatch * s * words);
    }
    // one thread, before the CTA's barrier
    __device__ __forceinline__ void init(int readers) const {
        for (int s = 0; s < kFactorSlots; ++s) {
            ptx::mbar_init(full(s), 32);        // every lane's copies
            ptx::mbar_init(empty(s), readers);  // warps
        }
    }
};
// Position in the ring of batches.
struct Slot {
    int s = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next() {
        if (++s == kFactorSlots) {
            s = 0;
            ph ^= 1;
        }
    }
};
// Four blocks' (those of the first `blocks`) factors of N (a multiple of 8) rows from `first`
// of base [.., ld], the rows from `count` on as 0; `dst`: where the first block's go.
template <int N>
__device__ __forceinline__ void factors_copy(uint32_t dst, int words, const float *base, int64_t first, int64_t ld,
                                             int count, int blocks, int lane) {
    const int k = lane & 3, r = lane >> 2;
    const float *src = base + (first + r) * ld + k;
    const uint32_t to = dst + 4u * (k * words + r);
    const int64_t step = 8 * ld;
#pragma unroll 4
    for (int j = 0; j < N; j += 8, src += step) {
        const bool in = k < blocks && j + r < count;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to + 4u * j), "l"(in ? src : base),
                     "r"(in ? 4 : 0)
                     : "memory");
    }
}
__device__ __forceinline__ void factors_done(const Factors &f, int s) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(f.full(s)) : "memory");
}

}  // namespace mmb
}  // namespace vlmce
