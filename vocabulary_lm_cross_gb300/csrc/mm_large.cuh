// mm_large.cuh -- forward product of a linear or gated layer on CTA pairs:
// acc = x W^T on tcgen05 tensor cores, the layer's epilogue fused.
//
// A tile is 256 tokens x 256 weight rows (mm_pair.cuh).  A gated layer's tile
// takes 128 gate rows (staged by the pair's leader) and the 128 up rows of the
// same outputs (staged by its peer), so gate and up of an output meet in one
// thread.  Tensor-bound: T = 4096, K = 6656, 2n = 32768 bf16 911-925 us in a burst
// (1.93-1.96 PFLOP/s, above the measured burst rate of the library), 1043-1062 us back
// to back, where the power cap sets the clock (98-100 % of the library's sustained
// rate); tensor pipe 86 % busy before two chunks made a stage.  Tile order: groups of kGroupM token tiles, weight tiles outer within a
// group, so that the ~76 tiles in flight read about 8 token and 9.5 weight tiles.
#pragma once

#include <cuda.h>

#include "mm_pair.cuh"
#include "mm_types.h"

namespace vlmce {
namespace mm {

constexpr int kGroupM = 8;

struct LargeParams {
    int T, N;          // tokens, outputs
    int up_row;        // gated: first up row of the weight
    int chunks;        // K in 128-byte chunks
    int mt, nt;
    int dealt;
    Epi e;
    int *err;
};

struct LargeTile {
    int m0, n0;
};
template <bool GATED>
__device__ __forceinline__ LargeTile large_tile(const LargeParams &p, int t) {
    const int per_group = kGroupM * p.nt;
    const int g = t / per_group, r = t - g * per_group;
    const int gm = min(kGroupM, p.mt - g * kGroupM);
    const int n = r / gm;
    return {(g * kGroupM + (r - n * gm)) * kPairM, n * (GATED ? 128 : 256)};
}

struct LargeMaps {
    CUtensorMap x, w;          // operands
    CUtensorMap y, z, z_up;    // outputs with 16-byte aligned rows
};

// A warp's accumulators of 32 tokens (one per lane) x 32 outputs from `col`, as z:
// scaled, the bias added.
__device__ __forceinline__ void acc_seg(uint32_t acc, const Epi &e, int col, int scale_col, int N,
                                        float xs, bool bias, float (&v)[32]) {
    uint32_t r[32];
    tc::tmem_ld32(acc, r);
    tc::tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
    if (e.ws) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (col + j < N) v[j] *= xs * e.ws[scale_col + j];
    }
    if (bias && e.bias) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (col + j < N) v[j] += act::from16(e.bias[col + j], e.f16 != 0);
    }
}

template <bool GATED, bool FP8>
__global__ void __launch_bounds__(kPairThreads, 1)
    mm_large_kernel(const __grid_constant__ LargeMaps maps, const __grid_constant__ LargeParams p) {
    constexpr int kPer = 2;
    extern __shared__ unsigned char smem_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        tc::prefetch_tensormap(&maps.x);
        tc::prefetch_tensormap(&maps.w);
    }
    const Pair<kPer> q = pair_setup<kPer>(smem_raw, p.err, p.dealt);
    Tiles tiles;
    const int rank = static_cast<int>(q.rank);

    if (warp == 0 || warp == kWarpB) {
        if (lane == 0) {
            constexpr int kElts = FP8 ? 128 : 64;  // K elements of a 128-byte chunk
            const uint32_t full_leader = ptx::mapa(q.full(0), 0);
            Ring<kPer> r;
            int64_t issued = 0;
            for (int t; (t = tiles.next(q, lane)) >= 0;) {
                const LargeTile tl = large_tile<GATED>(p, t);
                if (warp == 0) {
                    const int ar = tl.m0 + kHalfRows * rank;
                    for (int c = 0; c < p.chunks; c += kPer) {
                        const int n = min(kPer, p.chunks - c);
                        stage_begin<true, kPer>(q, r, n);
                        for (int i = 0; i < n; ++i)
                            tc::tma_load_2d_pair(q.ring + r.s * q.kStageBytes + i * kChunkBytes, &maps.x,
                                                 (c + i) * kElts, ar, full_leader + 8u * r.s);
                        r.next();
                    }
                } else {
                    const int br = GATED ? (rank == 0 ? tl.n0 : p.up_row + tl.n0)
                                         : tl.n0 + kHalfRows * rank;
                    for (int c = 0; c < p.chunks; c += kPer) {
                        const int n = min(kPer, p.chunks - c);
                        stage_begin<false, kPer>(q, r, n);
                        for (int i = 0; i < n; ++i)
                            tc::tma_load_2d_pair(
                                q.ring + r.s * q.kStageBytes + i * kChunkBytes + kOpBytes, &maps.w,
                                (c + i) * kElts, br, full_leader + 8u * r.s);
                        r.next();
                    }
                }
                issued += (p.chunks + kPer - 1) / kPer;
            }
            if (warp == 0) drain_loads(q, issued);
        }
    } else if (warp == 1) {
        if (rank == 0 && lane == 0) {
            const uint32_t idesc = tc::idesc_bf16_f32(256, 256, false, false, FP8 || p.e.f16);
            Ring<kPer> r;
            int it = 0;
            for (; tiles.next(q, lane) >= 0; ++it)
                mma_tile<FP8, kPer>(q, r, it, p.chunks, idesc, false, false);
            mma_finish(q);
        }
    } else if (warp == kWarpTiles) {
        if (rank == 0 && lane == 0) fetch_tiles(q);
    } else {
        const int half = (warp - 2) >> 2;
        uint32_t *buf = q.out_buffer(warp - 2);
        const uint32_t tempty_leader = ptx::mapa(q.tempty(0), 0);
        const Epi &e = p.e;
        const bool f16 = e.f16 != 0;
        const Out y = {e.y, e.y_ld, e.y_vec, &maps.y};
        const Out z = {e.preact, e.preact_ld, e.preact_vec, &maps.z};
        const Out z_up = {e.preact + p.N, e.preact_ld, e.preact_up_vec, &maps.z_up};
        const bool staged = y.vec < 16;  // y's segments leave the buffer empty
        int it = 0;
        for (int t; (t = tiles.next(q, lane)) >= 0; ++it) {
            const LargeTile tl = large_tile<GATED>(p, t);
            const int64_t row0 = tl.m0 + kHalfRows * rank + (warp & 3) * 32;
            const float xs = e.xs && row0 + lane < p.T ? e.xs[row0 + lane] : 1.f;
            const uint32_t acc = acc_wait(q, it, warp);
            // 64 columns at a time: one group of a gated tile's 128 outputs per
            // half, two of a linear tile's 256
            constexpr int kGroups = GATED ? 1 : 2;
#pragma unroll 1
            for (int g = kGroups * half; g < kGroups * (half + 1); ++g) {
                const int col = tl.n0 + 64 * g;
                if (col >= p.N || row0 >= p.T) continue;
                if (e.preact) {
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        float v[32];
                        const int c = col + 32 * h;
                        acc_seg(acc + 64 * g + 32 * h, e, c, c, p.N, xs, !GATED, v);
                        put_seg(z, row0, col, h, v, p.T, p.N, f16, buf, lane);
                    }
                    if constexpr (GATED) {
#pragma unroll 1
                        for (int h = 0; h < 2; ++h) {
                            float v[32];
                            const int c = col + 32 * h;
                            acc_seg(acc + 128 + 64 * g + 32 * h, e, c, p.up_row + c, p.N, xs,
                                    false, v);
                            put_seg(z_up, row0, col, h, v, p.T, p.N, f16, buf, lane);
                        }
                    }
                }
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    float v[32];
                    const int c = col + 32 * h;
                    acc_seg(acc + 64 * g + 32 * h, e, c, c, p.N, xs, !GATED, v);
                    act::apply_n(v, e.act);
                    if constexpr (GATED) {
                        float u[32];
                        acc_seg(acc + 128 + 64 * g + 32 * h, e, c, p.up_row + c, p.N, xs, false, u);
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] *= u[j];
                    } else if (e.residual) {
                        add_seg(e.residual, e.residual_ld, e.residual_vec, row0, c, v, p.T, p.N,
                                f16, staged, buf, lane);
                    }
                    __syncwarp();
                    put_seg(y, row0, col, h, v, p.T, p.N, f16, buf, lane);
                }
            }
            acc_release(tempty_leader, it, lane);
        }
        if (lane == 0) tc::bulk_wait();
    }
    pair_teardown(q);
}

}  // namespace mm
}  // namespace vlmce
