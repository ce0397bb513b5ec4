// mm_large.cuh -- forward product of a linear or gated layer on CTA pairs:
// acc = x W^T on tcgen05 tensor cores, the layer's epilogue fused.
//
// A tile is 256 tokens x 256 weight rows (mm_pair.cuh).  A gated layer's tile
// takes 128 gate rows (staged by the pair's leader) and the 128 up rows of the
// same outputs (staged by its peer), so gate and up of an output meet in one
// thread.  Tile order: groups of kGroupM token tiles, weight tiles outer within a
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

__device__ __forceinline__ void scale32(float (&v)[32], float xs, const float *ws, int nc) {
#pragma unroll
    for (int j = 0; j < 32; ++j)
        if (j < nc) v[j] *= xs * ws[j];
}

// Epilogue of a warp's 32 tokens from row0 x 32 outputs from col (Epi in
// mm_types.h), one token per lane.
__device__ __forceinline__ void linear_seg(const LargeParams &p, const uint32_t (&r)[32], int64_t row0,
                                           int col, float xs, uint32_t *stage, int lane) {
    const Epi &e = p.e;
    const bool f16 = e.f16 != 0;
    const int nr = static_cast<int>(min(int64_t{32}, p.T - row0)), nc = min(32, p.N - col);
    float v[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
    if (e.ws) scale32(v, xs, e.ws + col, nc);
    if (e.bias) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (j < nc) v[j] += act::from16(e.bias[col + j], f16);
    }
    if (e.preact)
        store_seg(e.preact + row0 * e.preact_ld + col, e.preact_ld, v, nr, nc, e.preact_vec, f16,
                  stage, lane);
    act::apply_n(v, e.act);
    if (e.residual)
        add_seg(e.residual + row0 * e.residual_ld + col, e.residual_ld, v, nr, nc, e.residual_vec,
                f16, stage, lane);
    store_seg(e.y + row0 * e.y_ld + col, e.y_ld, v, nr, nc, e.y_vec, f16, stage, lane);
}
__device__ __forceinline__ void gated_seg(const LargeParams &p, const uint32_t (&rg)[32],
                                          const uint32_t (&ru)[32], int64_t row0, int col,
                                          float xs,
                                          uint32_t *stage, int lane) {
    const Epi &e = p.e;
    const bool f16 = e.f16 != 0;
    const int nr = static_cast<int>(min(int64_t{32}, p.T - row0)), nc = min(32, p.N - col);
    float g[32], u[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        g[j] = __uint_as_float(rg[j]);
        u[j] = __uint_as_float(ru[j]);
    }
    if (e.ws) {
        scale32(g, xs, e.ws + col, nc);
        scale32(u, xs, e.ws + p.up_row + col, nc);
    }
    if (e.preact) {
        uint16_t *z = e.preact + row0 * e.preact_ld + col;
        store_seg(z, e.preact_ld, g, nr, nc, e.preact_vec, f16, stage, lane);
        store_seg(z + p.N, e.preact_ld, u, nr, nc, e.preact_up_vec, f16, stage, lane);
    }
    act::apply_n(g, e.act);
#pragma unroll
    for (int j = 0; j < 32; ++j) g[j] *= u[j];
    store_seg(e.y + row0 * e.y_ld + col, e.y_ld, g, nr, nc, e.y_vec, f16, stage, lane);
}

template <bool GATED, bool FP8>
__global__ void __launch_bounds__(kPairThreads, 1)
    mm_large_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
                    const __grid_constant__ LargeParams p) {
    constexpr int kPer = 2;
    extern __shared__ unsigned char smem_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        tc::prefetch_tensormap(&mx);
        tc::prefetch_tensormap(&mw);
    }
    const Pair<kPer> q = pair_setup<kPer>(smem_raw, p.err);
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
                            tc::tma_load_2d_pair(q.ring + r.s * q.kStageBytes + i * kChunkBytes, &mx,
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
                                q.ring + r.s * q.kStageBytes + i * kChunkBytes + kOpBytes, &mw,
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
        uint32_t *stage = q.stage_words(warp - 2);
        const uint32_t tempty_leader = ptx::mapa(q.tempty(0), 0);
        int it = 0;
        for (int t; (t = tiles.next(q, lane)) >= 0; ++it) {
            const LargeTile tl = large_tile<GATED>(p, t);
            const int64_t row0 = tl.m0 + kHalfRows * rank + (warp & 3) * 32;
            const float xs = p.e.xs && row0 + lane < p.T ? p.e.xs[row0 + lane] : 1.f;
            const uint32_t acc = acc_wait(q, it, warp);
            if constexpr (GATED) {
#pragma unroll 1
                for (int c = 2 * half; c < 2 * half + 2; ++c) {
                    uint32_t rg[32], ru[32];
                    tc::tmem_ld32(acc + 32 * c, rg);
                    tc::tmem_ld32(acc + 128 + 32 * c, ru);
                    tc::tmem_ld_wait();
                    const int col = tl.n0 + 32 * c;
                    if (col < p.N && row0 < p.T)
                        gated_seg(p, rg, ru, row0, col, xs, stage, lane);
                    __syncwarp();
                }
            } else {
#pragma unroll 1
                for (int c = 4 * half; c < 4 * half + 4; ++c) {
                    uint32_t r[32];
                    tc::tmem_ld32(acc + 32 * c, r);
                    tc::tmem_ld_wait();
                    const int col = tl.n0 + 32 * c;
                    if (col < p.N && row0 < p.T) linear_seg(p, r, row0, col, xs, stage, lane);
                    __syncwarp();
                }
            }
            acc_release(tempty_leader, it, lane);
        }
    }
    pair_teardown(q);
}

}  // namespace mm
}  // namespace vlmce
