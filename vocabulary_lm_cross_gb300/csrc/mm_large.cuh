// mm_large.cuh -- forward product of a linear or gated layer on CTA pairs:
// acc = x W^T on tcgen05 tensor cores, the layer's epilogue fused.
//
// A tile is 256 tokens x 256 weight rows (mm_pair.cuh).  A gated layer's tile
// takes 128 gate rows (staged by the pair's leader) and the 128 up rows of the
// same outputs (staged by its peer), so gate and up of an output meet in one
// thread.  Tensor-bound: T = 4096, K = 6656, 2n = 32768 bf16 902-940 us in a burst
// (1.90-1.98 PFLOP/s, the measured burst rate of the library), 1048-1086 us back to
// back, where the power cap sets the clock (96-100 % of the library's sustained rate);
// tensor pipe 93 % busy (86 % before two chunks made a stage).  Tile order: groups of kGroupM
// token tiles, weight tiles outer within a group, so that the ~76 tiles in flight read
// about 8 token and 9.5 weight tiles.
// `narrow` tiles have 128 weight rows (gated: 64 + 64), and four stages of the ring.
//
// The epilogue asks for what it reads from memory (scales, bias, residual) before it
// waits for a tile's accumulators, the residual's next 64 columns while it works on the
// present ones: behind the ring's copies an answer takes thousands of clocks (T 8192,
// K 2048, N 2048 bf16 with bias, preact and residual 61.3 us, asked for where used 89;
// N 2049 88.1 and 260).
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
    int narrow;        // tiles of 128 weight rows instead of 256
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
    return {(g * kGroupM + (r - n * gm)) * kPairM, n * ((GATED ? 128 : 256) >> p.narrow)};
}

struct LargeMaps {
    CUtensorMap x, w;          // operands
    CUtensorMap y, z, z_up;    // outputs with 16-byte aligned rows
};

// A warp's accumulators of 32 tokens (one per lane) x 32 outputs, as z: scaled, the
// bias added; lane j has output j's scale and bias.
__device__ __forceinline__ void acc_seg(uint32_t acc, bool scaled, float xs, float ws, bool biased,
                                        float bias, float (&v)[32]) {
    uint32_t r[32];
    tc::tmem_ld32(acc, r);
    tc::tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
    if (scaled) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] *= xs * __shfl_sync(0xffffffffu, ws, j);
    }
    if (biased) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] += __shfl_sync(0xffffffffu, bias, j);
    }
}

template <bool GATED, bool FP8, bool ADD>
__global__ void __launch_bounds__(kPairThreads, 1)
    mm_large_kernel(const __grid_constant__ LargeMaps maps, const __grid_constant__ LargeParams p) {
    constexpr int kPer = 2;
    extern __shared__ unsigned char smem_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        tc::prefetch_tensormap(&maps.x);
        tc::prefetch_tensormap(&maps.w);
    }
    const Pair<kPer> q = pair_setup<kPer>(smem_raw, p.err, p.dealt,
                                          kOpBytes + (kOpBytes >> p.narrow));
    Tiles tiles;
    const int rank = static_cast<int>(q.rank);

    if (warp == 0 || warp == kWarpB) {
        if (lane == 0) {
            constexpr int kElts = FP8 ? 128 : 64;  // K elements of a 128-byte chunk
            const uint32_t full_leader = ptx::mapa(q.full(0), 0);
            Ring<kPer> r;
            int64_t issued = 0;
            for (int t; (t = tiles.next<false>(q, lane)) >= 0;) {
                const LargeTile tl = large_tile<GATED>(p, t);
                if (warp == 0) {
                    const int ar = tl.m0 + kHalfRows * rank;
                    for (int c = 0; c < p.chunks; c += kPer) {
                        const int n = min(kPer, p.chunks - c);
                        stage_begin<true, kPer>(q, r, n);
                        for (int i = 0; i < n; ++i)
                            tc::tma_load_2d_pair(q.chunk(r.s, i), &maps.x,
                                                 (c + i) * kElts, ar, full_leader + 8u * r.s);
                        r.next(q);
                    }
                } else {
                    const int br = GATED ? (rank == 0 ? tl.n0 : p.up_row + tl.n0)
                                         : tl.n0 + (kHalfRows >> p.narrow) * rank;
                    for (int c = 0; c < p.chunks; c += kPer) {
                        const int n = min(kPer, p.chunks - c);
                        stage_begin<false, kPer>(q, r, n);
                        for (int i = 0; i < n; ++i)
                            tc::tma_load_2d_pair(
                                q.chunk(r.s, i) + kOpBytes, &maps.w,
                                (c + i) * kElts, br, full_leader + 8u * r.s);
                        r.next(q);
                    }
                }
                issued += (p.chunks + kPer - 1) / kPer;
            }
            if (warp == 0) drain_loads(q, issued);
        }
    } else if (warp == 1) {
        if (rank == 0 && lane == 0) {
            const uint32_t idesc = tc::idesc_bf16_f32(256, 256 >> p.narrow, false, false,
                                                     FP8 || p.e.f16);
            Ring<kPer> r;
            int it = 0;
            for (; tiles.next<false>(q, lane) >= 0; ++it)
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
        const bool ragged = (p.N & 7) != 0;  // rows end inside a granule
        const Out y = {e.y, e.y_ld, e.y_vec, &maps.y};
        const Out z = {e.preact, e.preact_ld, e.preact_vec, &maps.z};
        const Out z_up = {e.preact + p.N, e.preact_ld, e.preact_up_vec, &maps.z_up};
        int it = 0;
        for (int t; (t = tiles.next<true>(q, lane)) >= 0; ++it) {
            const LargeTile tl = large_tile<GATED>(p, t);
            const int64_t row0 = tl.m0 + kHalfRows * rank + (warp & 3) * 32;
            // 64 columns at a time: one group of a gated tile's 128 outputs per
            // half of the warps, two of a linear tile's 256; of a narrow tile one of
            // 128, and a gated one's 64 outputs are one half's, in turn
            const bool idle = GATED && p.narrow && (it & 1) != half;
            const int groups = GATED || p.narrow ? 1 : 2;
            const int part = GATED && p.narrow ? 0 : 64 * groups * half;
            const int col0 = tl.n0 + part;
            // what the outputs take from memory comes while the tile's sums do
            const float xs = e.xs && row0 + lane < p.T ? e.xs[row0 + lane] : 1.f;
            float ws[4], bias[4];  // of columns col0 + 32 i + lane (gated: two of gate, two of up)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = col0 + 32 * (GATED ? i & 1 : i) + lane;
                const int up = GATED && i >= 2 ? p.up_row : 0;
                ws[i] = FP8 && c < p.N ? e.ws[up + c] : 1.f;
                bias[i] = !GATED && e.bias && c < p.N ? act::from16(e.bias[c], f16) : 0.f;
            }
            RowFetch next;
            if constexpr (ADD)
                fetch_row(e.residual, e.residual_ld, row0 + lane, col0, p.T, p.N, next);
            const uint32_t acc = acc_wait(q, it, warp) + part;
#pragma unroll 1
            for (int g = 0; g < groups; ++g) {
                const int col = col0 + 64 * g;
                if (col >= p.N || row0 >= p.T || idle) break;
                uint32_t add[32];
                bool whole = false;
                if constexpr (ADD) {
                    whole = next.whole;
                    align_row(next, add);
                    if (g + 1 < groups)
                        fetch_row(e.residual, e.residual_ld, row0 + lane, col + 64, p.T, p.N, next);
                }
                auto z_seg = [&](int h, float (&v)[32]) {
                    acc_seg(acc + 64 * g + 32 * h, FP8, xs, h ? ws[1] : ws[0],
                            !GATED && e.bias, h ? bias[1] : bias[0], v);
                };
                auto up_seg = [&](int h, float (&v)[32]) {
                    acc_seg(acc + (128 >> p.narrow) + 32 * h, FP8, xs, h ? ws[3] : ws[2], false, 0.f, v);
                };
                if (e.preact) {
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        float v[32];
                        z_seg(h, v);
                        put_seg(z, row0, col, h, v, p.T, p.N, f16, buf, lane);
                    }
                    if (ragged) put_rest(z, row0, col, p.T, p.N, buf, lane);
                    if constexpr (GATED) {
#pragma unroll 1
                        for (int h = 0; h < 2; ++h) {
                            float v[32];
                            up_seg(h, v);
                            put_seg(z_up, row0, col, h, v, p.T, p.N, f16, buf, lane);
                        }
                    }
                }
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    float v[32];
                    z_seg(h, v);
                    act::apply_n(v, e.act);
                    if constexpr (GATED) {
                        float u[32];
                        up_seg(h, u);
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] *= u[j];
                    }
                    if constexpr (ADD) {
                        const int c = col + 32 * h;
                        if (whole) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                float a, b;
                                act::unpack16x2(add[j], a, b, f16);
                                v[2 * j] += a;
                                v[2 * j + 1] += b;
                                add[j] = add[16 + j];
                            }
                        } else if (row0 + lane < p.T) {
                            const uint16_t *at = e.residual + (row0 + lane) * e.residual_ld + c;
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (c + j < p.N) v[j] += act::from16(at[j], f16);
                        }
                        __syncwarp();
                    }
                    put_seg(y, row0, col, h, v, p.T, p.N, f16, buf, lane);
                }
                if (ragged) put_rest(y, row0, col, p.T, p.N, buf, lane);
                if constexpr (!GATED) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        ws[i] = ws[2 + i];
                        bias[i] = bias[2 + i];
                    }
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
