// mm_grad.cuh -- the two gradient products of a linear or gated layer in one
// launch on CTA pairs (mm_pair.cuh):
//   dx = dz W     A = dz [T, rows] K-major,       B = W: N(=K_in)-major
//   dW = dz^T x   A = dz: M(=rows)-major,         B = x: N(=K_in)-major
// with either operand K-major or MN-major, so nothing is transposed in memory.
//
// Tensor-bound: T = 4096, K = 6656, 2n = 32768 both products 1.82-1.90 ms in a burst
// (1.88-1.97 PFLOP/s; with the library's older GEMM 2.18), 2.09-2.14 back to back under
// the power cap (97-100 % of the library's sustained rate).
// For few tokens bound by dW's stores (T = 16, K = 4096, N = 16384 39 us for 134 MB; a
// plain fill takes 34).
//
// The tiles of both products are numbered one after the other, the longer
// inner size first.
#pragma once

#include <cuda.h>

#include "mm_pair.cuh"
#include "mm_types.h"

namespace vlmce {
namespace mm {

// C[M, N] (+)= A B^T.
struct GradProblem {
    int M, N, chunks;
    int a_mn, b_mn;
    int mt, nt, tile0;
    int f32, accumulate;   // C fp32 (added to where accumulate is set), else 16 bits
    void *C;               // rows 16-byte aligned
    int64_t ld;
};
struct GradParams {
    GradProblem p[2];
    int nprob;
    int f16;
    int dealt;
    int *err;
};
struct GradMaps {
    CUtensorMap a[2], b[2], c[2];
};

struct GradTile {
    int p, m0, n0;
};
__device__ __forceinline__ GradTile grad_tile(const GradParams &a, int t) {
    const int p = a.nprob > 1 && t >= a.p[1].tile0 ? 1 : 0;
    const GradProblem &P = a.p[p];
    constexpr int kGroup = 8;  // as kGroupM of the forward product
    const int lt = t - P.tile0;
    const int per_group = kGroup * P.nt;
    const int g = lt / per_group, r = lt - g * per_group;
    const int gm = min(kGroup, P.mt - g * kGroup);
    const int n = r / gm;
    return {p, (g * kGroup + (r - n * gm)) * 256, n * 256};
}

__global__ void __launch_bounds__(kPairThreads, 1)
    mm_grad_kernel(const __grid_constant__ GradMaps maps, const __grid_constant__ GradParams a) {
    constexpr int kPer = 1;
    extern __shared__ unsigned char smem_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < a.nprob; ++i) {
            tc::prefetch_tensormap(&maps.a[i]);
            tc::prefetch_tensormap(&maps.b[i]);
        }
    }
    const Pair<kPer> q = pair_setup<kPer>(smem_raw, a.err, a.dealt);
    Tiles tiles;

    if (warp == 0 || warp == kWarpB) {
        if (lane == 0) {
            const uint32_t full_leader = ptx::mapa(q.full(0), 0);
            Ring<kPer> r;
            int64_t issued = 0;
            for (int t; (t = tiles.next<false>(q, lane)) >= 0;) {
                const GradTile tl = grad_tile(a, t);
                const int chunks = a.p[tl.p].chunks;
                const bool mn = warp == 0 ? a.p[tl.p].a_mn != 0 : a.p[tl.p].b_mn != 0;
                const CUtensorMap *m = warp == 0 ? &maps.a[tl.p] : &maps.b[tl.p];
                const int row =
                    (warp == 0 ? tl.m0 : tl.n0) + kHalfRows * static_cast<int>(q.rank);
                const uint32_t side = warp == 0 ? 0 : kOpBytes;
                for (int c = 0; c < chunks; c += kPer) {
                    const int n = min(kPer, chunks - c);
                    if (warp == 0)
                        stage_begin<true, kPer>(q, r, n);
                    else
                        stage_begin<false, kPer>(q, r, n);
                    const uint32_t fb = full_leader + 8u * r.s;
                    for (int i = 0; i < n; ++i) {
                        const uint32_t to = q.chunk(r.s, i) + side;
                        const int k = 64 * (c + i);
                        if (!mn) {
                            tc::tma_load_2d_pair(to, m, k, row, fb);
                        } else {
                            tc::tma_load_2d_pair(to, m, row, k, fb);
                            tc::tma_load_2d_pair(to + 8192, m, row + 64, k, fb);
                        }
                    }
                    r.next(q);
                }
                issued += (chunks + kPer - 1) / kPer;
            }
            if (warp == 0) drain_loads(q, issued);
        }
    } else if (warp == 1) {
        if (q.rank == 0 && lane == 0) {
            Ring<kPer> r;
            int it = 0;
            for (int t; (t = tiles.next<false>(q, lane)) >= 0; ++it) {
                const GradProblem &P = a.p[grad_tile(a, t).p];
                mma_tile<false, kPer>(q, r, it, P.chunks,
                                tc::idesc_bf16_f32(256, 256, P.a_mn != 0, P.b_mn != 0, a.f16 != 0),
                                P.a_mn != 0, P.b_mn != 0);
            }
            mma_finish(q);
        }
    } else if (warp == kWarpTiles) {
        if (q.rank == 0 && lane == 0) fetch_tiles(q);
    } else {
        const int half = (warp - 2) >> 2;
        uint32_t *buf = q.out_buffer(warp - 2);
        const uint32_t tempty_leader = ptx::mapa(q.tempty(0), 0);
        int it = 0;
        for (int t; (t = tiles.next<true>(q, lane)) >= 0; ++it) {
            const GradTile tl = grad_tile(a, t);
            const GradProblem &P = a.p[tl.p];
            const CUtensorMap *map = &maps.c[tl.p];
            const int64_t row0 = tl.m0 + kHalfRows * static_cast<int>(q.rank) + (warp & 3) * 32;
            const Out o = {static_cast<uint16_t *>(P.C), P.ld, 16, map};
            const uint32_t acc = acc_wait(q, it, warp);
#pragma unroll 1
            for (int c = 4 * half; c < 4 * half + 4; ++c) {
                uint32_t r[32];
                tc::tmem_ld32(acc + 32 * c, r);
                tc::tmem_ld_wait();
                const int col = tl.n0 + 32 * c;
                if (row0 < P.M) {
                    if (P.f32) {
                        if (col < P.N)
                            put_f32(map, row0, col, r, P.accumulate != 0, buf, lane);
                    } else if (tl.n0 + 64 * (c >> 1) < P.N) {
                        float v[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
                        put_seg(o, row0, tl.n0 + 64 * (c >> 1), c & 1, v, P.M, P.N, a.f16 != 0, buf,
                                lane);
                    }
                }
                __syncwarp();
            }
            acc_release(tempty_leader, it, lane);
        }
        if (lane == 0) tc::bulk_wait();
    }
    pair_teardown(q);
}

}  // namespace mm
}  // namespace vlmce
