// mm_large.cuh -- forward product of a linear or gated layer on CTA pairs:
// acc = x W^T on tcgen05 tensor cores, the layer's epilogue fused.
//
// A cluster of 2 CTAs computes one tile of 256 tokens x 256 weight rows with
// tcgen05.mma.cta_group::2.  Each CTA stages its own 128 tokens of x and 128
// rows of the weight tile (128 bytes of K per row, 128-byte swizzle) in a ring
// of 32 KB stages filled by TMA.  A gated layer's tile takes 128 gate rows
// (staged by the pair's leader) and the 128 up rows of the same outputs
// (staged by its peer), so gate and up of an output meet in one thread.
//
// Accumulators: two of 256 fp32 TMEM columns, so the epilogue of one tile
// overlaps the products of the next.  CTA = 10 warps:
//   warp 0     one lane issues the TMA loads of this CTA's halves;
//   warp 1     allocates TMEM; in the leader one lane issues the pair MMAs;
//   warps 2-9  epilogue: TMEM subpartition warp % 4 (one token per thread),
//              two warps per subpartition, each on half of the columns.
// Persistent grid of co-resident pairs; tile order: groups of kGroupM token
// tiles, weight tiles outer within a group, so that the ~76 tiles in flight
// read about 8 token and 9.5 weight tiles.
#pragma once

#include <cuda.h>

#include "act.cuh"
#include "mbar_wait.cuh"
#include "mm_types.h"
#include "ptx.cuh"
#include "tcgen05.cuh"

namespace vlmce {
namespace mm {

constexpr int kPairM = 256;                    // tokens of a pair tile
constexpr int kHalfRows = 128;                 // rows of x, and of W, staged by one CTA
constexpr int kOpBytes = kHalfRows * 128;      // one operand of a stage: 16 KB
constexpr int kStageBytes = 2 * kOpBytes;
constexpr int kStages = 6;
constexpr int kLargeThreads = 320;
constexpr int kEpiWarps = 8;
constexpr int kLargeTmemCols = 512;
constexpr int kGroupM = 8;
constexpr int kLargeBars = 2 * kStages + 5;    // full, empty, tmem full x2, tmem empty x2, drain
constexpr int kLargeTail = 8 * kLargeBars + 16;  // barriers, TMEM slot, abort flag
constexpr int kStageWords = 32 * 17;             // an epilogue warp's transposing buffer
constexpr int kLargeSmem = 1024 + kStages * kStageBytes + kLargeTail + kEpiWarps * kStageWords * 4;

struct LargeParams {
    int T, N;          // tokens, outputs
    int up_row;        // gated: first up row of the weight
    int chunks;        // K in 128-byte chunks
    int mt, nt, tiles;
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

// ---------------------------------------------------------- row segments
// A warp's 32 rows x 32 consecutive 16-bit columns, one row per lane, `nr`
// rows and `nc` columns of which exist.  vec: bytes an access may use where all
// 32 columns exist (32, 16 or 2).  Rows without 16-byte alignment, and the last
// columns, pass through `stage` (the warp's 32 x 17 words of shared memory),
// so that a warp's accesses still cover consecutive addresses of a row.
__device__ __forceinline__ void store_seg(uint16_t *base, int64_t ld, const float (&v)[32], int nr,
                                          int nc, int vec, bool f16, uint32_t *stage, int lane) {
    uint32_t u[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) u[j] = act::pack16x2(v[2 * j], v[2 * j + 1], f16);
    if (nc == 32 && vec >= 16) {
        if (lane >= nr) return;
        uint16_t *p = base + lane * ld;
        if (vec >= 32) {
            ptx::st_global_v8(p, u[0], u[1], u[2], u[3], u[4], u[5], u[6], u[7]);
            ptx::st_global_v8(p + 16, u[8], u[9], u[10], u[11], u[12], u[13], u[14], u[15]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<uint4 *>(p + 8 * j) =
                    make_uint4(u[4 * j], u[4 * j + 1], u[4 * j + 2], u[4 * j + 3]);
        }
        return;
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 16; ++j) stage[lane * 17 + j] = u[j];
    __syncwarp();
    const uint16_t *s16 = reinterpret_cast<const uint16_t *>(stage);
    if (lane < nc) {
#pragma unroll 8
        for (int r = 0; r < nr; ++r) base[r * ld + lane] = s16[r * 34 + lane];
    }
}
__device__ __forceinline__ void add_seg(const uint16_t *base, int64_t ld, float (&v)[32], int nr,
                                        int nc, int vec, bool f16, uint32_t *stage, int lane) {
    uint32_t u[16];
    if (nc == 32 && vec >= 16) {
        if (lane >= nr) return;
        const uint16_t *p = base + lane * ld;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint4 q = *reinterpret_cast<const uint4 *>(p + 8 * j);
            u[4 * j] = q.x;
            u[4 * j + 1] = q.y;
            u[4 * j + 2] = q.z;
            u[4 * j + 3] = q.w;
        }
    } else {
        uint16_t *s16 = reinterpret_cast<uint16_t *>(stage);
        __syncwarp();
        if (lane < nc) {
#pragma unroll 8
            for (int r = 0; r < nr; ++r) s16[r * 34 + lane] = base[r * ld + lane];
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 16; ++j) u[j] = stage[lane * 17 + j];
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        float a, b;
        act::unpack16x2(u[j], a, b, f16);
        v[2 * j] += a;
        v[2 * j + 1] += b;
    }
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
__global__ void __launch_bounds__(kLargeThreads, 1)
    mm_large_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
                    const __grid_constant__ LargeParams p) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kStages * kStageBytes);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kLargeBars);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const uint32_t ring = ptx::smem_addr(smem);
    const uint32_t bar0 = ptx::smem_addr(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (kStages + s); };
    auto tfull = [&](int b) { return bar0 + 8u * (2 * kStages + b); };
    auto tempty = [&](int b) { return bar0 + 8u * (2 * kStages + 2 + b); };
    const uint32_t drain = bar0 + 8u * (2 * kStages + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t prank = ptx::cluster_ctarank();  // 0: the pair's leader
    const int cluster = static_cast<int>(ptx::cluster_id_x());
    const int nclusters = static_cast<int>(ptx::ncluster_x());

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(full(s), 1);   // leader: its producer + the bytes of both CTAs
            ptx::mbar_init(empty(s), 1);  // one commit from the leader's MMA issuer
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(tfull(b), 1);
            ptx::mbar_init(tempty(b), 2 * kEpiWarps);  // leader: both CTAs' epilogue warps
        }
        ptx::mbar_init(drain, 1);
        *abort = 0;
        ptx::fence_mbar_init_cluster();
    }
    if (warp == 0 && lane == 0) {
        tc::prefetch_tensormap(&mx);
        tc::prefetch_tensormap(&mw);
    }
    if (warp == 1) {
        tc::tmem_alloc_pair(ptx::smem_addr(tmem_slot), kLargeTmemCols);
        tc::tmem_relinquish_pair();
    }
    tc::fence_before_sync();
    ptx::cluster_sync_any();  // barrier inits and the TMEM address visible to the cluster
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    // TMEM is held: the next kernel of the stream may set itself up; this one
    // waits for its predecessor's results before it touches global memory
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    constexpr int kElts = FP8 ? 128 : 64;  // K elements of a 128-byte chunk

    if (warp == 0) {
        if (lane == 0) {
            const uint32_t full_leader = ptx::mapa(full(0), 0);
            int s = 0;
            uint32_t ph = 0;
            int64_t issued = 0;
            for (int t = cluster; t < p.tiles; t += nclusters) {
                const LargeTile tl = large_tile<GATED>(p, t);
                const int ar = tl.m0 + kHalfRows * static_cast<int>(prank);
                const int br = GATED ? (prank == 0 ? tl.n0 : p.up_row + tl.n0)
                                     : tl.n0 + kHalfRows * static_cast<int>(prank);
                for (int c = 0; c < p.chunks; ++c) {
                    wait_bar(empty(s), ph ^ 1, abort, p.err);
                    if (prank == 0) ptx::mbar_arrive_expect_tx(full(s), 2 * kStageBytes);
                    const uint32_t sa = ring + s * kStageBytes;
                    tc::tma_load_2d_pair(sa, &mx, c * kElts, ar, full_leader + 8u * s);
                    tc::tma_load_2d_pair(sa + kOpBytes, &mw, c * kElts, br, full_leader + 8u * s);
                    ++issued;
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
            // every copy into the pair has landed once the full phases of the
            // last kStages loads completed at the leader
            if (prank == 0) {
                for (int i = 0; i < kStages && i < issued; ++i) {
                    const int64_t q = issued - 1 - i;
                    drain_bar(full(static_cast<int>(q % kStages)),
                              static_cast<uint32_t>((q / kStages) & 1), p.err);
                }
            }
        }
    } else if (warp == 1) {
        if (prank == 0 && lane == 0) {
            const uint32_t idesc = tc::idesc_bf16_f32(256, 256, false, false, FP8 || p.e.f16);
            int s = 0;
            uint32_t ph = 0;
            int it = 0;
            for (int t = cluster; t < p.tiles; t += nclusters, ++it) {
                const int b = it & 1;
                wait_bar<true>(tempty(b), ((it >> 1) & 1) ^ 1, abort, p.err);
                tc::fence_after_sync();
                const uint32_t d = tmem + static_cast<uint32_t>(b * 256);
                for (int c = 0; c < p.chunks; ++c) {
                    wait_bar(full(s), ph, abort, p.err);
                    tc::fence_after_sync();
                    const uint32_t sa = ring + s * kStageBytes;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint64_t ad = tc::smem_desc_sw128(sa + 32 * k, 16, 1024);
                        const uint64_t bd = tc::smem_desc_sw128(sa + kOpBytes + 32 * k, 16, 1024);
                        if constexpr (FP8)
                            tc::mma_f8_pair(d, ad, bd, idesc, (c | k) != 0);
                        else
                            tc::mma_bf16_pair(d, ad, bd, idesc, (c | k) != 0);
                    }
                    tc::mma_commit_pair(empty(s), 3u);
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1;
                    }
                }
                tc::mma_commit_pair(tfull(b), 3u);
            }
            tc::mma_commit_pair(drain, 1u);
            drain_bar(drain, 0, p.err);
        }
    } else {
        const int q = warp & 3, half = (warp - 2) >> 2;
        uint32_t *stage = reinterpret_cast<uint32_t *>(smem + kStages * kStageBytes + kLargeTail) +
                          (warp - 2) * kStageWords;
        const uint32_t tempty_leader = ptx::mapa(tempty(0), 0);
        const Epi &e = p.e;
        int it = 0;
        for (int t = cluster; t < p.tiles; t += nclusters, ++it) {
            const LargeTile tl = large_tile<GATED>(p, t);
            const int b = it & 1;
            wait_bar(tfull(b), (it >> 1) & 1, abort, p.err);
            tc::fence_after_sync();
            const int64_t row0 = tl.m0 + kHalfRows * static_cast<int>(prank) + q * 32;
            const float xs = e.xs && row0 + lane < p.T ? e.xs[row0 + lane] : 1.f;
            const uint32_t tbase = tmem + (static_cast<uint32_t>(q * 32) << 16) + b * 256;
            if constexpr (GATED) {
#pragma unroll 1
                for (int c = 2 * half; c < 2 * half + 2; ++c) {
                    uint32_t rg[32], ru[32];
                    tc::tmem_ld32(tbase + 32 * c, rg);
                    tc::tmem_ld32(tbase + 128 + 32 * c, ru);
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
                    tc::tmem_ld32(tbase + 32 * c, r);
                    tc::tmem_ld_wait();
                    const int col = tl.n0 + 32 * c;
                    if (col < p.N && row0 < p.T) linear_seg(p, r, row0, col, xs, stage, lane);
                    __syncwarp();
                }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) ptx::mbar_remote_arrive_release(tempty_leader + 8u * b);
        }
    }
    // every MMA of the pair has completed (drain) and every copy has landed;
    // the pair meets before TMEM is released and either CTA exits
    tc::fence_before_sync();
    __syncthreads();
    ptx::cluster_sync_any();
    if (warp == 1) {
        __syncwarp();
        tc::fence_after_sync();
        tc::tmem_dealloc_pair(tmem, kLargeTmemCols);
    }
}

}  // namespace mm
}  // namespace vlmce
