// mm_small.cuh -- forward product of a linear or gated layer for few tokens:
// acc[n, t] = W x^T on one CTA per 128 weight rows, the layer's epilogue fused.
//
// With few tokens the product is bound by streaming the weight once, so the
// weight rows take the tensor core's M side (128 rows, whatever T is) and the
// tokens its N side (bn = 16 .. 256, rounded up to 16; rows beyond T read as
// zero).  A gated layer's CTA holds the 128 gate rows and the 128 up rows of
// the same outputs, with an accumulator each.  A ring of stages (128 bytes of
// K of the weight rows and of the tokens, 128-byte swizzle) is filled by TMA.
//
// Where the weight has too few row tiles to occupy every SM, `split` CTAs of
// a cluster share a tile, each on its own part of K; their fp32 accumulators
// meet in shared memory and are added in rank order (fixed, so the result does
// not depend on timing).
//
// Two CTAs of this kernel, or one and another kernel's, may share an SM.  TMEM
// allocation blocks while columns are short, and a blocked CTA of a cluster
// could wait on one that waits on it; so every kernel of the library that
// allocates TMEM takes at least the same share of the SM's shared memory
// (kSmemPerTmemCol per column), so that TMEM never runs out first.
//
// CTA = 6 warps: warp 0 TMA producer, warp 1 TMEM and MMA issuer, warps 2-5
// epilogue (one weight row per thread).
#pragma once

#include <cuda.h>

#include "act.cuh"
#include "mbar_wait.cuh"
#include "mm_types.h"
#include "ptx.cuh"
#include "tcgen05.cuh"

namespace vlmce {
namespace mm {

constexpr int kSmallThreads = 192;
constexpr int kWTileBytes = 128 * 128;  // 128 weight rows x 128 bytes of K
constexpr int kMaxSmallStages = 12;
constexpr int kMaxSplit = 8;
constexpr int kSmallTail = 8 * (2 * kMaxSmallStages + 2) + 16;  // barriers, TMEM slot, abort flag
// Shared memory of an SM (228 KB, 1 KB of it reserved per resident CTA) over its
// 512 TMEM columns; and a floor that does not fit beside a pair kernel, which
// holds all 512 columns with 198 KB.
constexpr int kSmemPerTmemCol = 456;
constexpr int kSmemReserved = 1024;
constexpr int kSmallSmemMin = 34816;

struct SmallParams {
    int T, N;
    int up_row;
    int chunks;       // K in 128-byte chunks
    int split;        // CTAs of a cluster sharing a tile's K
    int bn;           // tokens per tile (multiple of 16)
    int stages;
    int tmem_cols;
    int red_tokens;   // tokens reduced at a time when split > 1 (multiple of 16)
    Epi e;
    int *err;
};

// One output: token t, column n of acc (linear) or of (g, u) (gated).
__device__ __forceinline__ void small_linear(const SmallParams &p, float v, int t, int n) {
    const Epi &e = p.e;
    const bool f16 = e.f16 != 0;
    if (e.ws) v *= e.xs[t] * e.ws[n];
    if (e.bias) v += act::from16(e.bias[n], f16);
    if (e.preact) e.preact[static_cast<int64_t>(t) * e.preact_ld + n] = act::to16(v, f16);
    v = act::apply(v, e.act);
    if (e.residual) v += act::from16(e.residual[static_cast<int64_t>(t) * e.residual_ld + n], f16);
    e.y[static_cast<int64_t>(t) * e.y_ld + n] = act::to16(v, f16);
}
__device__ __forceinline__ void small_gated(const SmallParams &p, float g, float u, int t, int n) {
    const Epi &e = p.e;
    const bool f16 = e.f16 != 0;
    if (e.ws) {
        const float xs = e.xs[t];
        g *= xs * e.ws[n];
        u *= xs * e.ws[p.up_row + n];
    }
    if (e.preact) {
        uint16_t *z = e.preact + static_cast<int64_t>(t) * e.preact_ld + n;
        z[0] = act::to16(g, f16);
        z[p.N] = act::to16(u, f16);
    }
    e.y[static_cast<int64_t>(t) * e.y_ld + n] = act::to16(act::apply(g, e.act) * u, f16);
}

template <bool GATED, bool FP8>
__global__ void __launch_bounds__(kSmallThreads)
    mm_small_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mx,
                    const __grid_constant__ SmallParams p) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    constexpr int kW = GATED ? 2 : 1;
    constexpr int kElts = FP8 ? 128 : 64;
    const int stage_bytes = kW * kWTileBytes + p.bn * 128;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + p.stages * stage_bytes);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * kMaxSmallStages + 2);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const uint32_t ring = ptx::smem_addr(smem);
    const uint32_t bar0 = ptx::smem_addr(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (kMaxSmallStages + s); };
    const uint32_t done = bar0 + 8u * (2 * kMaxSmallStages);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = p.split > 1 ? static_cast<int>(ptx::cluster_ctarank()) : 0;
    const int n0 = static_cast<int>(blockIdx.x / p.split) * 128;
    const int t0 = static_cast<int>(blockIdx.y) * p.bn;
    const int nt = min(p.bn, p.T - t0);  // tokens of this tile
    const int c0 = static_cast<int>(static_cast<int64_t>(p.chunks) * rank / p.split);
    const int c1 = static_cast<int>(static_cast<int64_t>(p.chunks) * (rank + 1) / p.split);

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            ptx::mbar_init(full(s), 1);
            ptx::mbar_init(empty(s), 1);
        }
        ptx::mbar_init(done, 1);
        *abort = 0;
        ptx::fence_mbar_init_cluster();
    }
    if (warp == 0 && lane == 0) {
        tc::prefetch_tensormap(&mw);
        tc::prefetch_tensormap(&mx);
    }
    if (warp == 1) {
        tc::tmem_alloc(ptx::smem_addr(tmem_slot), static_cast<uint32_t>(p.tmem_cols));
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0;
            for (int c = c0; c < c1; ++c) {
                wait_bar(empty(s), ph ^ 1, abort, p.err);
                ptx::mbar_arrive_expect_tx(full(s), static_cast<uint32_t>(stage_bytes));
                const uint32_t sa = ring + s * stage_bytes;
                tc::tma_load_2d(sa, &mw, c * kElts, n0, full(s));
                if constexpr (GATED)
                    tc::tma_load_2d(sa + kWTileBytes, &mw, c * kElts, p.up_row + n0, full(s));
                tc::tma_load_2d(sa + kW * kWTileBytes, &mx, c * kElts, t0, full(s));
                if (++s == p.stages) {
                    s = 0;
                    ph ^= 1;
                }
            }
            // every copy has landed once the last full phase of each stage completed
            const int issued = c1 - c0;
            for (int i = 0; i < p.stages && i < issued; ++i) {
                const int k = issued - 1 - i;
                drain_bar(full(k % p.stages), static_cast<uint32_t>((k / p.stages) & 1), p.err);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = tc::idesc_bf16_f32(128, p.bn, false, false, FP8 || p.e.f16);
            int s = 0;
            uint32_t ph = 0;
            for (int c = c0; c < c1; ++c) {
                wait_bar(full(s), ph, abort, p.err);
                tc::fence_after_sync();
                const uint32_t sa = ring + s * stage_bytes;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint64_t xd =
                        tc::smem_desc_sw128(sa + kW * kWTileBytes + 32 * k, 16, 1024);
#pragma unroll
                    for (int w = 0; w < kW; ++w) {
                        const uint64_t wd =
                            tc::smem_desc_sw128(sa + w * kWTileBytes + 32 * k, 16, 1024);
                        const uint32_t d = tmem + static_cast<uint32_t>(w * p.bn);
                        if constexpr (FP8)
                            tc::mma_f8(d, wd, xd, idesc, c > c0 || k != 0);
                        else
                            tc::mma_bf16(d, wd, xd, idesc, c > c0 || k != 0);
                    }
                }
                tc::mma_commit(empty(s));
                if (++s == p.stages) {
                    s = 0;
                    ph ^= 1;
                }
            }
            tc::mma_commit(done);
            drain_bar(done, 0, p.err);
        }
    } else {
        wait_bar(done, 0, abort, p.err);
        tc::fence_after_sync();
    }

    const int q = warp & 3;  // TMEM subpartition of an epilogue warp
    const int row = q * 32 + lane;
    const uint32_t tbase = tmem + (static_cast<uint32_t>(q * 32) << 16);
    if (p.split == 1) {
        if (warp >= 2) {
            const bool row_ok = n0 + row < p.N;
#pragma unroll 1
            for (int j0 = 0; j0 < nt; j0 += 16) {
                uint32_t a[16], b[16];
                tc::tmem_ld16(tbase + j0, a);
                if constexpr (GATED) tc::tmem_ld16(tbase + p.bn + j0, b);
                tc::tmem_ld_wait();
                if (row_ok) {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (j0 + j < nt) {
                            if constexpr (GATED)
                                small_gated(p, __uint_as_float(a[j]), __uint_as_float(b[j]),
                                            t0 + j0 + j, n0 + row);
                            else
                                small_linear(p, __uint_as_float(a[j]), t0 + j0 + j, n0 + row);
                        }
                }
                __syncwarp();
            }
        }
    } else {
        // the ring is free (every copy landed, every MMA completed): it holds
        // this CTA's accumulators as [kW][token][128 rows], red_tokens at a time
        __syncthreads();
        float *part = reinterpret_cast<float *>(smem);
        const uint32_t part_s = ptx::smem_addr(part);
        const int plane = p.red_tokens * 128;
#pragma unroll 1
        for (int jb = 0; jb < nt; jb += p.red_tokens) {
            const int je = min(p.red_tokens, nt - jb);
            if (warp >= 2) {
#pragma unroll 1
                for (int j0 = 0; j0 < je; j0 += 16) {
#pragma unroll
                    for (int w = 0; w < kW; ++w) {
                        uint32_t a[16];
                        tc::tmem_ld16(tbase + w * p.bn + jb + j0, a);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            part[w * plane + (j0 + j) * 128 + row] = __uint_as_float(a[j]);
                    }
                }
            }
            ptx::cluster_sync_any();
            if (warp >= 2 && n0 + row < p.N) {
#pragma unroll 1
                for (int j = rank; j < je; j += p.split) {
                    float v[kW];
#pragma unroll
                    for (int w = 0; w < kW; ++w) v[w] = 0.f;
#pragma unroll 1
                    for (int r = 0; r < p.split; ++r) {
                        const uint32_t src = ptx::mapa(part_s + 4u * (j * 128 + row), r);
#pragma unroll
                        for (int w = 0; w < kW; ++w) v[w] += ptx::ld_dsmem_f32(src + 4u * w * plane);
                    }
                    if constexpr (GATED)
                        small_gated(p, v[0], v[kW - 1], t0 + jb + j, n0 + row);
                    else
                        small_linear(p, v[0], t0 + jb + j, n0 + row);
                }
            }
            ptx::cluster_sync_any();  // the peers have read this CTA's part
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, static_cast<uint32_t>(p.tmem_cols));
    }
}

}  // namespace mm
}  // namespace vlmce
