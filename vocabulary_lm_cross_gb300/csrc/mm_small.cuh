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
// a cluster share a tile, each on its own part of K.  Each CTA owns a run of
// the tile's tokens: the others push their fp32 accumulators of those tokens
// into its shared memory (four tokens of a row per 16-byte store; stores do
// not wait for the other SM), and it adds them in rank order (fixed, so the
// result does not depend on timing).
//
// Two CTAs of this kernel may share an SM.  TMEM allocation blocks while columns are
// short, and a blocked CTA of a cluster could wait on one that waits on it; so CTAs of
// this kernel take at least the same share of the SM's shared memory as of its TMEM
// (kSmemPerTmemCol per column), and TMEM never runs out first.  The library's pair
// kernels hold all 512 columns with less than all of the shared memory (the GEMM
// engine 198 KB): kSmallSmemMin keeps a CTA of this kernel from fitting beside one.
//
// Measured on GB300 (a call among others): T = 1, K = 4096, 2n = 24576 bf16 35.4 us
// (201 MB of weight: 5.7 TB/s with the launch's 4 us), T = 64, K = 16384, N = 6656
// e4m3 25.5 us (4.4 TB/s), T = 300, K = 4096, 2n = 20480 e4m3 33.1 us (1.52 PFLOP/s:
// bound by the operands' way from L2, 53 of 64 bytes a clock on the SMs with two CTAs).
//
// CTA = 10 warps: warp 0 TMA producer, warp 1 TMEM and MMA issuer, warps 2-9
// epilogue (one weight row per thread, two threads on alternate groups of
// tokens).
#pragma once

#include <cuda.h>

#include "act.cuh"
#include "mbar_wait.cuh"
#include "mm_types.h"
#include "ptx_async.cuh"
#include "tcgen05.cuh"

namespace vlmce {
namespace mm {

constexpr int kSmallThreads = 320;
// An SM's four quarters hold warps w, w + 4, ... of a block: 10 warps take the
// registers of 12 where two blocks share it.
constexpr int kSmallBound = 384;
constexpr int kWTileBytes = 128 * 128;  // 128 weight rows x 128 bytes of K
constexpr int kMaxSmallStages = 12;
constexpr int kMaxSplit = 8;
// barriers, TMEM slot, abort flag, the tokens' factors
constexpr int kSmallTail = 8 * (2 * kMaxSmallStages + 2) + 16 + 4 * 256;
// Shared memory of an SM (228 KB, 1 KB of it reserved per resident CTA) over its
// 512 TMEM columns; and the floor beside the pair kernels.
constexpr int kSmSmem = 233472;
constexpr int kSmemPerTmemCol = 456;
constexpr int kSmemReserved = 1024;
constexpr int kSmallSmemMin = 34816;
static_assert(kSmemPerTmemCol * 512 >= kSmSmem, "TMEM would run out first");

struct SmallParams {
    int T, N;
    int up_row;
    int chunks;       // K in 128-byte chunks
    int split;        // CTAs of a cluster sharing a tile's K
    int bn;           // tokens per tile (multiple of 16)
    int stages;
    int per_stage;    // chunks of a stage
    int tmem_cols;
    int red_tokens;   // tokens reduced at a time when split > 1 (multiple of 16)
    int part_offset;  // where they are collected: 0, the ring, or behind the rest
    Epi e;
    int *err;
};

// What the epilogue reads besides the accumulators is fetched ahead of it, while
// the products run: with the ring's copies in flight everywhere a load takes
// microseconds (T = 64, K = 16384, N = 6656 in e4m3: a residual read in the
// epilogue cost 7.5 of 32.5 us).
struct RowFactors {
    float ws, ws_up, bias;
};
template <bool GATED>
__device__ __forceinline__ RowFactors row_factors(const SmallParams &p, int n) {
    const Epi &e = p.e;
    RowFactors f = {1.f, 1.f, 0.f};
    if (e.ws) {
        f.ws = e.ws[n];
        if constexpr (GATED) f.ws_up = e.ws[p.up_row + n];
    }
    if constexpr (!GATED)
        if (e.bias) f.bias = act::from16(e.bias[n], e.f16 != 0);
    return f;
}
// A thread's tokens come in units of 16: token i of the unit starting at j is
// j + i (`run` = 16), or j + i % 4 + i / 4 * 8 (`run` = 4: two threads share
// every eight tokens).  Tokens at or after `end` do not exist.
__device__ __forceinline__ int unit_token(int j, int i, int run) {
    return run == 16 ? j + i : j + (i & 3) + (i >> 2) * 8;
}
__device__ __forceinline__ void fetch_residual(const SmallParams &p, uint16_t (&r)[16], int j,
                                               int end, int run, int64_t t0, int n) {
    const Epi &e = p.e;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int t = unit_token(j, i, run);
        r[i] = t < end ? e.residual[(t0 + t) * e.residual_ld + n] : 0;
    }
}
// The epilogue of NJ consecutive tokens t0 + j .. of one weight row n (Epi in
// mm_types.h); tokens from `count` on do not exist.  xs: their factors, r: the
// residual's values.
template <bool GATED, int NJ>
__device__ __forceinline__ void small_epilogue(const SmallParams &p, const RowFactors &f,
                                               float (&g)[NJ], float (&u)[NJ], int64_t t,
                                               int count, int n, const float *xs,
                                               const uint16_t *r) {
    const Epi &e = p.e;
    const bool f16 = e.f16 != 0;
    if (e.ws) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            g[j] *= xs[j] * f.ws;
            if constexpr (GATED) u[j] *= xs[j] * f.ws_up;
        }
    }
    if constexpr (!GATED) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) g[j] += f.bias;
    }
    if (e.preact) {
        uint16_t *z = e.preact + t * e.preact_ld + n;
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            if (j < count) {
                z[j * e.preact_ld] = act::to16(g[j], f16);
                if constexpr (GATED) z[j * e.preact_ld + p.N] = act::to16(u[j], f16);
            }
    }
    act::apply_n(g, e.act);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        if constexpr (GATED)
            g[j] *= u[j];
        else if (e.residual)
            g[j] += act::from16(r[j], f16);
    }
    uint16_t *y = e.y + t * e.y_ld + n;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
        if (j < count) y[j * e.y_ld] = act::to16(g[j], f16);
}

// W_MN: the weight is stored with its outputs contiguous ([K, N], as the gradient
// dx = dz W reads W): 128 outputs x 64 of K come as two boxes of 64 x 64, MN-major.
template <bool GATED, bool FP8, bool W_MN>
__global__ void __launch_bounds__(kSmallBound, 2)
    mm_small_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mx,
                    const __grid_constant__ SmallParams p) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    constexpr int kW = GATED ? 2 : 1;
    constexpr int kElts = FP8 ? 128 : 64;
    const int chunk_bytes = kW * kWTileBytes + p.bn * 128;
    const int stage_bytes = p.per_stage * chunk_bytes;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + p.stages * stage_bytes);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * kMaxSmallStages + 2);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    float *xs_s = reinterpret_cast<float *>(tmem_slot + 4);  // [256] the tokens' factors
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
    // TMEM is held: the next kernel of the stream may set itself up; this one
    // waits for its predecessor's results before it touches global memory
    ptx::griddep_launch_dependents();
    if (p.split > 1) ptx::cluster_arrive_any();  // this CTA has started
    const int ring_chunks = p.stages * p.per_stage;
    if (warp == 0 && lane == 0 && c1 - c0 >= 3 * ring_chunks) {
        // a long walk: the weight's first tiles may already come into L2 (T = 64, K =
        // 16384, N = 6656 in e4m3 25.5 -> 24.8 us; short ones lose by it)
        for (int c = c0; c < c0 + ring_chunks; ++c) {
            if constexpr (W_MN) {
                tc::tma_prefetch_2d(&mw, n0, c * kElts);
                tc::tma_prefetch_2d(&mw, n0 + 64, c * kElts);
            } else {
                tc::tma_prefetch_2d(&mw, c * kElts, n0);
            }
            if constexpr (GATED) tc::tma_prefetch_2d(&mw, c * kElts, p.up_row + n0);
        }
    }
    ptx::griddep_wait();

    if (warp == 0) {
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0;
            for (int c = c0; c < c1; c += p.per_stage) {
                wait_bar(empty(s), ph ^ 1, abort, p.err);
                const int n = min(p.per_stage, c1 - c);
                ptx::mbar_arrive_expect_tx(full(s), static_cast<uint32_t>(n * chunk_bytes));
                for (int i = 0; i < n; ++i) {
                    const uint32_t sa = ring + s * stage_bytes + i * chunk_bytes;
                    const int k = (c + i) * kElts;
                    if constexpr (W_MN) {
                        tc::tma_load_2d(sa, &mw, n0, k, full(s));
                        tc::tma_load_2d(sa + kWTileBytes / 2, &mw, n0 + 64, k, full(s));
                    } else {
                        tc::tma_load_2d(sa, &mw, k, n0, full(s));
                    }
                    if constexpr (GATED)
                        tc::tma_load_2d(sa + kWTileBytes, &mw, k, p.up_row + n0, full(s));
                    tc::tma_load_2d(sa + kW * kWTileBytes, &mx, k, t0, full(s));
                }
                if (++s == p.stages) {
                    s = 0;
                    ph ^= 1;
                }
            }
            // every copy has landed once the last full phase of each stage completed
            const int issued = (c1 - c0 + p.per_stage - 1) / p.per_stage;
            for (int i = 0; i < p.stages && i < issued; ++i) {
                const int k = issued - 1 - i;
                drain_bar(full(k % p.stages), static_cast<uint32_t>((k / p.stages) & 1), p.err);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = tc::idesc_bf16_f32(128, p.bn, W_MN, false, FP8 || p.e.f16);
            int s = 0;
            uint32_t ph = 0;
            for (int c = c0; c < c1; c += p.per_stage) {
                wait_bar(full(s), ph, abort, p.err);
                tc::fence_after_sync();
                const int n = min(p.per_stage, c1 - c);
                for (int i = 0; i < n; ++i) {
                    const uint32_t sa = ring + s * stage_bytes + i * chunk_bytes;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint64_t xd =
                            tc::smem_desc_sw128(sa + kW * kWTileBytes + 32 * k, 16, 1024);
#pragma unroll
                        for (int w = 0; w < kW; ++w) {
                            const uint64_t wd =
                                W_MN ? tc::smem_desc_sw128(sa + 2048 * k, kWTileBytes / 2, 1024)
                                     : tc::smem_desc_sw128(sa + w * kWTileBytes + 32 * k, 16, 1024);
                            const uint32_t d = tmem + static_cast<uint32_t>(w * p.bn);
                            const uint32_t add = c + i > c0 || k != 0;
                            if constexpr (FP8)
                                tc::mma_f8(d, wd, xd, idesc, add);
                            else
                                tc::mma_bf16(d, wd, xd, idesc, add);
                        }
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
    }

    const int q = warp & 3;            // TMEM subpartition of an epilogue warp
    const int half = (warp - 2) >> 2;  // which of the subpartition's two warps
    const int row = q * 32 + lane;
    const bool row_ok = n0 + row < p.N;
    const uint32_t tbase = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const int n = n0 + row;
    const bool res = !GATED && p.e.residual != nullptr;
    const int own = p.split == 1 ? p.bn : (p.red_tokens / 4 + p.split - 1) / p.split * 4;
    RowFactors f = {1.f, 1.f, 0.f};
    uint16_t r_next[16];
    if (warp >= 2) {
        if (p.e.ws) {
            const int j = threadIdx.x - 64;  // 256 threads, at most 256 tokens
            if (j < nt) xs_s[j] = p.e.xs[t0 + j];
        }
        if (row_ok) {
            f = row_factors<GATED>(p, n);
            if (res) {
                if (p.split == 1)
                    fetch_residual(p, r_next, 16 * half, nt, 16, t0, n);
                else
                    fetch_residual(p, r_next, rank * own + 4 * half,
                                   min((rank + 1) * own, min(p.red_tokens, nt)), 4, t0, n);
            }
        }
        wait_bar(done, 0, abort, p.err);
        __syncwarp();  // each lane left the wait by itself; what follows takes the whole warp
        tc::fence_after_sync();
        asm volatile("bar.sync 1, 256;" ::: "memory");  // xs_s is complete
    }
    if (p.split == 1) {
        if (warp >= 2) {
#pragma unroll 1
            for (int j0 = 16 * half; j0 < nt; j0 += 32) {
                uint32_t a[16], b[16];
                tc::tmem_ld16(tbase + j0, a);
                if constexpr (GATED) tc::tmem_ld16(tbase + p.bn + j0, b);
                uint16_t r[16];
                if (res) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) r[i] = r_next[i];
                    if (row_ok) fetch_residual(p, r_next, j0 + 32, nt, 16, t0, n);
                }
                tc::tmem_ld_wait();
                if (row_ok) {
#pragma unroll
                    for (int h = 0; h < 16; h += 8) {
                        float g[8], u[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            g[j] = __uint_as_float(a[h + j]);
                            u[j] = GATED ? __uint_as_float(b[h + j]) : 0.f;
                        }
                        if (j0 + h < nt)
                            small_epilogue<GATED, 8>(p, f, g, u, t0 + j0 + h, nt - j0 - h, n,
                                                     xs_s + j0 + h, r + h);
                    }
                }
                __syncwarp();
            }
        }
    } else {
        // For this CTA's run of `own` tokens of a block of red_tokens, the accumulators
        // [from][kW][token / 4][128 rows][4]: in shared memory of their own where that
        // is little (then it is enough that every CTA has started), else in the ring,
        // which is free once every CTA's copies have landed and MMAs completed.
        float *part_f = reinterpret_cast<float *>(smem + p.part_offset);
        const uint32_t part = ptx::smem_addr(part_f);
        ptx::cluster_wait_any();
        const int plane = own * 128;  // floats of one accumulator of one sender
#pragma unroll 1
        for (int jb = 0; jb < nt; jb += p.red_tokens) {
            if (p.part_offset == 0) ptx::cluster_sync_any();
            const int je = min(p.red_tokens, nt - jb);
            if (warp >= 2) {
#pragma unroll 1
                for (int j0 = 16 * half; j0 < je; j0 += 32) {
                    uint32_t a[16], b[16];
                    tc::tmem_ld16(tbase + jb + j0, a);
                    if constexpr (GATED) tc::tmem_ld16(tbase + p.bn + jb + j0, b);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        if (j0 + j < je) {
                            const int to = (j0 + j) / own, i = (j0 + j) - to * own;
                            const uint32_t dst = ptx::mapa(
                                part + 4u * (rank * kW * plane + i * 128 + 4 * row), to);
                            ptx::st_dsmem_v4(dst, make_uint4(a[j], a[j + 1], a[j + 2], a[j + 3]));
                            if constexpr (GATED)
                                ptx::st_dsmem_v4(dst + 4u * plane, make_uint4(b[j], b[j + 1],
                                                                              b[j + 2], b[j + 3]));
                        }
                    }
                }
            }
            ptx::cluster_sync_any();
            if (warp >= 2 && row_ok) {
                const int first = rank * own, end = min(first + own, je);  // of the block
                const float *src = part_f + 4 * row;
                if (res && jb > 0)
                    fetch_residual(p, r_next, jb + first + 4 * half, jb + end, 4, t0, n);
#pragma unroll 1
                for (int j0 = first + 4 * half; j0 < end; j0 += 32) {
                    uint16_t r[16];
                    if (res) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) r[i] = r_next[i];
                        fetch_residual(p, r_next, jb + j0 + 32, jb + end, 4, t0, n);
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int j = j0 + 8 * c;
                        if (j < end) {
                            float g[4] = {0.f, 0.f, 0.f, 0.f}, u[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
                            for (int s = 0; s < p.split; ++s) {
                                const float4 v = *reinterpret_cast<const float4 *>(
                                    src + s * kW * plane + (j - first) * 128);
                                g[0] += v.x;
                                g[1] += v.y;
                                g[2] += v.z;
                                g[3] += v.w;
                                if constexpr (GATED) {
                                    const float4 w = *reinterpret_cast<const float4 *>(
                                        src + (s * kW + 1) * plane + (j - first) * 128);
                                    u[0] += w.x;
                                    u[1] += w.y;
                                    u[2] += w.z;
                                    u[3] += w.w;
                                }
                            }
                            small_epilogue<GATED, 4>(p, f, g, u, t0 + jb + j, end - j, n,
                                                     xs_s + jb + j, r + 4 * c);
                        }
                    }
                }
            }
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
