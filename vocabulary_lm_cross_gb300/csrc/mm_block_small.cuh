// mm_block_small.cuh -- forward product with block scales for few rows (of an expert):
// acc[n, t] = W x^T on 128 weight rows x bn rows of x.
//
// With few rows the product is bound by streaming the weights, so these take the tensor
// core's M side and x's rows its N side (bn = 16 .. 128).  A ring of stages is filled by
// TMA; a CTA walks over tiles, so the next tile's weights are on their way while the last
// one's sums leave.  Four TMEM buffers of bn columns hold the sums of the last four blocks.
//
// Each of the eight epilogue warps has 32 weight rows (a lane each) x bn / 2 rows of x:
// the weight's factor is a lane's own, x's are read by all.
//
// Where there are too few tiles for the SMs, `split` CTAs of a cluster share a tile's K;
// each owns as many of the rows, the others push their sums of those into its shared
// memory, and it adds them in rank order (so the result does not depend on timing).
//
// Bound by the weights' way from HBM where rows are few (T 64, 8 of 32 experts, K 4096, N
// 4096: 95 us, 560 MB, 5.9 TB/s; T 1, K 4096, N 12288: 13.5 us, 50 MB, of which 4-5 us are the
// launch, the first fetch and the last block's way out), and by the epilogue's instructions
// from 64 rows a tile on (64 rows an expert of 4096 x 4096 132 us; each thread with four weight
// rows, so that x's factors are read a quarter as often, 136).
//
// CTA = 11 warps: warp 0 TMA producer, warp 1 TMEM and MMA issuer, warps 2-9 epilogue, warp
// 10 the factors.
#pragma once

#include <cuda.h>

#include "act.cuh"
#include "mm_block.cuh"

namespace vlmce {
namespace mmb {

constexpr int kSmallThreads = 352;
constexpr int kSmallWords = factor_words(128 + 128);  // a block's factors: the weight's rows, rows of x
constexpr int kSmallFactors = 4 * kFactorSlots * kFactorBatch * kSmallWords;
constexpr int kSmallBufs = 4;             // TMEM buffers
constexpr int kSmallWBytes = 128 * 128;   // 128 weight rows x a block of K
constexpr int kMaxStages = 12;
constexpr int kMaxSplit = 8;
// barriers: full, empty per stage; full, empty per TMEM buffer; done; TMEM slot, abort flag
constexpr int kSmallBars = 2 * kMaxStages + 2 * kSmallBufs + 1;
constexpr int kSmallTail = 8 * kSmallBars + 16;

// Two CTAs may share an SM where a thread has few sums.
constexpr int kSmallTwoNc = 16;

struct SmallTile {
    int g, row, end, n;  // group, first row of x and the group's end, first weight row of the group
};
__device__ __forceinline__ SmallTile small_tile(const SmallParams &p, const Table &t, int i, int bn) {
    const int g = group_of(t, p.groups, i / p.nt);
    const int l = i - t.tile0[g] * p.nt;
    const int mt = t.tile0[g + 1] - t.tile0[g];
    const int n = l / mt;
    return {g, t.row[g] + (l - n * mt) * bn, t.row[g + 1], n * 128};
}

template <int NC, bool RES>
__global__ void __launch_bounds__(kSmallThreads, NC <= kSmallTwoNc ? 2 : 1)
    mm_block_small_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mx,
                          const __grid_constant__ SmallParams p) {
    constexpr int bn = 2 * NC;
    constexpr int chunk_bytes = kSmallWBytes + bn * 128;
    constexpr uint32_t tmem_cols = kSmallBufs * bn;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int stage_bytes = p.per_stage * chunk_bytes;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + p.bar_offset);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kSmallBars);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const Table table = table_at(smem + p.table_offset, p.groups);
    const uint32_t ring = ptx::smem_addr(smem);
    const uint32_t bar0 = ptx::smem_addr(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
    auto tfull = [&](int b) { return bar0 + 8u * (2 * kMaxStages + b); };
    auto tempty = [&](int b) { return bar0 + 8u * (2 * kMaxStages + kSmallBufs + b); };
    const uint32_t done = bar0 + 8u * (2 * kMaxStages + 2 * kSmallBufs);

    const Factors factors = {ptx::smem_addr(smem + p.factor_offset),
                             ptx::smem_addr(smem + p.factor_offset) + kSmallFactors, kSmallWords};

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;
    const int rank = p.split > 1 ? static_cast<int>(ptx::cluster_ctarank()) : 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            ptx::mbar_init(full(s), 1);
            ptx::mbar_init(empty(s), 1);
        }
        for (int b = 0; b < kSmallBufs; ++b) {
            ptx::mbar_init(tfull(b), 1);
            ptx::mbar_init(tempty(b), 8);
        }
        ptx::mbar_init(done, 1);
        factors.init(8);
        *abort = 0;
        ptx::fence_mbar_init_cluster();
    }
    if (warp == 0 && lane == 0) {
        tc::prefetch_tensormap(&mw);
        tc::prefetch_tensormap(&mx);
    }
    if (warp == 1) {
        tc::tmem_alloc(ptx::smem_addr(tmem_slot), tmem_cols);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    ptx::griddep_launch_dependents();
    if (p.split > 1) ptx::cluster_arrive_any();  // this CTA has started
    ptx::griddep_wait();
    table_fill(table, p.offsets, p.groups, p.T, bn, 1, p.err);

    // the CTA's (cluster's) tiles, and its blocks of each
    const int first = static_cast<int>(blockIdx.x) / p.split;
    const int step = static_cast<int>(gridDim.x) / p.split;
    // (one tile of a cluster that shares it)
    const int total = p.split > 1 ? min(first + 1, table.tile0[p.groups] * p.nt) : table.tile0[p.groups] * p.nt;
    const int c0 = static_cast<int>(static_cast<int64_t>(p.chunks) * rank / p.split);
    const int c1 = static_cast<int>(static_cast<int64_t>(p.chunks) * (rank + 1) / p.split);

    if (warp == 0) {
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0;
            int64_t issued = 0;
            for (int i = first; i < total; i += step) {
                const SmallTile t = small_tile(p, table, i, bn);
                for (int c = c0; c < c1; c += p.per_stage) {
                    wait_bar(empty(s), ph ^ 1, abort, p.err);
                    const int n = min(p.per_stage, c1 - c);
                    ptx::mbar_arrive_expect_tx(full(s), static_cast<uint32_t>(n * chunk_bytes));
                    for (int j = 0; j < n; ++j) {
                        const uint32_t sa = ring + s * stage_bytes + j * chunk_bytes;
                        tc::tma_load_2d(sa, &mw, (c + j) * 128, t.g * p.N + t.n, full(s));
                        tc::tma_load_2d(sa + kSmallWBytes, &mx, (c + j) * 128, t.row, full(s));
                    }
                    ++issued;
                    if (++s == p.stages) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
            // every copy has landed once the last full phase of each stage completed
            for (int j = 0; j < p.stages && j < issued; ++j) {
                const int64_t k = issued - 1 - j;
                drain_bar(full(static_cast<int>(k % p.stages)),
                          static_cast<uint32_t>((k / p.stages) & 1), p.err);
            }
        }
    } else if (warp == 1) {
        // the whole warp walks, so that descriptors are uniform values (mm_block_pair.cuh)
        const uint32_t idesc = tc::idesc_bf16_f32(128, bn, false, false, true);
        int s = 0;
        uint32_t ph = 0;
        int it = 0;
        for (int i = first; i < total; i += step) {
            for (int c = c0; c < c1; c += p.per_stage) {
                wait_bar(full(s), ph, abort, p.err);
                const int n = min(p.per_stage, c1 - c);
                for (int j = 0; j < n; ++j, ++it) {
                    const int b = it % kSmallBufs;
                    const uint32_t sa = ring + s * stage_bytes + j * chunk_bytes;
                    const uint64_t wd = tc::smem_desc_sw128(sa, 16, 1024);
                    const uint64_t xd = tc::smem_desc_sw128(sa + kSmallWBytes, 16, 1024);
                    wait_bar(tempty(b), ((it / kSmallBufs) & 1) ^ 1, abort, p.err);
                    __syncwarp();
                    tc::fence_after_sync();
                    if (lane == 0) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)  // (32 bytes on: 2 in a descriptor)
                            tc::mma_f8(tmem + static_cast<uint32_t>(b * bn), wd + 2 * k, xd + 2 * k, idesc, k != 0);
                        tc::mma_commit(tfull(b));
                    }
                    __syncwarp();
                }
                if (lane == 0) tc::mma_commit(empty(s));
                if (++s == p.stages) {
                    s = 0;
                    ph ^= 1;
                }
            }
        }
        if (lane == 0) {
            tc::mma_commit(done);
            drain_bar(done, 0, p.err);
        }
        __syncwarp();
    } else if (warp == 10) {
        Slot at;
        for (int i = first; i < total; i += step) {
            const SmallTile t = small_tile(p, table, i, bn);
            const int64_t w0 = static_cast<int64_t>(t.g) * p.scale_rows;
            for (int c = c0; c < c1; c += kFactorBatch) {
                wait_bar(factors.empty(at.s), at.ph ^ 1, abort, p.err);
                const uint32_t to = factors.at(at.s);
                if (p.block == 1)
                    factors_copy<128>(to, kSmallWords, p.ws + c, w0 + t.n, p.ws_ld, p.N - t.n, c1 - c, lane);
                else
                    factors_copy<8>(to, kSmallWords, p.ws + c, w0 + t.n / 128, p.ws_ld, 1, c1 - c, lane);
                factors_copy<bn>(to + 512, kSmallWords, p.xs + c, t.row, p.xs_ld, t.end - t.row, c1 - c, lane);
                factors_done(factors, at.s);
                at.next();
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        const int half = (warp - 2) >> 2;
        const int wrow = (warp & 3) * 32 + lane;  // weight row of the tile
        const uint32_t tbase = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + half * NC;
        const float *slots = reinterpret_cast<const float *>(smem + p.factor_offset);
        const int wf = p.block == 1 ? wrow : 0;
        float *part = reinterpret_cast<float *>(smem + p.part_offset);
        Slot at;
        int it = 0;
        for (int i = first; i < total; i += step) {
            const SmallTile t = small_tile(p, table, i, bn);
            const int n = t.n + wrow;
            const int row = t.row + half * NC;  // of x: this thread's first
            // rows of x whose sums this thread stores, from `row` (split: below)
            constexpr bool kAhead = RES && NC <= 8;  // (more would take the sums' registers)
            uint16_t res[kAhead ? NC : 1];
            if constexpr (kAhead) {
                if (p.split == 1) {
#pragma unroll
                    for (int j = 0; j < NC; ++j)
                        res[j] = n < p.N && row + j < t.end
                                     ? p.residual[static_cast<int64_t>(row + j) * p.residual_ld + n]
                                     : 0;
                }
            }
            float acc[NC];
#pragma unroll
            for (int j = 0; j < NC; ++j) acc[j] = 0.f;
            const float *f = nullptr;
#pragma unroll 1
            for (int c = c0; c < c1; ++c, ++it) {
                if ((c - c0) % kFactorBatch == 0) {
                    if (c > c0) {
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(factors.empty(at.s));
                        at.next();
                    }
                    wait_bar(factors.full(at.s), at.ph, abort, p.err);
                    f = slots + at.s * (kFactorBatch * kSmallWords);
                } else {
                    f += kSmallWords;
                }
                const float w = f[wf];
                const int b = it % kSmallBufs;
                wait_bar(tfull(b), (it / kSmallBufs) & 1, abort, p.err);
                __syncwarp();  // what follows takes the whole warp
                tc::fence_after_sync();
                constexpr int kPiece = NC < 32 ? NC : 32;
#pragma unroll
                for (int h = 0; h < NC; h += kPiece) {
                    uint32_t d[kPiece];
                    if constexpr (NC == 8)
                        tc::tmem_ld8(tbase + b * bn, d);
                    else if constexpr (NC == 16)
                        tc::tmem_ld16(tbase + b * bn, d);
                    else
                        tc::tmem_ld32(tbase + b * bn + h, d);
                    tc::tmem_ld_wait();
                    if (h + kPiece == NC) {
                        tc::fence_before_sync();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(tempty(b));
                    }
#pragma unroll
                    for (int j = 0; j < kPiece; j += 4) {
                        const float4 x4 = *reinterpret_cast<const float4 *>(f + 128 + half * NC + h + j);
                        float *to = acc + h + j;
                        to[0] = fmaf(__uint_as_float(d[j]), x4.x * w, to[0]);
                        to[1] = fmaf(__uint_as_float(d[j + 1]), x4.y * w, to[1]);
                        to[2] = fmaf(__uint_as_float(d[j + 2]), x4.z * w, to[2]);
                        to[3] = fmaf(__uint_as_float(d[j + 3]), x4.w * w, to[3]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(factors.empty(at.s));
            at.next();
            if (p.split == 1) {
                uint16_t *y = p.y + static_cast<int64_t>(row) * p.y_ld + n;
#pragma unroll
                for (int j = 0; j < NC; ++j)
                    if (n < p.N && row + j < t.end) {
                        float v = acc[j];
                        if constexpr (kAhead)
                            v += act::from16(res[j], p.f16);
                        else if constexpr (RES)
                            v += act::from16(p.residual[static_cast<int64_t>(row + j) * p.residual_ld + n], p.f16);
                        y[static_cast<int64_t>(j) * p.y_ld] = act::to16(v, p.f16);
                    }
            } else {
                // [from][own rows of x][128 weight rows]
                const int own = (bn + p.split - 1) / p.split;
                ptx::cluster_wait_any();
                const uint32_t at = ptx::smem_addr(part) + 4u * (rank * own * 128 + wrow);
#pragma unroll
                for (int j = 0; j < NC; ++j) {
                    const int r = half * NC + j, to = r / own;
                    ptx::st_dsmem_u32(ptx::mapa(at + 512u * (r - to * own), to), __float_as_uint(acc[j]));
                }
                ptx::cluster_sync_any();
                for (int r = half; r < own; r += 2) {
                    const int64_t to = t.row + rank * own + r;
                    if (n >= p.N || to >= t.end || rank * own + r >= bn) continue;
                    float v = 0.f;
                    for (int from = 0; from < p.split; ++from) v += part[(from * own + r) * 128 + wrow];
                    if constexpr (RES) v += act::from16(p.residual[to * p.residual_ld + n], p.f16);
                    p.y[to * p.y_ld + n] = act::to16(v, p.f16);
                }
            }
        }
    }
    if (p.split > 1 && (warp < 2 || warp == 10 || first >= total)) {
        ptx::cluster_wait_any();
        if (first < total) ptx::cluster_sync_any();  // as the epilogue warps, once
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, tmem_cols);
    }
}

}  // namespace mmb
}  // namespace vlmce
