// mm_block_pair.cuh -- products with block scales on CTA pairs (mm_pair.cuh): tiles of
// 256 x 256, each CTA with 128 rows of operand A and all 256 of B in its accumulators.
//
//   forward   A = x (rows of one group), B = the group's weight
//   dweight   A = dyt, B = xt, over a group's part of their common columns
//
// A pair's products of one block (128 of K) take about 540 clocks at the tensor cores'
// rate, and so long the other TMEM buffer has to be emptied: 8 epilogue warps, each with 32
// rows x 128 columns of sums in registers (128 a thread, 224 with what else it needs: the
// control warps give theirs up), 64 columns a load.  A's factor is a thread's own.  B's is
// one for the 128 columns (a weight's blocks of 128 x 128: acc += (a b) d, one packed
// multiply-add), or one for each column (B_ROWS), put into shared memory by the lanes that
// fetched them.  Factors are fetched some blocks ahead.
//
// The tiles are dealt out in order; a group's tiles go down 8 tiles of rows before they go
// across, so those in flight share operands.
//
// Warps: 0 and 2 fetch A and B, 1 TMEM and MMA issuer, 3 idle, 4-11 epilogue.
#pragma once

#include <cuda.h>

#include "mm_block.cuh"
#include "mm_pair.cuh"

namespace vlmce {
namespace mmb {

constexpr int kPairStages = 5;  // of mm_pair.cuh's ring; its last chunk's memory is the
                                // groups' table and the columns' factors
constexpr int kPairFactors = 8 * 2 * 128 * 4;
constexpr int kPairGroupM = 8;
constexpr int kControlRegs = 56, kEpilogueRegs = 224;
static_assert((kControlRegs + 2 * kEpilogueRegs) * 128 <= 65536 / mm::kPairThreads / 8 * 8 * mm::kPairThreads,
              "more registers than a launch has");
static_assert(kPairFactors + table_bytes(VLMCE_MOE_MAX_EXPERTS) <= mm::kChunkBytes, "in one chunk");

struct PairMaps {
    CUtensorMap a, b, y;
};

struct PairTile {
    int g, row, end, col;  // group; first row of A (dweight: of its dw) and its end; first column
    int c0, chunks;        // blocks of K
};
template <bool DW>
__device__ __forceinline__ PairTile pair_tile(const PairParams &p, const Table &t, int i) {
    if constexpr (DW) {
        const int per = p.mt * p.nt, g = i / per, l = i - g * per, n = l / p.mt;
        const int r0 = t.row0[g], rows = t.row1[g] - r0;
        return {g, (l - n * p.mt) * 256, p.N, n * 256, r0 / 128, (rows + 127) / 128};
    } else {
        const int g = group_of(t, p.groups, i / p.nt);
        const int l = i - t.tile0[g] * p.nt, mt = t.tile0[g + 1] - t.tile0[g];
        const int per = kPairGroupM * p.nt, q = l / per, r = l - q * per;
        const int gm = min(kPairGroupM, mt - q * kPairGroupM), n = r / gm;
        return {g, t.row0[g] + (q * kPairGroupM + r - n * gm) * 256, t.row1[g], n * 256, 0, p.chunks};
    }
}

// 32 rows x 32 columns of fp32 whose rows TMA cannot take: through the warp's buffer, so
// that its accesses cover consecutive addresses.
__device__ __forceinline__ void put_f32_rows(float *base, int64_t ld, int64_t row0, int col, const float (&v)[32],
                                             int64_t rows, int cols, bool add, uint32_t *buf, int lane) {
    mm::buffer_free(lane);
    float *f = reinterpret_cast<float *>(buf);
#pragma unroll
    for (int j = 0; j < 32; ++j) f[lane * 32 + (j ^ lane)] = v[j];
    __syncwarp();
    const int nr = static_cast<int>(min(int64_t{32}, rows - row0));
    float *to = base + row0 * ld + col + lane;
    if (col + lane < cols) {
#pragma unroll 4
        for (int r = 0; r < nr; ++r) {
            const float x = f[r * 32 + (lane ^ r)];
            to[r * ld] = add ? to[r * ld] + x : x;
        }
    }
}

// G blocks' factors: of a thread's row of A, and of B's columns lane, lane + 32, .. (B_ROWS)
// or of its rows' block.
template <bool B_ROWS, int G>
struct PairScales {
    float a[G], b[B_ROWS ? 4 : 1][G];
};

template <bool DW, bool B_ROWS>
__global__ void __launch_bounds__(mm::kPairThreads, 1)
    mm_block_pair_kernel(const __grid_constant__ PairMaps maps, const __grid_constant__ PairParams p) {
    extern __shared__ unsigned char smem_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        tc::prefetch_tensormap(&maps.a);
        tc::prefetch_tensormap(&maps.b);
    }
    mm::Pair<1> q = mm::pair_setup<1>(smem_raw, p.err, 1);
    q.stages = kPairStages;
    unsigned char *rest = q.smem + kPairStages * mm::kChunkBytes;
    const Table table = table_at(rest + kPairFactors, p.groups);
    table_fill(table, p.offsets, p.groups, p.T, DW ? 1 : 256, DW ? 128 : 1, p.err);
    const int rank = static_cast<int>(q.rank);
    const int first = static_cast<int>(ptx::cluster_id_x()), step = static_cast<int>(ptx::ncluster_x());
    const int total = DW ? p.groups * p.mt * p.nt : table.tile0[p.groups] * p.nt;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kControlRegs));
        if (warp == 0 || warp == 2) {
            if (lane == 0) {
                const uint32_t full_leader = ptx::mapa(q.full(0), 0);
                mm::Ring<1> r;
                int64_t issued = 0;
                for (int i = first; i < total; i += step) {
                    const PairTile t = pair_tile<DW>(p, table, i);
                    const int row = (warp == 0 ? t.row : DW ? t.col : t.g * p.N + t.col) + mm::kHalfRows * rank;
                    for (int c = 0; c < t.chunks; ++c) {
                        if (warp == 0) {
                            mm::stage_begin<true, 1>(q, r, 1);
                            tc::tma_load_2d_pair(q.chunk(r.s, 0), &maps.a, (t.c0 + c) * 128, row,
                                                 full_leader + 8u * r.s);
                        } else {
                            mm::stage_begin<false, 1>(q, r, 1);
                            tc::tma_load_2d_pair(q.chunk(r.s, 0) + mm::kOpBytes, &maps.b, (t.c0 + c) * 128, row,
                                                 full_leader + 8u * r.s);
                        }
                        r.next(q);
                    }
                    issued += t.chunks;
                }
                if (warp == 0) mm::drain_loads(q, issued);
            }
        } else if (warp == 1) {
            if (rank == 0 && lane == 0) {
                const uint32_t idesc = tc::idesc_bf16_f32(256, 256, false, false, true);
                mm::Ring<1> r;
                int it = 0;
                for (int i = first; i < total; i += step) {
                    const int chunks = pair_tile<DW>(p, table, i).chunks;
                    for (int c = 0; c < chunks; ++c) mm::mma_tile<true, 1>(q, r, it++, 1, idesc, false, false);
                }
                mm::mma_finish(q);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpilogueRegs));
        constexpr int G = 2;
        using Scales = PairScales<B_ROWS, G>;
        const int half = (warp - 4) >> 2;
        uint32_t *buf = q.out_buffer(warp - 4);
        float *bf = reinterpret_cast<float *>(rest) + (warp - 4) * 256;  // [2][128]
        const uint32_t tempty_leader = ptx::mapa(q.tempty(0), 0);
        const int in_tile = mm::kHalfRows * rank + (warp & 3) * 32;  // the warp's first row
        const int cols = DW ? p.K : p.N;
        auto fetch = [&](Scales &f, const PairTile &t, int c) {
            const int row = t.row + in_tile + lane;
            const float *pa = p.as + static_cast<int64_t>(row) * p.as_ld + t.c0 + c;
#pragma unroll
            for (int k = 0; k < G; ++k) f.a[k] = row < t.end && c + k < t.chunks ? pa[k] : 0.f;
            if constexpr (B_ROWS) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int col = t.col + 128 * half + 32 * j + lane;
                    const int64_t at = DW ? col : static_cast<int64_t>(t.g) * p.N + col;
                    const float *pb = p.bs + at * p.bs_ld + t.c0 + c;
#pragma unroll
                    for (int k = 0; k < G; ++k) f.b[j][k] = col < cols && c + k < t.chunks ? pb[k] : 0.f;
                }
            } else {
                const int block = t.col / 128 + half;
                const float *pb = p.bs + (static_cast<int64_t>(t.g) * p.scale_rows + block) * p.bs_ld + c;
#pragma unroll
                for (int k = 0; k < G; ++k) f.b[0][k] = block < p.scale_rows && c + k < t.chunks ? pb[k] : 0.f;
            }
        };
        PairTile t = {};
        Scales next = {};
        if (first < total) {
            t = pair_tile<DW>(p, table, first);
            fetch(next, t, 0);
        }
        int it = 0;
        for (int i = first; i < total; i += step) {
            float acc[128];
#pragma unroll
            for (int j = 0; j < 128; ++j) acc[j] = 0.f;
            if (t.chunks == 0 && i + step < total) fetch(next, pair_tile<DW>(p, table, i + step), 0);
#pragma unroll 1
            for (int c = 0; c < t.chunks; c += G) {
                const Scales f = next;
                if (c + G < t.chunks)
                    fetch(next, t, c + G);
                else if (i + step < total)
                    fetch(next, pair_tile<DW>(p, table, i + step), 0);
#pragma unroll
                for (int k = 0; k < G; ++k) {
                    if (c + k >= t.chunks) break;
                    float *slot = bf + (it & 1) * 128;
                    if constexpr (B_ROWS) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) slot[32 * j + lane] = f.b[j][k];
                    }
                    const float a = B_ROWS ? f.a[k] : f.a[k] * f.b[0][k];
                    const uint32_t d0 = mm::acc_wait(q, it, warp) + 128 * half;
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        uint32_t d[32];
                        tc::tmem_ld32(d0 + 32 * h, d);
                        tc::tmem_ld_wait();
                        if (h == 3) mm::acc_release(tempty_leader, it, lane);
                        if constexpr (B_ROWS) {
#pragma unroll
                            for (int j = 0; j < 32; j += 4) {
                                const float4 b = *reinterpret_cast<const float4 *>(slot + 32 * h + j);
                                float *to = acc + 32 * h + j;
                                to[0] = fmaf(__uint_as_float(d[j]), b.x * a, to[0]);
                                to[1] = fmaf(__uint_as_float(d[j + 1]), b.y * a, to[1]);
                                to[2] = fmaf(__uint_as_float(d[j + 2]), b.z * a, to[2]);
                                to[3] = fmaf(__uint_as_float(d[j + 3]), b.w * a, to[3]);
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                acc[32 * h + j] = fmaf(__uint_as_float(d[j]), a, acc[32 * h + j]);
                        }
                    }
                    ++it;
                }
            }
            const int64_t out0 = DW ? static_cast<int64_t>(t.g) * p.N : 0;  // dweight: a group's first row of y
            const int64_t row0 = out0 + t.row + in_tile, end = out0 + t.end;
            const int col0 = t.col + 128 * half;
            if (row0 < end && col0 < cols && !(p.add && t.chunks == 0)) {
                const bool whole = p.vec >= 16 && row0 + 32 <= end;
                const bool f16 = p.out == VLMCE_F16;
                const mm::Out y = {static_cast<uint16_t *>(p.y), p.y_ld, whole ? 16 : 2, &maps.y};
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int col = col0 + 32 * s;
                    float v[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = acc[32 * s + j];
                    if constexpr (DW) {
                        if (p.out == VLMCE_F32) {
                            if (col < cols) {
                                if (whole) {
                                    mm::put_f32(&maps.y, row0, col, reinterpret_cast<uint32_t(&)[32]>(v),
                                                p.add != 0, buf, lane);
                                } else {
                                    put_f32_rows(static_cast<float *>(p.y), p.y_ld, row0, col, v, end, cols,
                                                 p.add != 0, buf, lane);
                                }
                            }
                            continue;
                        }
                    } else if (p.residual && row0 + lane < end && col < cols) {
                        const uint16_t *at = p.residual + (row0 + lane) * p.residual_ld + col;
                        if ((reinterpret_cast<uintptr_t>(at) & 15) == 0 && col + 32 <= cols) {
#pragma unroll
                            for (int j = 0; j < 32; j += 8) {
                                const uint4 u = *reinterpret_cast<const uint4 *>(at + j);
                                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    float a, b;
                                    act::unpack16x2(w[k], a, b, f16);
                                    v[j + 2 * k] += a;
                                    v[j + 2 * k + 1] += b;
                                }
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (col + j < cols) v[j] += act::from16(at[j], f16);
                        }
                    }
                    __syncwarp();
                    const int pair = col0 + 64 * (s / 2);  // the 64 columns of this store
                    if (pair < cols) {
                        mm::put_seg(y, row0, pair, s & 1, v, end, cols, f16, buf, lane);
                        if (s & 1) mm::put_rest(y, row0, pair, end, cols, buf, lane);
                    }
                }
            }
            if (i + step < total) t = pair_tile<DW>(p, table, i + step);
        }
        if (lane == 0) tc::bulk_wait();
    }
    mm::pair_teardown(q);
}

}  // namespace mmb
}  // namespace vlmce
