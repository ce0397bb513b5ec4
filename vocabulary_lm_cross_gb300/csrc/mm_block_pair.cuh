// mm_block_pair.cuh -- products with block scales on CTA pairs (mm_pair.cuh): tiles of
// 256 x 256, each CTA with 128 rows of operand A and all 256 of B in its accumulators.
//
//   forward   A = x (rows of one group), B = the group's weight
//   dweight   A = dyt, B = xt, over a group's part of their common columns
//
// A block's sums are in one of two TMEM buffers while the next block's form in the other;
// eight epilogue warps, each with 32 rows x 128 columns of running sums in registers (128 a
// thread; the control warps give theirs up), empty it.  A's factor is a thread's own.  B's is
// one for the 128 columns (a weight's blocks of 128 x 128: acc += (a b) d, a row a lane, 16
// columns a load), or one for each column (B_ROWS: twice the arithmetic).  For those the sums
// come 16 rows x 32 columns a load, two columns of a group of eight in each lane, so that a
// lane has 32 of the columns' factors and keeps them in registers for all its rows (each of
// them read from shared memory by all lanes, 428 us instead of 349 at the size below).
//
// What bounds it: the time that the epilogue warps need to take a block's sums out, about 910
// clocks (dweight 1375; forward with a scale for each weight row 1490, 28 bytes spilled), where
// the products take 512 and their hand-over 400 (two buffers: (512 + 400 + the time a buffer is
// being read) / 2).  No unit is near its rate meanwhile (ncu, 4864 x 4096 x 4096 with a scale
// for 128 weight rows, for each, and a dweight: issue slots 44, 41 and 36 %, FMA pipe 32, 35 and
// 30 %, tensor pipe 49, 29 and 25 %): each warp goes from a load through its wait to the
// multiply-adds in a line, and two of them a scheduler do not cover the latencies.  Beside its
// blocks a tile takes 1.7 us (dweight into fp32 2.5, 16 bits 2.9, scale for each row 3.0).
// 8192 x 8192 x 4096 233 us = 2.36 PFLOP/s (one scale for a whole row, without this
// epilogue: linear_fwd 159 us), with a scale for each weight row 389 us, dweight into fp32 354 us.
// Tried: loads of 32 columns (255 us) and of 8 (247), a load ahead of its sums (273), two
// blocks an iteration (357), single instead of packed multiply-adds (254), four buffers of 128
// columns (330), 256 x 192 tiles on twelve warps without a change of registers (292), other
// splits of the registers (268).  One commit per block: "the stage is free" and "the block's
// sums are there" are the same event, and both CTAs' epilogue warps wait on the stage's
// barrier, as the copies do (a commit for each 267 us).
//
// What most tiles take to memory stands apart from the other ways out: unrolled among them, its
// instructions came from afar, and a tile's output took 4000 clocks (8192 rows of 16 experts, K
// 4096, N 4096 293 us, now 274; 9728 x 8192, K 256 50 and 46; one rolled loop for all the others
// is slower, N 16241 86 us instead of 48).
//
// A tile of dweight is stored in 32 x 32 pieces from two buffers a warp; it costs the
// epilogue about 2900 clocks (4096 x 4096, 1024 rows: 36.0 us, without the stores 29.8).  Three
// buffers, or several pieces handed over at once, were not faster (36.8, 37.3).  Its fp32 map
// has the matrices as a third dimension, so that a matrix's last rows leave like any others
// (34 of 223 x 3568 46 -> 22 us).
//
// The tiles are dealt out in order; a group's tiles go down 8 tiles of rows before they go
// across, so those in flight share operands.
//
// Warps: 0 and 2 fetch A and B, 1 TMEM and MMA issuer, 3 fetches the factors, 4-11 epilogue.
#pragma once

#include <cuda.h>

#include "mm_block.cuh"
#include "mm_pair.cuh"

namespace vlmce {
namespace mmb {

constexpr int kPairThreads = 384;
constexpr int kPairN = 256;
constexpr int kPairEpiWarps = 8;
constexpr int kPairCols = 4 * kPairN / kPairEpiWarps;  // columns of a warp
constexpr int kControlRegs = 56, kEpilogueRegs = 224;
static_assert((kControlRegs + 2 * kEpilogueRegs) * 128 <= 65536 / kPairThreads / 8 * 8 * kPairThreads,
              "more registers than a launch has");
constexpr int kPairBBytes = kPairN / 2 * 128;  // a CTA's part of B, of a block
constexpr int kPairChunk = mm::kOpBytes + kPairBBytes;
constexpr int kPairGroupM = 8;
// Shared memory: mm_pair.cuh's, whose ring and output buffers are these instead.
// Five stages' room, of which the ring takes four; the last one's memory is a second output
// buffer of each warp, and with a factor for each column where sums change their layout.
constexpr int kPairStages = 5;
constexpr int kPairStagesUsed = 4;
static_assert(kPairEpiWarps * mm::kOutBytes <= kPairChunk, "32 x 32 sums of each warp");
constexpr int kPairWords = factor_words(128 + kPairN);  // a block's factors: the CTA's rows of A, the columns
constexpr int kPairOutAt = kPairStages * kPairChunk;
constexpr int kPairFactorsAt = kPairOutAt + kPairEpiWarps * mm::kOutBytes;
constexpr int kPairBarsAt = kPairFactorsAt + 4 * kFactorSlots * kFactorBatch * kPairWords + kFactorBarBytes;
constexpr int kPairTableAt = kPairBarsAt + 16;
static_assert(kPairTableAt + table_bytes(VLMCE_MOE_MAX_EXPERTS) <= mm::kRingBytes + mm::kEpiWarps * mm::kOutBytes,
              "in mm_pair.cuh's ring and output buffers");
static_assert(kPairOutAt % 1024 == 0, "the output buffers' swizzle");

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
        const int r0 = t.row[g], rows = t.row[g + 1] - r0;
        return {g, (l - n * p.mt) * 256, p.N, n * kPairN, r0 / 128, (rows + 127) / 128};
    } else {
        const int g = group_of(t, p.groups, i / p.nt);
        const int l = i - t.tile0[g] * p.nt, mt = t.tile0[g + 1] - t.tile0[g];
        const int per = kPairGroupM * p.nt, q = l / per, r = l - q * per;
        const int gm = min(kPairGroupM, mt - q * kPairGroupM), n = r / gm;
        return {g, t.row[g] + (q * kPairGroupM + r - n * gm) * 256, t.row[g + 1], n * kPairN, 0, p.chunks};
    }
}

// 32 x 32 sums as tmem_ld_16x32 lays them out (v[16 i + 4 g + 2 r + e]: row 16 i + 8 r +
// lane / 4, column 8 g + 2 (lane % 4) + e) into a buffer of 32 rows of 128 bytes, as a TMA
// store takes them.
__device__ __forceinline__ void put_fragment(const float (&v)[32], unsigned char *buf, int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = 8 * i + (lane >> 2);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int unit = 2 * g + ((lane & 3) >> 1);  // of 16 bytes
            *reinterpret_cast<float2 *>(buf + row * 128 + ((unit ^ (row & 7)) << 4) + 8 * (lane & 1)) =
                make_float2(v[16 * (i >> 1) + 4 * g + 2 * (i & 1)], v[16 * (i >> 1) + 4 * g + 2 * (i & 1) + 1]);
        }
    }
}
// The same, to a row per lane.
__device__ __forceinline__ void to_rows(float (&v)[32], unsigned char *buf, int lane) {
    if (lane == 0) tc::bulk_wait_read();
    __syncwarp();
    put_fragment(v, buf, lane);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float4 u = *reinterpret_cast<const float4 *>(buf + lane * 128 + ((j ^ (lane & 7)) << 4));
        v[4 * j] = u.x, v[4 * j + 1] = u.y, v[4 * j + 2] = u.z, v[4 * j + 3] = u.w;
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

// 64 columns of 32 rows (a row a lane) of an output whose rows are whole 16-byte units apart,
// on their way by a TMA store; where the group ends before the last row, the rows there are in
// such units.  The columns after a row's last whole unit singly.
template <bool F16>
__device__ __forceinline__ void put_units(const mm::Out &y, int64_t row0, int64_t end, int col, const uint64_t *acc,
                                          int cols, unsigned char *buf, int lane) {
    // (of two buffers in turn: the store before this one may still read the other)
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
    __syncwarp();
    unsigned char *row = buf + lane * 128;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float a, b;
            unpack2(acc[4 * j + k], a, b);
            w[k] = act::pack16x2(a, b, F16);
        }
        *reinterpret_cast<uint4 *>(row + ((j ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (row0 + 32 <= end) {
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && cols - col >= 8) tc::tma_store_2d(y.map, ptx::smem_addr(buf), col, static_cast<int>(row0));
    } else {
        __syncwarp();
        const int unit = lane & 7, rows = static_cast<int>(end - row0);
        if (col + 8 * unit + 8 <= cols) {
            uint16_t *to = y.base + row0 * y.ld + col + 8 * unit;
#pragma unroll 1
            for (int r = lane >> 3; r < rows; r += 4)
                *reinterpret_cast<uint4 *>(to + r * y.ld) =
                    *reinterpret_cast<const uint4 *>(buf + r * 128 + ((unit ^ (r & 7)) << 4));
        }
    }
    if (lane == 0) tc::bulk_commit();
    mm::put_rest(y, row0, col, end, cols, reinterpret_cast<const uint32_t *>(buf), lane);
}

template <bool DW, bool B_ROWS>
__global__ void __launch_bounds__(kPairThreads, 1)
    mm_block_pair_kernel(const __grid_constant__ PairMaps maps, const __grid_constant__ PairParams p) {
    extern __shared__ unsigned char smem_raw[];
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        tc::prefetch_tensormap(&maps.a);
        tc::prefetch_tensormap(&maps.b);
    }
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                            ~static_cast<uintptr_t>(1023));
    const uint32_t smem_at = ptx::smem_addr(smem);
    const Factors factors = {smem_at + kPairFactorsAt, smem_at + kPairFactorsAt + 4 * kFactorSlots * kFactorBatch * kPairWords, kPairWords};
    const uint32_t buf_empty = smem_at + kPairBarsAt;  // [2], the leader's
    if (threadIdx.x == 0) {
        factors.init(kPairEpiWarps);
        for (int b = 0; b < 2; ++b) ptx::mbar_init(buf_empty + 8u * b, 2 * kPairEpiWarps);  // of both CTAs
    }
    mm::Pair<1> q = mm::pair_setup<1>(smem_raw, p.err, 1, kPairChunk);
    q.stages = kPairStagesUsed;
    const Table table = table_at(smem + kPairTableAt, p.groups);
    table_fill(table, p.offsets, p.groups, p.T, DW ? 1 : 256, DW ? 128 : 1, p.err);
    const uint32_t tmem = __shfl_sync(0xffffffffu, q.tmem, 0);
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
                    const int row = warp == 0 ? t.row + mm::kHalfRows * rank
                                              : (DW ? t.col : t.g * p.N + t.col) + kPairN / 2 * rank;
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
            if (rank == 0) {
                // The whole warp walks, so that descriptors and addresses are uniform values
                // (in a branch of one lane each product waited about 100 clocks for them).
                const uint32_t idesc = tc::idesc_bf16_f32(256, kPairN, false, false, true);
                mm::Ring<1> r;
                int it = 0;
                for (int i = first; i < total; i += step) {
                    const int chunks = __shfl_sync(0xffffffffu, pair_tile<DW>(p, table, i).chunks, 0);
                    for (int c = 0; c < chunks; ++c, ++it) {
                        const int b = it & 1;
                        const uint32_t d = tmem + static_cast<uint32_t>(b * 256);
                        wait_bar(q.full(r.s), r.ph, q.abort, q.err);
                        const uint64_t ad = tc::smem_desc_sw128(q.chunk(r.s, 0), 16, 1024);
                        const uint64_t bd = tc::smem_desc_sw128(q.chunk(r.s, 0) + mm::kOpBytes, 16, 1024);
                        wait_bar<true>(buf_empty + 8u * b, ((it >> 1) & 1) ^ 1, q.abort, q.err);
                        __syncwarp();
                        tc::fence_after_sync();
                        if (lane == 0) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)  // (32 bytes on: 2 in a descriptor)
                                tc::mma_f8_pair(d, ad + 2 * k, bd + 2 * k, idesc, k != 0);
                            // in both CTAs: the stage is free, and its block's sums are there
                            tc::mma_commit_pair(q.empty(r.s), 3u);
                        }
                        __syncwarp();
                        r.next(q);
                    }
                }
                if (lane == 0) mm::mma_finish(q);
            }
        } else {
            Slot at;
            for (int i = first; i < total; i += step) {
                const PairTile t = pair_tile<DW>(p, table, i);
                const int row = t.row + mm::kHalfRows * rank;
                for (int c = 0; c < t.chunks; c += kFactorBatch) {
                    wait_bar(factors.empty(at.s), at.ph ^ 1, q.abort, q.err);
                    const uint32_t to = factors.at(at.s);
                    const int n = t.chunks - c;
                    factors_copy<128>(to, kPairWords, p.as + t.c0 + c, row, p.as_ld, t.end - row, n, lane);
                    if constexpr (B_ROWS) {
                        factors_copy<kPairN>(to + 512, kPairWords, p.bs + t.c0 + c,
                                             DW ? t.col : static_cast<int64_t>(t.g) * p.N + t.col, p.bs_ld,
                                             (DW ? p.K : p.N) - t.col, n, lane);
                    } else {
                        // of the columns' two blocks
                        factors_copy<8>(to + 512, kPairWords, p.bs + c,
                                        static_cast<int64_t>(t.g) * p.scale_rows + t.col / 128, p.bs_ld,
                                        min(2, p.scale_rows - t.col / 128), n, lane);
                    }
                    factors_done(factors, at.s);
                    at.next();
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpilogueRegs));
        const int part = kPairCols * ((warp - 4) >> 2);  // the warp's first column of the tile
        uint32_t *buf = reinterpret_cast<uint32_t *>(smem + kPairOutAt + (warp - 4) * mm::kOutBytes);
        unsigned char *scratch = smem + kPairStagesUsed * kPairChunk + (warp - 4) * mm::kOutBytes;
        const float *slots = reinterpret_cast<const float *>(smem + kPairFactorsAt);
        const uint32_t empty_leader = ptx::mapa(buf_empty, 0);
        const int in_tile = mm::kHalfRows * rank + (warp & 3) * 32;  // the warp's first row
        const int cols = DW ? p.K : p.N;
        Slot at;
        mm::Ring<1> r;
        int it = 0, turn = 0;  // turn: of the output buffers, over all tiles
        for (int i = first; i < total; i += step) {
            const PairTile t = pair_tile<DW>(p, table, i);
            const int block = 128 + (DW ? 0 : ((t.col + part) >> 7) - (t.col >> 7));  // B's factor in a slot
            uint64_t acc[kPairCols / 2];  // two columns each
#pragma unroll
            for (int j = 0; j < kPairCols / 2; ++j) acc[j] = 0;
            const float *f = slots;
            auto advance = [&](int c) {  // f: block c's factors, in order
                if (c % kFactorBatch == 0) {
                    if (c > 0) {
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(factors.empty(at.s));
                        at.next();
                    }
                    wait_bar(factors.full(at.s), at.ph, q.abort, q.err);
                    f = slots + at.s * (kFactorBatch * kPairWords);
                } else {
                    f += kPairWords;
                }
            };
            const uint32_t d0 = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + part;
#pragma unroll 1
            for (int c = 0; c < t.chunks; ++c, ++it) {
                advance(c);
                // (fetching it a block ahead costs: 237 -> 267 us)
                float af[B_ROWS ? 4 : 1];
#pragma unroll
                for (int i = 0; i < (B_ROWS ? 4 : 1); ++i)
                    af[i] = f[(warp & 3) * 32 + (B_ROWS ? 8 * i + (lane >> 2) : lane)];
                if constexpr (!B_ROWS) af[0] *= f[block];
                uint64_t b[B_ROWS ? 16 : 1];
                if constexpr (B_ROWS) {
#pragma unroll
                    for (int g = 0; g < 16; ++g)
                        b[g] = *reinterpret_cast<const uint64_t *>(f + 128 + part + 8 * g + 2 * (lane & 3));
                }
                wait_bar(q.empty(r.s), r.ph, q.abort, q.err);
                r.next(q);
                __syncwarp();  // each lane left the wait by itself; TMEM loads take the whole warp
                tc::fence_after_sync();
                const uint32_t from = d0 + 256 * (it & 1);
                auto release = [&] {
                    tc::fence_before_sync();
                    __syncwarp();
                    // (TMEM was read, nothing written: the fences of tcgen05 order it across the
                    // cluster, and a release's fence took longer than the sums)
                    if (lane == 0) ptx::mbar_remote_arrive_relaxed(empty_leader + 8u * (it & 1));
                };
                if constexpr (B_ROWS) {
#pragma unroll
                    for (int h = 0; h < kPairCols; h += 32) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {  // 16 rows each
                            uint32_t d[16];
                            tc::tmem_ld_16x32(from + (static_cast<uint32_t>(16 * i) << 16) + h, d);
                            tc::tmem_ld_wait();
                            if (h + 32 == kPairCols && i == 1) release();
                            uint64_t *to = acc + h / 2 + 8 * i;
#pragma unroll
                            for (int g = 0; g < 4; ++g) {
                                to[2 * g] = fma2(pack2(d[4 * g], d[4 * g + 1]), mul2(b[h / 8 + g], both(af[2 * i])), to[2 * g]);
                                to[2 * g + 1] = fma2(pack2(d[4 * g + 2], d[4 * g + 3]), mul2(b[h / 8 + g], both(af[2 * i + 1])),
                                                     to[2 * g + 1]);
                            }
                        }
                    }
                } else {
                    const uint64_t a = both(af[0]);
#pragma unroll
                    for (int h = 0; h < kPairCols; h += 16) {
                        uint32_t d[16];
                        tc::tmem_ld16(from + h, d);
                        tc::tmem_ld_wait();
                        if (h + 16 == kPairCols) release();
                        uint64_t *to = acc + h / 2;
#pragma unroll
                        for (int j = 0; j < 8; ++j) to[j] = fma2(pack2(d[2 * j], d[2 * j + 1]), a, to[j]);
                    }
                }
            }
            if (t.chunks > 0) {
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(factors.empty(at.s));
                at.next();
            }
            const int64_t out0 = DW ? static_cast<int64_t>(t.g) * p.N : 0;  // dweight: a group's first row of y
            const int64_t row0 = out0 + t.row + in_tile, end = out0 + t.end;
            const int col0 = t.col + part;
            if (row0 < end && col0 < cols && !(p.add && t.chunks == 0)) {
                const bool whole = p.vec >= 16 && row0 + 32 <= end;
                const bool f16 = p.out == VLMCE_F16;
                const mm::Out y = {static_cast<uint16_t *>(p.y), p.y_ld, whole ? 16 : 2, &maps.y};
                // What most tiles take stands by itself: among the other ways out, unrolled with
                // them, its instructions came from afar.
                bool done = false;
                if constexpr (DW) {
                    if (p.out == VLMCE_F32 && p.vec >= 16) {
                        done = true;
#pragma unroll
                        for (int s = 0; s < kPairCols / 32; ++s) {
                            const int col = col0 + 32 * s;
                            if (col >= cols) break;
                            float v[32];
#pragma unroll
                            for (int j = 0; j < 16; ++j) unpack2(acc[16 * s + j], v[2 * j], v[2 * j + 1]);
                            // from two buffers in turn: the store before this one may still read
                            unsigned char *from = turn ? scratch : reinterpret_cast<unsigned char *>(buf);
                            turn ^= 1;
                            if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                            __syncwarp();
                            put_fragment(v, from, lane);
                            ptx::fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) {
                                // (rows behind the matrix's last are not stored)
                                if (p.add)
                                    tc::tma_add_3d(&maps.y, ptx::smem_addr(from), col, t.row + in_tile, t.g);
                                else
                                    tc::tma_store_3d(&maps.y, ptx::smem_addr(from), col, t.row + in_tile, t.g);
                                tc::bulk_commit();
                            }
                        }
                    }
                } else if constexpr (!B_ROWS) {
                    if (p.vec >= 16 && !p.residual) {
                        done = true;
                        const mm::Out units = {static_cast<uint16_t *>(p.y), p.y_ld, 16, &maps.y};
#pragma unroll
                        for (int s = 0; s < kPairCols / 64; ++s) {
                            const int col = col0 + 64 * s;
                            if (col >= cols) break;
                            unsigned char *from = turn ? scratch : reinterpret_cast<unsigned char *>(buf);
                            turn ^= 1;
                            if (f16)
                                put_units<true>(units, row0, end, col, acc + 32 * s, cols, from, lane);
                            else
                                put_units<false>(units, row0, end, col, acc + 32 * s, cols, from, lane);
                        }
                    }
                }
                if (!done) {
#pragma unroll
                for (int s = 0; s < kPairCols / 32; ++s) {
                    const int col = col0 + 32 * s;
                    float v[32];
#pragma unroll
                    for (int j = 0; j < 16; ++j) unpack2(acc[16 * s + j], v[2 * j], v[2 * j + 1]);
                    if constexpr (B_ROWS) to_rows(v, scratch, lane);
                    if constexpr (DW) {
                        if (p.out == VLMCE_F32) {
                            if (col < cols)
                                put_f32_rows(static_cast<float *>(p.y), p.y_ld, row0, col, v, end, cols, p.add != 0,
                                             buf, lane);
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
                    const int pair = col0 + 64 * (s / 2);  // the 64 columns of a store
                    if (pair < cols) {
                        mm::put_seg(y, row0, pair, s & 1, v, end, cols, f16, buf, lane);
                        if (s & 1) mm::put_rest(y, row0, pair, end, cols, buf, lane);
                    }
                }
                }
            }
        }
        if (lane == 0) tc::bulk_wait();
    }
    mm::pair_teardown(q);
}

}  // namespace mmb
}  // namespace vlmce
