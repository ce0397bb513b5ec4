// mm_pair.cuh -- the machinery of the kernels that run on CTA pairs: a cluster of
// 2 CTAs computes tiles of 256 x 256 with tcgen05.mma.cta_group::2, each CTA
// staging its own 128 rows of either operand (128 bytes of K per row, 128-byte
// swizzle) in a ring filled by TMA.
//
// Accumulators: two of 256 fp32 TMEM columns, so the epilogue of one tile
// overlaps the products of the next.  Roles: one lane of warps 0 and 10 issues the
// TMA loads of operand A and of operand B; warp 1 allocates TMEM and, in the
// leader, one lane issues the MMAs; warps 2-9 epilogue: TMEM subpartition warp %
// 4 (one row per thread), two warps per subpartition, each on half of the
// columns; warp 11 (leader) fetches the tiles.
//
// Tiles: of long tiles one cluster each is launched, and the clusters that fit at
// once stay: each takes over the work of one that has not started (cluster launch
// control), one tile ahead of its slowest role.  So they are handed out in order as
// pairs become free, without a counter in memory.  (Dealt out in advance, T = 4096,
// K = 6656, 2n = 32768's gradient products would leave pairs idle for one of its 138
// us dx tiles.)  Short tiles are dealt out: their answers would not keep up.
//
// Operand layouts of a stage (16-bit operands): K-major, 128 rows of 64 K (8-row
// groups 1024 B apart, a K step of 16 advances 32 B); MN-major, two boxes of 64
// K rows x 64 M or N (8-row groups 1024 B apart, the boxes 8192 B apart, a K
// step of 16 rows advances 2048 B).  8-bit operands: K-major, 128 K per row.
#pragma once

#include <cuda.h>

#include "act.cuh"
#include "mbar_wait.cuh"
#include "ptx_async.cuh"
#include "tcgen05.cuh"

namespace vlmce {
namespace mm {

constexpr int kPairM = 256;                    // tokens of a pair tile
constexpr int kHalfRows = 128;                 // rows of x, and of W, staged by one CTA
constexpr int kOpBytes = kHalfRows * 128;      // one operand of a chunk (128 bytes of K): 16 KB
constexpr int kChunkBytes = 2 * kOpBytes;
constexpr int kRingChunks = 6;                 // 192 KB
constexpr int kRingBytes = kRingChunks * kChunkBytes;
constexpr int kPairThreads = 384;
constexpr int kEpiWarps = 8;
constexpr int kPairTmemCols = 512;
constexpr int kWarpB = 10, kWarpTiles = 11;
constexpr int kTileQ = 2;                      // answers about the next tile
constexpr int kTileConsumers = 5 + 2 * kEpiWarps;  // 4 producers, MMA issuer, epilogue warps
// full, empty, tmem full x2, tmem empty x2, drain, tile full x2, tile empty x2
constexpr int kPairBars = 2 * kRingChunks + 5 + 2 * kTileQ;
constexpr int kPairTail = 16 * kTileQ + 8 * kPairBars + 16;  // answers, barriers, TMEM slot, abort flag
constexpr int kOutBytes = 32 * 128;              // an epilogue warp's output buffer: 32 rows x 128 bytes
constexpr int kPairSmem = 1024 + kRingBytes + kEpiWarps * kOutBytes + kPairTail;


// A CTA's view of the pair's pipeline; PER chunks make a stage (one barrier round
// trip).  Two are faster where both operands are K-major (T 4096, K 6656, 2n 32768
// forward 1065 -> 1048 us: 256 contiguous bytes of a row are fetched together), one
// where an operand is MN-major (its gradient products 2158 against 2166 us).
template <int PER>
struct Pair {
    unsigned char *smem;  // ring, output buffers, tail
    uint32_t ring, bar0;
    volatile int *abort;
    int *err;
    uint32_t rank;        // 0: the pair's leader
    uint32_t tmem;
    int dealt;            // > 0: so many tiles are dealt out to the clusters in turn
    int chunk_bytes;      // both operands' part of a chunk
    int stages;           // of the ring

    __device__ __forceinline__ uint32_t full(int s) const { return bar0 + 8u * s; }
    __device__ __forceinline__ uint32_t empty(int s) const { return bar0 + 8u * (kRingChunks + s); }
    __device__ __forceinline__ uint32_t tfull(int b) const { return bar0 + 8u * (2 * kRingChunks + b); }
    __device__ __forceinline__ uint32_t tempty(int b) const {
        return bar0 + 8u * (2 * kRingChunks + 2 + b);
    }
    __device__ __forceinline__ uint32_t drain() const { return bar0 + 8u * (2 * kRingChunks + 4); }
    __device__ __forceinline__ uint32_t qfull(int i) const { return bar0 + 8u * (2 * kRingChunks + 5 + i); }
    __device__ __forceinline__ uint32_t qempty(int i) const {
        return bar0 + 8u * (2 * kRingChunks + 5 + kTileQ + i);
    }
    __device__ __forceinline__ uint32_t chunk(int s, int i) const {
        return ring + (s * PER + i) * chunk_bytes;
    }
    __device__ __forceinline__ uint32_t answer(int i) const {
        return ring + kRingBytes + kEpiWarps * kOutBytes + 16u * i;
    }
    __device__ __forceinline__ uint32_t *out_buffer(int epi_warp) const {
        return reinterpret_cast<uint32_t *>(smem + kRingBytes + epi_warp * kOutBytes);
    }
};

// Position in the ring.
template <int PER>
struct Ring {
    int s = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next(const Pair<PER> &q) {
        if (++s == q.stages) {
            s = 0;
            ph ^= 1;
        }
    }
};

// All threads: barriers and TMEM.  Then the next kernel of the stream may set itself up (TMEM is
// held), and this one waits for its predecessor's results before it touches
// global memory.
template <int PER>
__device__ __forceinline__ Pair<PER> pair_setup(unsigned char *smem_raw, int *err, int dealt,
                                                int chunk_bytes = kChunkBytes) {
    Pair<PER> q;
    q.dealt = dealt;
    q.chunk_bytes = chunk_bytes;
    q.stages = min(kRingChunks, kRingBytes / chunk_bytes / PER);
    q.smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint64_t *bars =
        reinterpret_cast<uint64_t *>(q.smem + kRingBytes + kEpiWarps * kOutBytes + 16 * kTileQ);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kPairBars);
    q.abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    q.ring = ptx::smem_addr(q.smem);
    q.bar0 = ptx::smem_addr(bars);
    q.err = err;
    q.rank = ptx::cluster_ctarank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < q.stages; ++s) {
            ptx::mbar_init(q.full(s), 1);   // leader: its producer + the bytes of both CTAs
            ptx::mbar_init(q.empty(s), 1);  // one commit from the leader's MMA issuer
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(q.tfull(b), 1);
            ptx::mbar_init(q.tempty(b), 2 * kEpiWarps);  // leader: both CTAs' epilogue warps
        }
        ptx::mbar_init(q.drain(), 1);
        for (int i = 0; i < kTileQ; ++i) {
            ptx::mbar_init(q.qfull(i), 1);                // the leader's fetching lane + 16 bytes
            ptx::mbar_init(q.qempty(i), kTileConsumers);  // used at the leader only
        }
        *q.abort = 0;
        ptx::fence_mbar_init_cluster();
    }
    if (threadIdx.x >> 5 == 1) {
        tc::tmem_alloc_pair(ptx::smem_addr(tmem_slot), kPairTmemCols);
        tc::tmem_relinquish_pair();
    }
    tc::fence_before_sync();
    ptx::cluster_sync_any();
    tc::fence_after_sync();
    q.tmem = *tmem_slot;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    return q;
}
// The sequence of tiles of a pair, one object per role; -1 after the last (or after a
// wait that gave up).  A role is one lane, or (WARP) a whole warp: its lane 0 reads the
// answer for all 32, so no lane is behind when it gives the slot back, and all lanes
// get the same tile.
struct Tiles {
    int j = -1;
    template <bool WARP, int PER>
    __device__ __forceinline__ int next(const Pair<PER> &q, int lane) {
        const int own = static_cast<int>(ptx::cluster_id_x());
        if (++j == 0) return own;
        if (q.dealt > 0) {
            const int64_t t = own + static_cast<int64_t>(j) * ptx::ncluster_x();
            return t < q.dealt ? static_cast<int>(t) : -1;
        }
        int t = -1;
        if (!WARP || lane == 0) {
            const int i = (j - 1) % kTileQ;
            if (wait_bar<true>(q.qfull(i), ((j - 1) / kTileQ) & 1, q.abort, q.err)) {
                t = ptx::clc_first_cta(q.answer(i));
                if (t >= 0) t >>= 1;  // two CTAs per tile
            }
            ptx::fence_proxy_async_smem();  // the answer is read before it is overwritten
            if (q.rank == 0)
                ptx::mbar_arrive(q.qempty(i));
            else
                ptx::mbar_remote_arrive_release(ptx::mapa(q.qempty(i), 0));
        }
        return WARP ? __shfl_sync(0xffffffffu, t, 0) : t;
    }
};
// The leader's fetching lane.
template <int PER>
__device__ __forceinline__ void fetch_tiles(const Pair<PER> &q) {
    if (q.dealt > 0) return;
    for (int n = 0;; ++n) {
        const int i = n % kTileQ;
        if (n >= kTileQ && !wait_bar<true>(q.qempty(i), ((n / kTileQ) - 1) & 1, q.abort, q.err))
            return;
        ptx::mbar_remote_arrive_expect_tx(ptx::mapa(q.qfull(i), 1), 16);
        ptx::mbar_arrive_expect_tx(q.qfull(i), 16);
        ptx::clc_try_cancel(q.answer(i), q.qfull(i));
        if (!wait_bar<true>(q.qfull(i), (n / kTileQ) & 1, q.abort, q.err)) return;
        if (ptx::clc_first_cta(q.answer(i)) < 0) return;
        ptx::fence_proxy_async_smem();
    }
}

// All threads, after every MMA of the pair has completed and every copy landed:
// the pair meets before TMEM is released and either CTA exits.
template <int PER>
__device__ __forceinline__ void pair_teardown(const Pair<PER> &q) {
    tc::fence_before_sync();
    __syncthreads();
    ptx::cluster_sync_any();
    if (threadIdx.x >> 5 == 1) {
        __syncwarp();
        tc::fence_after_sync();
        tc::tmem_dealloc_pair(q.tmem, kPairTmemCols);
    }
}

// Producer lanes: wait for a stage's slot, for n chunks; operand A's lane of the leader announces
// the stage's bytes (copies may land before that).
template <bool A, int PER>
__device__ __forceinline__ void stage_begin(const Pair<PER> &q, const Ring<PER> &r, int n) {
    wait_bar(q.empty(r.s), r.ph ^ 1, q.abort, q.err);
    if (A && q.rank == 0)
        ptx::mbar_arrive_expect_tx(q.full(r.s), static_cast<uint32_t>(n * 2 * q.chunk_bytes));
}
// Operand A's lane of the leader, at the end: every copy into the pair has landed
// once the full phases of the last `stages` loads completed.
template <int PER>
__device__ __forceinline__ void drain_loads(const Pair<PER> &q, int64_t issued) {
    if (q.rank != 0) return;
    for (int i = 0; i < q.stages && i < issued; ++i) {
        const int64_t k = issued - 1 - i;
        drain_bar(q.full(static_cast<int>(k % q.stages)),
                  static_cast<uint32_t>((k / q.stages) & 1), q.err);
    }
}
// MMA lane of the leader: the products of the it-th tile.
template <bool FP8, int PER>
__device__ __forceinline__ void mma_tile(const Pair<PER> &q, Ring<PER> &r, int it, int chunks, uint32_t idesc,
                                         bool a_mn, bool b_mn) {
    const int b = it & 1;
    wait_bar<true>(q.tempty(b), ((it >> 1) & 1) ^ 1, q.abort, q.err);
    tc::fence_after_sync();
    const uint32_t d = q.tmem + static_cast<uint32_t>(b * 256);
    for (int c = 0; c < chunks; c += PER) {
        wait_bar(q.full(r.s), r.ph, q.abort, q.err);
        tc::fence_after_sync();
        const int n = min(PER, chunks - c);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (i < n) {
                const uint32_t sa = q.chunk(r.s, i);
                const uint32_t sb = sa + kOpBytes;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint64_t ad = a_mn ? tc::smem_desc_sw128(sa + 2048 * k, 8192, 1024)
                                             : tc::smem_desc_sw128(sa + 32 * k, 16, 1024);
                    const uint64_t bd = b_mn ? tc::smem_desc_sw128(sb + 2048 * k, 8192, 1024)
                                             : tc::smem_desc_sw128(sb + 32 * k, 16, 1024);
                    if constexpr (FP8)
                        tc::mma_f8_pair(d, ad, bd, idesc, (c + i | k) != 0);
                    else
                        tc::mma_bf16_pair(d, ad, bd, idesc, (c + i | k) != 0);
                }
            }
        }
        tc::mma_commit_pair(q.empty(r.s), 3u);  // the stage is free in both CTAs
        r.next(q);
    }
    tc::mma_commit_pair(q.tfull(b), 3u);
}
template <int PER>
__device__ __forceinline__ void mma_finish(const Pair<PER> &q) {
    tc::mma_commit_pair(q.drain(), 1u);
    drain_bar(q.drain(), 0, q.err);
}
// Epilogue warps: the it-th tile's accumulators (TMEM address of the warp's
// lanes), and their release.
template <int PER>
__device__ __forceinline__ uint32_t acc_wait(const Pair<PER> &q, int it, int warp) {
    wait_bar(q.tfull(it & 1), (it >> 1) & 1, q.abort, q.err);
    __syncwarp();  // each lane left the wait by itself; TMEM loads take the whole warp
    tc::fence_after_sync();
    return q.tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + (it & 1) * 256;
}
__device__ __forceinline__ void acc_release(uint32_t tempty_leader, int it, int lane) {
    tc::fence_before_sync();
    __syncwarp();
    if (lane == 0) ptx::mbar_remote_arrive_release(tempty_leader + 8u * (it & 1));
}

// ---------------------------------------------------------- outputs
// A warp's 32 rows x 64 consecutive columns of a 16-bit output come as two
// segments of 32 columns, one row per lane.  Where the output's rows are 16-byte
// aligned both are put into the warp's buffer (128-byte swizzle) and one TMA store
// takes it to memory as whole 128-byte lines, leaving out what is not there; else
// (`vec` = 2) a segment passes through the buffer on its own, so that a warp's
// 2-byte accesses cover consecutive addresses of a row.
//
// A TMA store cuts a row off at 16 bytes, not at the element: measured, it writes the
// whole last granule.  So the maps end with the last whole granule, and the up to 7
// columns after it are stored one by one.
struct Out {
    uint16_t *base;
    int64_t ld;
    int vec;                 // bytes an access may use: >= 16, or 2
    const CUtensorMap *map;  // boxes of 64 columns x 32 rows, of whole granules
};

// The warp's buffer may be written: its TMA stores have read it.  (A second buffer,
// for a ring of five chunks, measured the same.)
__device__ __forceinline__ void buffer_free(int lane) {
    if (lane == 0) tc::bulk_wait_read();
    __syncwarp();
}
// Segment h (0 or 1) of the 64 columns from `col`.
__device__ __forceinline__ void put_seg(const Out &o, int64_t row0, int col, int h,
                                        const float (&v)[32], int64_t rows, int cols, bool f16,
                                        uint32_t *buf, int lane) {
    uint32_t u[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) u[j] = act::pack16x2(v[2 * j], v[2 * j + 1], f16);
    if (o.vec >= 16) {
        if (h == 0) buffer_free(lane);
        unsigned char *row = reinterpret_cast<unsigned char *>(buf) + lane * 128;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4 *>(row + (((4 * h + j) ^ (lane & 7)) << 4)) =
                make_uint4(u[4 * j], u[4 * j + 1], u[4 * j + 2], u[4 * j + 3]);
        if (h == 1) {
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && cols - col >= 8) {
                tc::tma_store_2d(o.map, ptx::smem_addr(buf), col, static_cast<int>(row0));
                tc::bulk_commit();
            }
        }
        return;
    }
    buffer_free(lane);
#pragma unroll
    for (int j = 0; j < 16; ++j) buf[lane * 17 + j] = u[j];
    __syncwarp();
    const int nr = static_cast<int>(min(int64_t{32}, rows - row0));
    const uint16_t *s16 = reinterpret_cast<const uint16_t *>(buf);
    uint16_t *p = o.base + row0 * o.ld + col + 32 * h + lane;
    if (col + 32 * h + lane < cols) {
#pragma unroll 8
        for (int r = 0; r < nr; ++r) p[r * o.ld] = s16[r * 34 + lane];
    }
}
// The up to 7 columns after a row's last whole granule, from the warp's buffer, which
// still holds the 64 columns from `col`.
__device__ __forceinline__ void put_rest(const Out &o, int64_t row0, int col, int64_t rows,
                                         int cols, const uint32_t *buf, int lane) {
    const int left = cols - col;
    if (o.vec < 16 || left >= 64 || row0 + lane >= rows) return;
    const uint16_t *at = reinterpret_cast<const uint16_t *>(
        reinterpret_cast<const unsigned char *>(buf) + lane * 128 +
        (((left >> 3) ^ (lane & 7)) << 4));
    uint16_t *p = o.base + (row0 + lane) * o.ld + (cols & ~7);
#pragma unroll 1
    for (int j = 0; j < (left & 7); ++j) p[j] = at[j];
}
// 64 columns from `col` of row `row` of a 16-bit tensor, one row per lane, on their
// way in registers: the 16-byte granules of the memory that hold them, at any
// alignment.  Fetched a group of columns ahead: behind the ring's copies an answer
// takes thousands of clocks.
struct RowFetch {
    uint4 q[9];
    const uint16_t *at;
    bool whole;  // every granule lies inside the tensor; else take the elements one by one
};
__device__ __forceinline__ void fetch_row(const uint16_t *base, int64_t ld, int64_t row, int col,
                                          int64_t rows, int cols, RowFetch &f) {
    f.at = base + row * ld + col;
    const uintptr_t a = reinterpret_cast<uintptr_t>(f.at);
    const uintptr_t first = a & ~uintptr_t{15}, last = a + 2 * min(64, cols - col);
    f.whole = row < rows && col < cols && first >= reinterpret_cast<uintptr_t>(base) &&
              ((last + 15) & ~uintptr_t{15}) <=
                  reinterpret_cast<uintptr_t>(base + (rows - 1) * ld + cols);
    if (f.whole) {
#pragma unroll
        for (int i = 0; i < 9; ++i)
            if (first + 16 * i < last) f.q[i] = *reinterpret_cast<const uint4 *>(first + 16 * i);
    }
}
// The columns' 32 words, moved to the front.
__device__ __forceinline__ void align_row(const RowFetch &f, uint32_t (&u)[32]) {
    const uint32_t s = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(f.at));
    uint32_t w[36];
#pragma unroll
    for (int i = 0; i < 9; ++i) {
        w[4 * i] = f.q[i].x;
        w[4 * i + 1] = f.q[i].y;
        w[4 * i + 2] = f.q[i].z;
        w[4 * i + 3] = f.q[i].w;
    }
#pragma unroll
    for (int i = 0; i < 34; ++i) w[i] = s & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 33; ++i) w[i] = s & 4 ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < 32; ++i) u[i] = __funnelshift_r(w[i], w[i + 1], (s & 2) * 8);
}
// 32 fp32 columns from `col` (boxes of 32 columns x 32 rows): stored, or added.
__device__ __forceinline__ void put_f32(const CUtensorMap *map, int64_t row0, int col,
                                        const uint32_t (&r)[32], bool add, uint32_t *buf,
                                        int lane) {
    buffer_free(lane);
    unsigned char *row = reinterpret_cast<unsigned char *>(buf) + lane * 128;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        *reinterpret_cast<uint4 *>(row + ((j ^ (lane & 7)) << 4)) =
            make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
        if (add)
            tc::tma_add_2d(map, ptx::smem_addr(buf), col, static_cast<int>(row0));
        else
            tc::tma_store_2d(map, ptx::smem_addr(buf), col, static_cast<int>(row0));
        tc::bulk_commit();
    }
}

}  // namespace mm
}  // namespace vlmce
