// moe.cu -- tokens to their experts and back: the order of the (token, slot) pairs by
// expert, the tokens' rows in that order (as they are, or in e4m3 by blocks of 128), the
// experts' rows brought back with weights, and the gradients of both.
//
//   sort      position[t, j] = offsets[e] + rank of (t, j) among the pairs of e = experts[t, j]
//             offsets[e + 1] = offsets[e] + count[e] rounded up to `align`
//   gather    rows[position[t, j]] = x[t]
//   combine   y[t] = sum_j w[t, j] rows[position[t, j]] + residual[t]   (j in order)
//   gradient  drows[position[t, j]] = w[t, j] dy[t],  dw[t, j] = <dy[t], rows[position[t, j]]>
//
// Everything but the sort goes token by token: a token's row is read (and quantised)
// once, however many experts it has, and no inverse of `position` is needed.  Those
// kernels are bound by memory; what keeps loads in flight is a token's k rows, which a
// thread asks for together.  8192 tokens, k = 4, H = 4096 bf16: gather to e4m3 31.8 us (206
// MB, 6.5 TB/s), the gradient of combine 90.3 us (604 MB, 6.7 TB/s).  Few tokens are bound by
// the launch and two trips to memory one after the other (a position, then its row): combine
// of 16 tokens, k = 8, H = 4096 2.3 us, sort of 64 x 8 pairs 3.8 us.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <initializer_list>
#include <mutex>
#include <type_traits>

#include "blocks.cuh"
#include "host_util.h"
#include "ptx.cuh"
#include "rows_host.h"
#include "vlmce.h"

namespace vlmce {
namespace moe {
namespace {

// ------------------------------------------------------------------- sort
// One launch of one cluster.  The pairs are dealt to its warps in consecutive runs, which a
// warp walks 32 pairs at a time: pairs of one expert find one another (each sets its lane's
// bit in the expert's word of shared memory) and take their rank from the warp's count of
// that expert.  The counts are summed over the warps of a CTA and then over the CTAs
// (through distributed shared memory), and every CTA scans the experts' totals; then a
// pair's row is its rank in the warp's run and where the run's pairs of the expert start.
// So the order is that of the pairs, whatever the timing: the only atomics set bits.  A run
// of up to kSortKeep groups of 32 stays in registers; a longer one is walked twice, its pairs
// found by match, which needs no second table (a match of 32 different experts takes 260
// clocks: 131072 pairs of 256 experts 21 us by it, 10 by bits; 160000 pairs, walked twice, 46 us,
// 1048576 262).
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxExperts = VLMCE_MOE_MAX_EXPERTS;
static_assert(kMaxExperts <= kSortThreads, "a thread scans an expert");
constexpr int kMaxSortCtas = 8;
constexpr int kSortKeep = 16;
// The pairs are numbered in 32 bits, also where a warp's last step begins before the last
// pair and ends 32 kSortKeep after it: a step begins at a multiple of 32 below kMaxPairs.
constexpr int64_t kMaxPairs = (int64_t(1) << 31) - 32 * kSortKeep;
static_assert(kMaxPairs % 32 == 0 && kMaxPairs - 32 + 32 * kSortKeep <= INT32_MAX, "a step's end is a number");

struct SortParams {
    const void *experts;
    int64_t ld;
    int pairs, k, E, align, wide, ctas;
    int *position, *offsets, *counts;
};

__device__ __forceinline__ int sort_load(const SortParams &p, int i) {
    int64_t at = i;
    if (p.ld != p.k) {
        const int t = i / p.k;
        at = t * p.ld + (i - t * p.k);
    }
    if (p.wide) {
        const int64_t e = static_cast<const int64_t *>(p.experts)[at];
        return e >= 0 && e < p.E ? static_cast<int>(e) : -1;
    }
    const int e = static_cast<const int *>(p.experts)[at];
    return e >= 0 && e < p.E ? e : -1;
}

__global__ void __launch_bounds__(kSortThreads, 1) sort_kernel(const SortParams p) {
    extern __shared__ int cursor[];          // [kSortWarps][E]: a warp's counts, then where its rows start
    __shared__ int total[kMaxExperts];       // of this CTA
    __shared__ int warp_sum[kSortWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = p.ctas > 1 ? static_cast<int>(ptx::cluster_ctarank()) : 0;
    // whole groups of 32 pairs to a warp
    const int groups = (p.pairs + 31) / 32, warps = p.ctas * kSortWarps;
    const int per = (groups + warps - 1) / warps;
    const int first = min(groups, (rank * kSortWarps + warp) * per) * 32;
    const int last = min(p.pairs, min(groups, (rank * kSortWarps + warp + 1) * per) * 32);
    int *mine = cursor + warp * p.E;

    uint16_t *few = reinterpret_cast<uint16_t *>(cursor + kSortWarps * p.E) + warp * p.E;  // of a kept run
    for (int e = lane; e < p.E; e += 32) {
        mine[e] = 0;
        few[e] = 0;
    }
    __syncwarp();
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    // a pair: its expert and its rank among the run's pairs of that; -1: nobody's
    const bool kept = last - first <= 32 * kSortKeep;
    int kept_e[kSortKeep], kept_rank[kSortKeep];
    auto walk = [&](int from, auto &&rank_group) {
#pragma unroll
        for (int j = 0; j < kSortKeep; ++j) {
            const int i = from + 32 * j + lane;
            kept_e[j] = i < last ? sort_load(p, i) : -1;
        }
#pragma unroll
        for (int j = 0; j < kSortKeep; ++j) {
            if (from + 32 * j >= last) break;
            kept_rank[j] = rank_group(kept_e[j]);
        }
    };
    auto by_match = [&](int e) {  // counts in `mine`
        const unsigned peers = __match_any_sync(0xffffffffu, e);
        const int ahead = __popc(peers & ((1u << lane) - 1));
        const int r = e >= 0 ? mine[e] + ahead : 0;
        __syncwarp();
        if (e >= 0 && ahead == 0) mine[e] = r + __popc(peers);
        __syncwarp();
        return r;
    };
    auto by_bits = [&](int e) {  // bits in `mine`, counts in `few`
        if (e >= 0) atomicOr(mine + e, 1 << lane);
        __syncwarp();
        const unsigned peers = e >= 0 ? static_cast<unsigned>(mine[e]) : 0;
        const int ahead = __popc(peers & ((1u << lane) - 1));
        const int r = e >= 0 ? few[e] + ahead : 0;
        __syncwarp();
        if (e >= 0 && ahead == 0) {
            few[e] = static_cast<uint16_t>(r + __popc(peers));
            mine[e] = 0;
        }
        __syncwarp();
        return r;
    };
    if (kept) {
        walk(first, by_bits);
        __syncwarp();
        for (int e = lane; e < p.E; e += 32) mine[e] = few[e];
    } else {
        for (int g = first; g < last; g += 32 * kSortKeep) walk(g, by_match);
    }
    __syncthreads();
    // where each warp's pairs of an expert start among the CTA's
    int count = 0;  // of expert `tid`: this CTA's, then the sum over all
    if (tid < p.E) {
#pragma unroll 8
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = cursor[w * p.E + tid];
            cursor[w * p.E + tid] = count;
            count += c;
        }
        total[tid] = count;
    }
    int before = 0;  // pairs of the expert in the CTAs before this one
    if (p.ctas > 1) {
        ptx::cluster_sync();
        if (tid < p.E) {
            count = 0;
            for (int c = 0; c < p.ctas; ++c) {
                int v;
                asm volatile("ld.shared::cluster.u32 %0, [%1];"
                             : "=r"(v)
                             : "r"(ptx::mapa(ptx::smem_addr(total + tid), c))
                             : "memory");
                if (c < rank) before += v;
                count += v;
            }
        }
    }
    // exclusive sums of the rounded counts over the experts
    const int padded = (count + p.align - 1) / p.align * p.align;
    int sum = padded;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int v = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += v;
    }
    if (lane == 31) warp_sum[warp] = sum;
    __syncthreads();
    if (warp == 0) {
        int s = warp_sum[lane];
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int v = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += v;
        }
        warp_sum[lane] = s;
    }
    __syncthreads();
    const int start = (warp > 0 ? warp_sum[warp - 1] : 0) + sum - padded;
    if (tid < p.E) {
        for (int w = 0; w < kSortWarps; ++w) cursor[w * p.E + tid] += start + before;
        if (rank == 0) {
            p.offsets[tid] = start;
            p.counts[tid] = count;
            if (tid == p.E - 1) p.offsets[p.E] = start + padded;
        }
    }
    __syncthreads();
    for (int g = first; g < last; g += 32 * kSortKeep) {
        if (!kept) walk(g, by_match);  // (the counts now start where the rows do)
#pragma unroll
        for (int j = 0; j < kSortKeep; ++j) {
            const int i = g + 32 * j + lane, e = kept_e[j];
            if (i < last) p.position[i] = e >= 0 ? kept_rank[j] + (kept ? mine[e] : 0) : -1;
        }
    }
    if (p.ctas > 1) ptx::cluster_sync();  // a CTA's totals are read until here
}

// ------------------------------------------------- rows of a token's experts
struct RowParams {
    const unsigned char *x;        // [T]: tokens' rows (gather), dy (combine's gradient)
    const unsigned char *rows_in;  // [R]: experts' rows (combine and its gradient)
    unsigned char *out;            // [R]: gather, drows; [T]: combine
    const unsigned char *residual;
    float *scale;                  // [R, ceil(H / 128)]: gather in e4m3
    float *dw;                     // [T, k]
    const int *position, *offsets, *counts;
    const void *w;
    int64_t x_ld, in_ld, out_ld, res_ld, w_ld;  // bytes; w_ld, scale_ld: elements
    int64_t scale_ld, T, R, H, row_bytes;  // row_bytes: of out
    int k, E, w_f32;
    uintptr_t first, last;         // x's memory
};

// Blocks of `x` index T .. T + E - 1 clear the rows between an expert's last and the next
// one's first (there are some where the counts were rounded up), so that a product over
// them adds nothing.
__device__ __forceinline__ void clear_rows(const RowParams &p, int e, int64_t row_bytes, float scale) {
    const int64_t a = max(int64_t{0}, static_cast<int64_t>(p.offsets[e]) + p.counts[e]);
    const int64_t b = min(p.R, static_cast<int64_t>(p.offsets[e + 1]));
    const int nthreads = blockDim.x * gridDim.y, tid = blockIdx.y * blockDim.x + threadIdx.x;
    for (int64_t r = a; r < b; ++r) {
        unsigned char *row = p.out + r * p.out_ld;
        // (up to 15 bytes before the first 16-byte unit and after the last one by themselves)
        const int64_t head = min(row_bytes, static_cast<int64_t>(
                                                (16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15));
        const int64_t units = (row_bytes - head) / 16;
        if (tid < head) row[tid] = 0;
        for (int64_t i = tid; i < units; i += nthreads)
            reinterpret_cast<uint4 *>(row + head)[i] = make_uint4(0, 0, 0, 0);
        const int64_t done = head + 16 * units;
        if (tid < row_bytes - done) row[done + tid] = 0;
        if (p.scale)
            for (int64_t i = tid; i < p.scale_ld; i += nthreads) p.scale[r * p.scale_ld + i] = scale;
    }
}

// Rows as they are, in units of U bytes; kCopyUnits<U> a thread, 32 apart (twice as many: 512
// rows of 4096 bf16 5.3 us instead of 4.4, 8192 rows 51.1 and 50.2).
template <int U>
constexpr int kCopyUnits = U == 16 ? 2 : 4;
template <int U>
__global__ void __launch_bounds__(256) gather_copy_kernel(const RowParams p) {
    using Unit = std::conditional_t<U == 16, uint4, std::conditional_t<U == 4, uint32_t, uint16_t>>;
    constexpr int N = kCopyUnits<U>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int64_t t = blockIdx.x;
    if (t >= p.T) {
        clear_rows(p, static_cast<int>(t - p.T), p.row_bytes, 0.f);
        return;
    }
    const int first = (static_cast<int>(blockIdx.y) * (blockDim.x >> 5) + warp) * (32 * N) + lane;
    const int left = static_cast<int>(p.row_bytes / U) - first;  // units of the row from there
    if (left <= 0) return;
    const int *pos = p.position + t * p.k;
    const Unit *from = reinterpret_cast<const Unit *>(p.x + t * p.x_ld) + first;
    Unit v[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (32 * i < left) v[i] = from[32 * i];
    for (int j = 0; j < p.k; ++j) {
        const int r = pos[j];
        if (r < 0 || r >= p.R) continue;
        Unit *to = reinterpret_cast<Unit *>(p.out + r * p.out_ld) + first;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (32 * i < left) to[32 * i] = v[i];
    }
}

// In e4m3 with 16 columns a thread, to rows of whole 16-byte units: bound by instructions
// with eight (8192 tokens to 4 rows of 4096 each 40 us, 77 % of the issue slots), of which the
// two divisions of a block and a row's address are a thread's, however many columns it has.
// ALIGNED: x's rows are whole units, too, and 16 divides H.  Else the units that hold a
// thread's columns are moved into place (8192 tokens to 4 rows of 4097 42.6 us, by elements 83).
template <int DT, bool ALIGNED>
__global__ void __launch_bounds__(256) gather_wide_kernel(const RowParams p) {
    constexpr bool k16 = DT != VLMCE_F32;
    constexpr int kWords = k16 ? 8 : 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int64_t t = blockIdx.x;
    if (t >= p.T) {
        float inv;
        const float zero = blocks::scale_of(0, inv);
        clear_rows(p, static_cast<int>(t - p.T), p.row_bytes, zero);
        return;
    }
    const int64_t c = (static_cast<int64_t>(blockIdx.y) * (blockDim.x >> 5) + warp) * 512 + 16 * lane;
    const int n = static_cast<int>(min(int64_t{16}, p.H - c));  // columns of the 16 there are
    const int *pos = p.position + t * p.k;
    const unsigned char *from = p.x + t * p.x_ld + c * blocks::elt_bytes<DT>;
    uint32_t u[kWords + 4];
    if constexpr (ALIGNED) {
#pragma unroll
        for (int i = 0; i < kWords; i += 4) {
            const uint4 q = n > 0 ? *reinterpret_cast<const uint4 *>(from + 4 * i) : make_uint4(0, 0, 0, 0);
            u[i] = q.x, u[i + 1] = q.y, u[i + 2] = q.z, u[i + 3] = q.w;
        }
    } else {
        const uintptr_t unit = reinterpret_cast<uintptr_t>(from) & ~uintptr_t{15};
        if (n == 16 && unit >= p.first && unit + 4 * kWords + 16 <= p.last) {
#pragma unroll
            for (int i = 0; i < kWords + 4; i += 4) {
                const uint4 q = *reinterpret_cast<const uint4 *>(unit + 4 * i);
                u[i] = q.x, u[i + 1] = q.y, u[i + 2] = q.z, u[i + 3] = q.w;
            }
            blocks::move_into_place<kWords, k16>(u, static_cast<uint32_t>(reinterpret_cast<uintptr_t>(from) & 15));
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if constexpr (k16) {
                    const uint32_t e = i < n ? reinterpret_cast<const uint16_t *>(from)[i] : 0;
                    u[i / 2] = i & 1 ? u[i / 2] | e << 16 : e;
                } else {
                    u[i] = i < n ? reinterpret_cast<const uint32_t *>(from)[i] : 0;
                }
            }
        }
    }
    uint32_t a = 0;  // magnitudes, 16-bit ones two at a time
#pragma unroll
    for (int i = 0; i < kWords; ++i)
        a = k16 ? __vmaxu2(a, u[i] & 0x7fff7fffu) : max(a, u[i] & 0x7fffffffu);
    if constexpr (k16)
        a = __float_as_uint(act::from16(static_cast<uint16_t>(max(a & 0xffffu, a >> 16)), DT == VLMCE_F16));
#pragma unroll
    for (int d = 4; d > 0; d /= 2) a = max(a, __shfl_xor_sync(0xffffffffu, a, d));  // a block: eight lanes
    float inv;
    const float scale = blocks::scale_of(a, inv);
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
            if constexpr (k16) {
                act::unpack16x2(u[2 * i + j / 2], v[j], v[j + 1], DT == VLMCE_F16);
            } else {
                v[j] = __uint_as_float(u[4 * i + j]);
                v[j + 1] = __uint_as_float(u[4 * i + j + 1]);
            }
        }
        q[i] = blocks::pack_e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    }
    if (n <= 0) return;
    for (int j = 0; j < p.k; ++j) {
        const int r = pos[j];
        if (r < 0 || r >= p.R) continue;
        unsigned char *to = p.out + r * p.out_ld + c;
        if (ALIGNED || n == 16) {
            *reinterpret_cast<uint4 *>(to) = make_uint4(q[0], q[1], q[2], q[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (i < n) to[i] = static_cast<unsigned char>(q[i / 4] >> (8 * (i & 3)));
        }
        if ((lane & 7) == 0) p.scale[r * p.scale_ld + c / blocks::kBlock] = scale;
    }
}

// In e4m3 to rows at any alignment: a warp a block, a lane four columns 32 apart.
template <int DT>
__global__ void __launch_bounds__(256) gather_bytes_kernel(const RowParams p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int64_t t = blockIdx.x;
    if (t >= p.T) {
        float inv;
        const float zero = blocks::scale_of(0, inv);
        clear_rows(p, static_cast<int>(t - p.T), p.row_bytes, zero);
        return;
    }
    const int64_t base = (static_cast<int64_t>(blockIdx.y) * (blockDim.x >> 5) + warp) * blocks::kBlock, c = base + lane;
    if (base >= p.H) return;
    const int *pos = p.position + t * p.k;
    const unsigned char *x = p.x + t * p.x_ld;
    float v[4];
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = c + 32 * i < p.H ? blocks::load1<DT>(x, c + 32 * i) : 0.f;
        a = max(a, blocks::magnitude(v[i]));
    }
    float inv;
    const float scale = blocks::scale_of(__reduce_max_sync(0xffffffffu, a), inv);
    const uint32_t q = blocks::pack_e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    for (int j = 0; j < p.k; ++j) {
        const int r = pos[j];
        if (r < 0 || r >= p.R) continue;
        unsigned char *row = p.out + r * p.out_ld;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + 32 * i < p.H) row[c + 32 * i] = static_cast<unsigned char>(q >> (8 * i));
        if (lane == 0) p.scale[r * p.scale_ld + base / blocks::kBlock] = scale;
    }
}

template <int DT>
__device__ __forceinline__ float weight_of(const RowParams &p, int64_t t, int j) {
    if (!p.w) return 1.f;
    const int64_t i = t * p.w_ld + j;
    if (p.w_f32) return static_cast<const float *>(p.w)[i];
    return blocks::load1<DT>(static_cast<const unsigned char *>(p.w), i);
}

// (Five CTAs per SM of up to 51 registers where a thread has four rows of 16-bit values:
// 8192 x 4 rows of 4096 68 us, as the compiler likes 72.  The gradient needs four of 64: 91
// us, with three 100.)
template <int DT, int U, int AT_ONCE>
__global__ void __launch_bounds__(256, AT_ONCE > 4 ? (DT == VLMCE_F32 || U == 2 ? 2 : 3) : DT == VLMCE_F32 || U == 2 ? 3 : 5)
    combine_kernel(const RowParams p) {
    using C = blocks::Cols<DT, U>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int64_t t = blockIdx.x;
    const int64_t base =
        (static_cast<int64_t>(blockIdx.y) * (blockDim.x >> 5) + warp) * C::kWarp;
    if (base >= p.H) return;
    const C cols(base, lane);
    const int *pos = p.position + t * p.k;
    typename C::Raw res;
    if (p.residual) cols.fetch(p.residual + t * p.res_ld, p.H, res);
    float y[C::N];
#pragma unroll
    for (int i = 0; i < C::N; ++i) y[i] = 0.f;
    for (int j0 = 0; j0 < p.k; j0 += AT_ONCE) {
        typename C::Raw v[AT_ONCE];
        float w[AT_ONCE];
        int r[AT_ONCE];
#pragma unroll
        for (int j = 0; j < AT_ONCE; ++j) {
            r[j] = j0 + j < p.k ? pos[j0 + j] : -1;
            w[j] = j0 + j < p.k ? weight_of<DT>(p, t, j0 + j) : 0.f;
            if (r[j] >= p.R) r[j] = -1;
        }
#pragma unroll
        for (int j = 0; j < AT_ONCE; ++j)
            if (r[j] >= 0) cols.fetch(p.rows_in + r[j] * p.in_ld, p.H, v[j]);
#pragma unroll
        for (int j = 0; j < AT_ONCE; ++j)
            if (r[j] >= 0) {
#pragma unroll
                for (int i = 0; i < C::N; ++i) y[i] = fmaf(w[j], C::value(v[j], i), y[i]);
            }
    }
    if (p.residual) {
#pragma unroll
        for (int i = 0; i < C::N; ++i) y[i] += C::value(res, i);
    }
    cols.store(p.out + t * p.out_ld, p.H, y);
}

// A CTA has the whole row of a token: dw's sums stay in it, in an order of their own.
template <int DT, int U, int AT_ONCE>
__global__ void __launch_bounds__(256, AT_ONCE > 4 || DT == VLMCE_F32 ? 2 : U == 2 ? 3 : 4)
    combine_bwd_kernel(const RowParams p) {
    using C = blocks::Cols<DT, U>;
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __shared__ float part[8][AT_ONCE];
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int64_t t = blockIdx.x;
    if (t >= p.T) {
        if (p.out)
            clear_rows(p, static_cast<int>(t - p.T), p.row_bytes, 0.f);
        return;
    }
    const int *pos = p.position + t * p.k;
    for (int j0 = 0; j0 < p.k; j0 += AT_ONCE) {
        int r[AT_ONCE];
        float w[AT_ONCE], sum[AT_ONCE];
#pragma unroll
        for (int j = 0; j < AT_ONCE; ++j) {
            r[j] = j0 + j < p.k ? pos[j0 + j] : -1;
            w[j] = j0 + j < p.k ? weight_of<DT>(p, t, j0 + j) : 0.f;
            if (r[j] >= p.R) r[j] = -1;
            sum[j] = 0.f;
        }
        for (int64_t base = static_cast<int64_t>(warp) * C::kWarp; base < p.H;
             base += static_cast<int64_t>(warps) * C::kWarp) {
            const C cols(base, lane);
            typename C::Raw d, v[AT_ONCE];
            cols.fetch(p.x + t * p.x_ld, p.H, d);
            if (p.dw) {
#pragma unroll
                for (int j = 0; j < AT_ONCE; ++j)
                    if (r[j] >= 0) cols.fetch(p.rows_in + r[j] * p.in_ld, p.H, v[j]);
#pragma unroll
                for (int j = 0; j < AT_ONCE; ++j)
                    if (r[j] >= 0) {
#pragma unroll
                        for (int i = 0; i < C::N; ++i)
                            sum[j] = fmaf(C::value(d, i), C::value(v[j], i), sum[j]);
                    }
            }
            if (p.out) {
#pragma unroll
                for (int j = 0; j < AT_ONCE; ++j)
                    if (r[j] >= 0) {
                        float o[C::N];
#pragma unroll
                        for (int i = 0; i < C::N; ++i) o[i] = w[j] * C::value(d, i);
                        cols.store(p.out + r[j] * p.out_ld, p.H, o);
                    }
            }
        }
        if (p.dw) {
#pragma unroll
            for (int j = 0; j < AT_ONCE; ++j) {
#pragma unroll
                for (int s = 16; s > 0; s /= 2) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], s);
                if (lane == 0) part[warp][j] = sum[j];
            }
            __syncthreads();
            if (threadIdx.x < AT_ONCE && j0 + static_cast<int>(threadIdx.x) < p.k) {
                float a = 0.f;
                for (int i = 0; i < warps; ++i) a += part[i][threadIdx.x];
                p.dw[t * p.k + j0 + threadIdx.x] = a;
            }
            __syncthreads();
        }
    }
}

// ------------------------------------------------------------------- host
using RowKernel = void (*)(const RowParams);

template <class P>
cudaError_t launch(void (*k)(const P), dim3 grid, int threads, size_t smem, unsigned ctas,
                   cudaStream_t s, const P &p) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k, p);
}

RowKernel gather_copy_of(int unit) {
    return unit == 16 ? gather_copy_kernel<16> : unit == 4 ? gather_copy_kernel<4> : gather_copy_kernel<2>;
}
template <bool ALIGNED>
RowKernel gather_wide_of(int dt) {
    switch (dt) {
        case VLMCE_F32: return gather_wide_kernel<VLMCE_F32, ALIGNED>;
        case VLMCE_F16: return gather_wide_kernel<VLMCE_F16, ALIGNED>;
        default: return gather_wide_kernel<VLMCE_BF16, ALIGNED>;
    }
}
RowKernel gather_bytes_of(int dt) {
    switch (dt) {
        case VLMCE_F32: return gather_bytes_kernel<VLMCE_F32>;
        case VLMCE_F16: return gather_bytes_kernel<VLMCE_F16>;
        default: return gather_bytes_kernel<VLMCE_BF16>;
    }
}
template <int DT, int U>
RowKernel combine_of(bool bwd, int64_t k) {
    // (unused places of eight cost registers: up to four rows of a token at a time, or eight)
    if (k <= 4) return bwd ? combine_bwd_kernel<DT, U, 4> : combine_kernel<DT, U, 4>;
    return bwd ? combine_bwd_kernel<DT, U, 8> : combine_kernel<DT, U, 8>;
}
template <int DT>
RowKernel combine_of16(int unit, bool bwd, int64_t k) {
    return unit == 16 ? combine_of<DT, 16>(bwd, k) : unit == 4 ? combine_of<DT, 4>(bwd, k) : combine_of<DT, 2>(bwd, k);
}
RowKernel combine_of(int dt, int unit, bool bwd, int64_t k) {
    switch (dt) {
        case VLMCE_F32: return unit == 16 ? combine_of<VLMCE_F32, 16>(bwd, k) : combine_of<VLMCE_F32, 4>(bwd, k);
        case VLMCE_F16: return combine_of16<VLMCE_F16>(unit, bwd, k);
        default: return combine_of16<VLMCE_BF16>(unit, bwd, k);
    }
}

constexpr int64_t kMaxH = int64_t(1) << 24;

bool dtype_ok(int32_t dt) { return dt == VLMCE_F32 || dt == VLMCE_BF16 || dt == VLMCE_F16; }
int elt_of(int32_t dt) { return dt == VLMCE_F32 ? 4 : 2; }

// T tokens of k experts of E: whether the calls that read positions take them, and sort.
vlmce_status order_ok(int64_t T, int64_t k, int64_t E) {
    if (T < 0 || k < 1 || E < 1) return VLMCE_ERR_INVALID_ARG;
    if (k > VLMCE_MOE_MAX_TOPK || E > kMaxExperts || T > INT32_MAX / k) return VLMCE_ERR_TOO_LARGE;
    return VLMCE_OK;
}
vlmce_status sort_ok(int64_t T, int64_t k, int64_t E) {
    const vlmce_status st = order_ok(T, k, E);
    return st == VLMCE_OK && T * k > kMaxPairs ? VLMCE_ERR_TOO_LARGE : st;
}
int64_t capacity(int64_t T, int64_t k, int64_t E, int64_t align) {
    return (T * k + std::min(E, T * k) * (align - 1)) / align * align;
}

// A matrix argument: rows of `bytes` bytes.
struct Mat {
    const void *p;
    int64_t rows, cols, ld;
    int elt;
    bool in_units(int u) const {
        return aligned(p, static_cast<uintptr_t>(u)) && ld * elt % u == 0 && cols * elt % u == 0;
    }
};
vlmce_status check(const Mat &m) {
    if (m.ld < m.cols || (m.rows > 0 && !m.p)) return VLMCE_ERR_INVALID_ARG;
    if (m.ld > (int64_t(1) << 60) / m.elt / std::max<int64_t>(m.rows, 1)) return VLMCE_ERR_TOO_LARGE;
    if (!aligned(m.p, static_cast<uintptr_t>(m.elt))) return VLMCE_ERR_MISALIGNED;
    return VLMCE_OK;
}
bool overlap(const Mat &a, const Mat &b) {
    return rows_overlap({a.p, a.rows, a.cols * a.elt, a.ld * a.elt},
                        {b.p, b.rows, b.cols * b.elt, b.ld * b.elt});
}

// The largest accesses that all of them take (an absent one takes any).  8192 tokens, k = 4,
// bf16, H 4096 in 16 bytes, 4100 in 4 and 4097 in 2: gather 50, 60 and 70 us, combine 68, 76
// and 112, its gradient 91, 97 and 132 (all in single elements, four a thread: 73, 130, 135).
int unit_of(std::initializer_list<const Mat *> mats, int elt) {
    for (const int u : {16, 4})
        if (std::all_of(mats.begin(), mats.end(), [u](const Mat *m) { return !m->p || m->in_units(u); })) return u;
    return elt;
}

// Threads of a CTA and CTAs of a row: warps of `per` columns, eight of them at most.
int threads_of(int64_t H, int per) {
    return static_cast<int>(32 * std::min<int64_t>(8, (H + per - 1) / per));
}
unsigned row_ctas(int64_t H, int per, int threads) {
    const int64_t cols = static_cast<int64_t>(threads / 32) * per;
    return static_cast<unsigned>((H + cols - 1) / cols);
}

vlmce_status common(int64_t T, int64_t R, int64_t H, int64_t k, int64_t E, const int32_t *position,
                    const int32_t *offsets, const int32_t *counts) {
    const vlmce_status st = order_ok(T, k, E);
    if (st != VLMCE_OK) return st;
    if (R < 0 || H < 1 || (T > 0 && !position) || !offsets || !counts) return VLMCE_ERR_INVALID_ARG;
    if (R > INT32_MAX || H > kMaxH || T + E > INT32_MAX) return VLMCE_ERR_TOO_LARGE;
    if (!aligned(position, 4) || !aligned(offsets, 4) || !aligned(counts, 4))
        return VLMCE_ERR_MISALIGNED;
    return VLMCE_OK;
}

}  // namespace
}  // namespace moe
}  // namespace vlmce

extern "C" int64_t vlmce_moe_rows(int64_t T, int64_t k, int64_t E, int64_t align) {
    using namespace vlmce::moe;
    if (sort_ok(T, k, E) != VLMCE_OK || align < 1 || align > INT32_MAX) return -1;
    const int64_t used = std::min(E, T * k);
    if (used > 0 && align > (INT32_MAX - T * k) / used) return -1;
    return capacity(T, k, E, align);
}

extern "C" vlmce_status moe_sort(const void *experts, int64_t experts_stride, int32_t wide,
                                 int64_t T, int64_t k, int64_t E, int64_t align, int32_t *position,
                                 int32_t *offsets, int32_t *counts, vlmce_stream_t stream) {
    using namespace vlmce;
    using namespace vlmce::moe;
    vlmce_status st = sort_ok(T, k, E);
    if (st != VLMCE_OK) return st;
    if (align < 1 || experts_stride < k || !offsets || !counts || (T > 0 && (!experts || !position)))
        return VLMCE_ERR_INVALID_ARG;
    if (vlmce_moe_rows(T, k, E, align) < 0 || experts_stride > (int64_t(1) << 56) / std::max<int64_t>(T, 1))
        return VLMCE_ERR_TOO_LARGE;
    if (!aligned(experts, wide ? 8 : 4) || !aligned(position, 4) || !aligned(offsets, 4) ||
        !aligned(counts, 4))
        return VLMCE_ERR_MISALIGNED;
    const Mat in{experts, T, k, experts_stride, wide ? 8 : 4}, pos{position, T, k, k, 4},
        off{offsets, 1, E + 1, E + 1, 4}, cnt{counts, 1, E, E, 4};
    if (overlap(pos, in) || overlap(off, in) || overlap(cnt, in) || overlap(pos, off) ||
        overlap(pos, cnt) || overlap(off, cnt))
        return VLMCE_ERR_INVALID_ARG;
    DeviceInfo dev;
    st = current_device(&dev);
    if (st != VLMCE_OK) return st;
    static std::mutex mu;
    static bool opted[64] = {};
    cudaError_t e = cudaSuccess;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!opted[dev.device]) {
            e = cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kSortWarps * kMaxExperts * 6);
            opted[dev.device] = e == cudaSuccess;
        }
    }
    if (e != cudaSuccess) return launch_status(e, "moe_sort");
    SortParams p = {};
    p.experts = experts;
    p.ld = experts_stride;
    p.pairs = static_cast<int>(T * k);
    p.k = static_cast<int>(k);
    p.E = static_cast<int>(E);
    p.align = static_cast<int>(align);
    p.wide = wide != 0;
    p.position = position;
    p.offsets = offsets;
    p.counts = counts;
    p.ctas = 1;
    while (p.ctas < kMaxSortCtas && p.pairs > p.ctas * kSortThreads) p.ctas *= 2;
    e = launch(sort_kernel, dim3(static_cast<unsigned>(p.ctas), 1, 1), kSortThreads,
               static_cast<size_t>(kSortWarps * E * 6), static_cast<unsigned>(p.ctas),
               reinterpret_cast<cudaStream_t>(stream), p);
    return launch_status(e, "moe_sort");
}

extern "C" vlmce_status moe_gather(const void *x, int64_t x_stride, int32_t dtype,
                                   const int32_t *position, const int32_t *offsets,
                                   const int32_t *counts, int64_t T, int64_t k, int64_t E,
                                   int64_t R, int64_t H, void *rows, int64_t rows_stride,
                                   int32_t rows_dtype, float *scale, vlmce_stream_t stream) {
    using namespace vlmce;
    using namespace vlmce::moe;
    if (!dtype_ok(dtype) || (rows_dtype != dtype && rows_dtype != VLMCE_E4M3))
        return VLMCE_ERR_UNSUPPORTED_DTYPE;
    const bool fp8 = rows_dtype == VLMCE_E4M3;
    vlmce_status st = common(T, R, H, k, E, position, offsets, counts);
    if (st != VLMCE_OK) return st;
    const int64_t nb = (H + blocks::kBlock - 1) / blocks::kBlock;
    const Mat in{x, T, H, x_stride, elt_of(dtype)}, out{rows, R, H, rows_stride, fp8 ? 1 : elt_of(dtype)},
        sc{scale, fp8 ? R : 0, nb, nb, 4}, pos{position, T, k, k, 4}, off{offsets, 1, E + 1, E + 1, 4},
        cnt{counts, 1, E, E, 4};
    if (!fp8 && scale) return VLMCE_ERR_INVALID_ARG;
    st = check(in);
    if (st == VLMCE_OK) st = check(out);
    if (st == VLMCE_OK) st = check(sc);
    if (st != VLMCE_OK) return st;
    if (overlap(out, in) || overlap(sc, in) || overlap(out, sc) || overlap(out, pos) || overlap(sc, pos) ||
        overlap(out, off) || overlap(sc, off) || overlap(out, cnt) || overlap(sc, cnt))
        return VLMCE_ERR_INVALID_ARG;
    if (R == 0) return VLMCE_OK;
    DeviceInfo dev;
    st = current_device(&dev);
    if (st != VLMCE_OK) return st;
    RowParams p = {};
    p.x = static_cast<const unsigned char *>(x);
    p.x_ld = x_stride * in.elt;
    p.out = static_cast<unsigned char *>(rows);
    p.out_ld = rows_stride * out.elt;
    p.row_bytes = H * out.elt;
    p.first = reinterpret_cast<uintptr_t>(x);
    p.last = p.first + (T > 0 ? static_cast<uintptr_t>(((T - 1) * x_stride + H) * in.elt) : 0);
    p.scale = scale;
    p.scale_ld = nb;
    p.position = position;
    p.offsets = offsets;
    p.counts = counts;
    p.T = T;
    p.R = R;
    p.H = H;
    p.k = static_cast<int>(k);
    p.E = static_cast<int>(E);
    const int unit = unit_of({&in, &out}, in.elt);
    const bool wide = aligned(rows, 16) && rows_stride % 16 == 0;  // e4m3
    const RowKernel kern = !fp8   ? gather_copy_of(unit)
                           : wide ? (H % 16 == 0 && in.in_units(16) ? gather_wide_of<true>(dtype) : gather_wide_of<false>(dtype))
                                  : gather_bytes_of(dtype);
    const int per = !fp8 ? 32 * unit / in.elt * (unit == 16 ? kCopyUnits<16> : kCopyUnits<4>) : wide ? 512 : blocks::kBlock;
    const int threads = threads_of(H, per);
    return launch_status(launch(kern, dim3(static_cast<unsigned>(T + E), row_ctas(H, per, threads), 1),
                                threads, 0, 1, reinterpret_cast<cudaStream_t>(stream), p),
                         "moe_gather");
}

extern "C" vlmce_status moe_combine(const void *rows, int64_t rows_stride, int32_t dtype,
                                    const int32_t *position, const void *weights,
                                    int64_t weights_stride, int32_t weights_dtype,
                                    const void *residual, int64_t residual_stride, int64_t T,
                                    int64_t k, int64_t R, int64_t H, void *y, int64_t y_stride,
                                    vlmce_stream_t stream) {
    using namespace vlmce;
    using namespace vlmce::moe;
    if (!dtype_ok(dtype) || (weights && weights_dtype != VLMCE_F32 && weights_dtype != dtype))
        return VLMCE_ERR_UNSUPPORTED_DTYPE;
    const int32_t none = 0;
    vlmce_status st = common(T, R, H, k, 1, position, &none, &none);
    if (st != VLMCE_OK) return st;
    const int elt = elt_of(dtype), welt = elt_of(weights_dtype);
    const Mat in{rows, R, H, rows_stride, elt}, out{y, T, H, y_stride, elt},
        res{residual, residual ? T : 0, H, residual_stride, elt}, pos{position, T, k, k, 4},
        w{weights, weights ? T : 0, k, weights_stride, welt};
    st = check(in);
    if (st == VLMCE_OK) st = check(out);
    if (st == VLMCE_OK && residual) st = check(res);
    if (st == VLMCE_OK && weights) st = check(w);
    if (st != VLMCE_OK) return st;
    if (overlap(out, in) || overlap(out, w) || overlap(out, pos) ||
        (overlap(out, res) && !(y == residual && (y_stride == residual_stride || T <= 1))))
        return VLMCE_ERR_INVALID_ARG;
    if (T == 0) return VLMCE_OK;
    DeviceInfo dev;
    st = current_device(&dev);
    if (st != VLMCE_OK) return st;
    const int unit = unit_of({&in, &out, &res}, elt);
    RowParams p = {};
    p.rows_in = static_cast<const unsigned char *>(rows);
    p.in_ld = rows_stride * elt;
    p.out = static_cast<unsigned char *>(y);
    p.out_ld = y_stride * elt;
    p.residual = static_cast<const unsigned char *>(residual);
    p.res_ld = residual_stride * elt;
    p.position = position;
    p.w = weights;
    p.w_ld = weights_stride;
    p.w_f32 = weights_dtype == VLMCE_F32;
    p.T = T;
    p.R = R;
    p.H = H;
    p.k = static_cast<int>(k);
    constexpr int per = blocks::Cols<VLMCE_F32, 16>::kWarp;
    const int threads = threads_of(H, per);
    return launch_status(
        launch(combine_of(dtype, unit, false, k),
               dim3(static_cast<unsigned>(T), row_ctas(H, per, threads), 1), threads, 0, 1,
               reinterpret_cast<cudaStream_t>(stream), p),
        "moe_combine");
}

extern "C" vlmce_status moe_combine_bwd(const void *dy, int64_t dy_stride, const void *rows,
                                        int64_t rows_stride, int32_t dtype, const int32_t *position,
                                        const int32_t *offsets, const int32_t *counts,
                                        const void *weights, int64_t weights_stride,
                                        int32_t weights_dtype, int64_t T, int64_t k, int64_t E,
                                        int64_t R, int64_t H, void *drows, int64_t drows_stride,
                                        float *dweights, vlmce_stream_t stream) {
    using namespace vlmce;
    using namespace vlmce::moe;
    if (!dtype_ok(dtype) || (weights && weights_dtype != VLMCE_F32 && weights_dtype != dtype))
        return VLMCE_ERR_UNSUPPORTED_DTYPE;
    vlmce_status st = common(T, R, H, k, E, position, offsets, counts);
    if (st != VLMCE_OK) return st;
    if (!drows && !dweights && T > 0) return VLMCE_ERR_INVALID_ARG;
    const int elt = elt_of(dtype), welt = elt_of(weights_dtype);
    const Mat d{dy, T, H, dy_stride, elt}, in{rows, dweights ? R : 0, H, rows_stride, elt},
        out{drows, drows ? R : 0, H, drows_stride, elt}, w{weights, weights ? T : 0, k, weights_stride, welt},
        dw{dweights, dweights ? T : 0, k, k, 4}, pos{position, T, k, k, 4}, off{offsets, 1, E + 1, E + 1, 4},
        cnt{counts, 1, E, E, 4};
    st = check(d);
    if (st == VLMCE_OK && dweights) st = check(in);
    if (st == VLMCE_OK && drows) st = check(out);
    if (st == VLMCE_OK && weights) st = check(w);
    if (st == VLMCE_OK && dweights) st = check(dw);
    if (st != VLMCE_OK) return st;
    if (overlap(out, d) || overlap(out, in) || overlap(out, w) || overlap(out, dw) || overlap(out, pos) ||
        overlap(dw, d) || overlap(dw, in) || overlap(dw, w) || overlap(dw, pos) || overlap(out, off) ||
        overlap(out, cnt) || overlap(dw, off) || overlap(dw, cnt))
        return VLMCE_ERR_INVALID_ARG;
    if (T == 0 && out.rows == 0) return VLMCE_OK;
    DeviceInfo dev;
    st = current_device(&dev);
    if (st != VLMCE_OK) return st;
    // (rows that are not read do not count)
    const int unit = dweights ? unit_of({&d, &in, &out}, elt) : unit_of({&d, &out}, elt);
    RowParams p = {};
    p.x = static_cast<const unsigned char *>(dy);
    p.x_ld = dy_stride * elt;
    p.rows_in = static_cast<const unsigned char *>(rows);
    p.in_ld = rows_stride * elt;
    p.out = static_cast<unsigned char *>(drows);
    p.out_ld = drows_stride * elt;
    p.row_bytes = H * elt;
    p.dw = dweights;
    p.position = position;
    p.offsets = offsets;
    p.counts = counts;
    p.w = weights;
    p.w_ld = weights_stride;
    p.w_f32 = weights_dtype == VLMCE_F32;
    p.T = T;
    p.R = R;
    p.H = H;
    p.k = static_cast<int>(k);
    p.E = static_cast<int>(E);
    constexpr int per = blocks::Cols<VLMCE_F32, 16>::kWarp;
    return launch_status(launch(combine_of(dtype, unit, true, k),
                                dim3(static_cast<unsigned>(T + E), 1, 1), threads_of(H, per), 0, 1,
                                reinterpret_cast<cudaStream_t>(stream), p),
                         "moe_combine_bwd");
}
