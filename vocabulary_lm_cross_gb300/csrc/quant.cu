// quant.cu -- e4m3 with one scale per block of 128 (blocks.cuh): of a row's 128
// columns, of a column's 128 rows (the result transposed), or of 128 x 128.
//
// A product of block-scaled operands sums over columns, so the same matrix is wanted
// along its rows (the forward product) and along its columns, transposed (the gradients
// of the weights, and of the inputs by the transposed weight).  Both come from one
// reading: a CTA has a tile of 128 x 128 in registers, a thread eight rows of eight
// columns, as they are in memory.  A row's maximum is found among the 16 lanes that share
// it, a column's among the warps in shared memory (maxima: no order in the result).  For
// the transposed form a thread's eight rows of a column are one 8-byte store into shared
// memory, the 8-byte units of a column swizzled by its group of eight columns (16 lanes then
// meet 32 different banks), and leave from there as whole 128-byte lines.
//
// Bound by memory and, both ways at once, by the instructions and barriers between reading a
// tile and writing it (8192 x 6656 bf16: 26.4 us along rows, 164 MB, 6.2 TB/s; both ways 39.8
// us, 222 MB, 5.6 TB/s, 60 % of the issue slots).  Four CTAs per SM of 64 registers: 51.8 us.
// Dealing out the tiles in blocks of 2 .. 16 rows of tiles changed nothing.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <mutex>

#include "blocks.cuh"
#include "f32x2.cuh"
#include "host_util.h"
#include "ptx.cuh"
#include "ptx_async.cuh"
#include "rows_host.h"
#include "vlmce.h"

namespace vlmce {
namespace quant {
namespace {

constexpr int kB = blocks::kBlock;
constexpr int kThreads = 256;

struct Params {
    const unsigned char *x;
    unsigned char *q, *qt;
    float *scale, *scale_t;
    int64_t x_ld, x_batch;        // bytes
    int64_t q_ld, q_batch, qt_ld, qt_batch;
    int64_t R, C;
    int batch, rt, ct;            // matrices, tiles down and across
    int square;
    int q_vec, qt_vec;            // q's rows take 8-byte stores, qt's 16-byte ones
    uintptr_t first, last;        // x's memory
};

// Whether a CTA goes on to other tiles, staged: aligned ones of 16-bit values (an fp32
// thread's 32 bytes are two copies, half a sector each: 4096 x 6656 both ways 45 us, a tile a
// CTA from registers 30; bf16, 8192 x 6656: along rows, transposed, both 26.4, 26.4 and 39.8 us
// so, 26.7, 29.5 and 41.4 a tile a CTA).  Squares go on for kSquareRun tiles, so that the
// last ones are dealt out as CTAs end (both ways 35.7, to the end 39.7, a tile a CTA 36.4).
template <int DT, bool ALIGNED>
constexpr bool kStaged = ALIGNED && DT != VLMCE_F32;
constexpr int kSquareRun = 4;
constexpr int kStage = kB * kB * 2;
template <int DT>
constexpr int kCtas = DT == VLMCE_F32 ? 2 : 3;

// A thread's eight rows of eight columns, as they are in memory: 16-bit ones two to a
// word.  Magnitudes are compared as they are, too (16-bit ones two at a time).
template <int DT>
struct Tile {
    static constexpr bool k16 = DT != VLMCE_F32;
    static constexpr int kWords = k16 ? 4 : 8;  // of a row
    uint32_t u[8][kWords];

    // The larger magnitudes of two words, signs aside (any sign in the result).
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
        uint32_t r;
        if constexpr (DT == VLMCE_BF16)
            asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        else if constexpr (DT == VLMCE_F16)
            asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        else {
            float m;
            asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(m) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
            r = __float_as_uint(m);
        }
        return r;
    }
    static __device__ __forceinline__ uint32_t magnitudes(uint32_t w) { return w & (k16 ? 0x7fff7fffu : 0x7fffffffu); }
    // Columns 2 k and 2 k + 1 of row i.
    __device__ __forceinline__ uint64_t pair(int i, int k) const {
        if constexpr (k16) {
            float a, b;
            act::unpack16x2(u[i][k], a, b, DT == VLMCE_F16);
            return pack2(__float_as_uint(a), __float_as_uint(b));
        } else {
            return pack2(u[i][2 * k], u[i][2 * k + 1]);
        }
    }
    // The larger magnitude of a word, as an fp32 number's bits.
    static __device__ __forceinline__ uint32_t widest(uint32_t w) {
        if constexpr (k16) {
            const uint16_t m = static_cast<uint16_t>(max(w & 0xffffu, w >> 16));
            return __float_as_uint(act::from16(m, DT == VLMCE_F16));
        } else {
            return w;
        }
    }
    // Row i from `from`, 16-byte aligned, or zeros.
    __device__ __forceinline__ void load16(int i, const unsigned char *from, bool in) {
#pragma unroll
        for (int k = 0; k < kWords / 4; ++k) {
            const uint4 q = in ? reinterpret_cast<const uint4 *>(from)[k] : make_uint4(0, 0, 0, 0);
            u[i][4 * k] = q.x, u[i][4 * k + 1] = q.y, u[i][4 * k + 2] = q.z, u[i][4 * k + 3] = q.w;
        }
    }
    // Row i out of the 16-byte units that hold it, of which it starts `off` bytes in.
    __device__ __forceinline__ void place(int i, uint32_t (&w)[kWords + 4], uint32_t off) {
        blocks::move_into_place<kWords, k16>(w, off);
#pragma unroll
        for (int k = 0; k < kWords; ++k) u[i][k] = w[k];
    }
    // At any alignment, eight rows `ld` bytes apart whose units lie within x's memory: four
    // rows' loads at a time (in a branch for each row they wait for one another: 7042 x 6722
    // bf16 along rows 54 us).
    __device__ __forceinline__ void load_units(const unsigned char *from, int64_t ld) {
#pragma unroll
        for (int h = 0; h < 8; h += 4) {
            uint32_t w[4][kWords + 4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uintptr_t unit = reinterpret_cast<uintptr_t>(from + (h + i) * ld) & ~uintptr_t{15};
#pragma unroll
                for (int k = 0; k <= kWords / 4; ++k) {
                    const uint4 q = *reinterpret_cast<const uint4 *>(unit + 16 * k);
                    w[i][4 * k] = q.x, w[i][4 * k + 1] = q.y, w[i][4 * k + 2] = q.z, w[i][4 * k + 3] = q.w;
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                place(h + i, w[i], static_cast<uint32_t>(reinterpret_cast<uintptr_t>(from + (h + i) * ld) & 15));
        }
    }
    static constexpr int kUnitBytes = 4 * kWords + 16;  // of a row's units
    // At any alignment, the first n values (n may be 0, or less): the units, where those lie
    // between `first` and `last`; else one by one.
    __device__ __forceinline__ void load(int i, const unsigned char *from, int64_t n, uintptr_t first,
                                         uintptr_t last) {
        constexpr int kElt = k16 ? 2 : 4;
        const uintptr_t a = reinterpret_cast<uintptr_t>(from), unit = a & ~uintptr_t{15};
        const uint32_t off = static_cast<uint32_t>(a & 15);
        const int64_t take = n < 8 ? n : 8;
        if (take > 0 && unit >= first && ((a + take * kElt + 15) & ~uintptr_t{15}) <= last) {
            uint32_t w[kWords + 4];
#pragma unroll
            for (int k = 0; k <= kWords / 4; ++k) {
                uint4 q = make_uint4(0, 0, 0, 0);
                if (16u * k < off + take * kElt) q = *reinterpret_cast<const uint4 *>(unit + 16 * k);
                w[4 * k] = q.x, w[4 * k + 1] = q.y, w[4 * k + 2] = q.z, w[4 * k + 3] = q.w;
            }
            place(i, w, off);
            if (take < 8) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j >= take) {
                        if constexpr (k16)
                            u[i][j / 2] &= j & 1 ? 0xffffu : 0xffff0000u;
                        else
                            u[i][j] = 0;
                    }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if constexpr (k16) {
                    const uint32_t e = j < take ? reinterpret_cast<const uint16_t *>(from)[j] : 0;
                    u[i][j / 2] = j & 1 ? u[i][j / 2] | e << 16 : e;
                } else {
                    u[i][j] = j < take ? reinterpret_cast<const uint32_t *>(from)[j] : 0;
                }
            }
        }
    }
};

// Where a tile is: its matrix, and its place down and across.
struct Where {
    int b, tr, tc;
    __device__ __forceinline__ Where(const Params &p, unsigned at) {
        int tile = static_cast<int>(at);
        b = tile / (p.rt * p.ct);
        tile -= b * (p.rt * p.ct);
        tr = tile / p.ct;
        tc = tile - tr * p.ct;
    }
};

template <int DT, bool ALIGNED, bool ROWS, bool TRANS>
__global__ void __launch_bounds__(kThreads, kCtas<DT>) quant_kernel(const Params p) {
    using T = Tile<DT>;
    constexpr int kWarps = kThreads / 32, kW = T::kWords;
    extern __shared__ __align__(16) unsigned char staged[];  // kStaged: kStage bytes
    __shared__ uint32_t tile_max[2][kWarps];
    __shared__ __align__(16) uint32_t col_max[TRANS ? kWarps : 1][16 * kW];
    __shared__ __align__(16) float col_inv[TRANS ? kB : 4];
    __shared__ __align__(16) unsigned char tq[TRANS ? kB * kB : 16];
    const int tid = threadIdx.x, lane = tid & 31;
    const int cg = tid & 15, rg = tid >> 4;  // eight columns, eight rows of the tile
    const unsigned tiles = static_cast<unsigned>(p.batch * p.rt * p.ct), step = gridDim.x;
    // Each thread's own part of a tile on its way to its own slots: no barrier, and the next
    // tile's loads are in flight while this one is worked on.
    const uint32_t slot = ptx::smem_addr(staged) + 16u * tid;
    auto fetch = [&](unsigned tile) {  // (16-bit values)
        const Where at(p, tile);
        const int64_t r0 = static_cast<int64_t>(at.tr) * kB + 8 * rg, c0 = static_cast<int64_t>(at.tc) * kB + 8 * cg;
        const unsigned char *from = p.x + at.b * p.x_batch + r0 * p.x_ld + c0 * blocks::elt_bytes<DT>;
        const bool in = c0 < p.C;
        const int rows_in = static_cast<int>(min(int64_t{8}, p.R - r0));
#pragma unroll
        for (int i = 0; i < 8; ++i, from += p.x_ld) {
            const bool have = in && i < rows_in;
            ptx::cp_async16_first(slot + i * (16 * kThreads), have ? from : p.x, have ? 16 : 0);
        }
        ptx::cp_async_commit();
    };
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    if constexpr (kStaged<DT, ALIGNED>) fetch(blockIdx.x);
    int parity = 0;
    for (unsigned tile = blockIdx.x; tile < tiles; tile += step, parity ^= 1) {
        const Where at(p, tile);
        const int64_t b = at.b;
        const int tr = at.tr, tc = at.tc;
        const int64_t r0 = static_cast<int64_t>(tr) * kB + 8 * rg, c0 = static_cast<int64_t>(tc) * kB + 8 * cg;
        const int rows_in = static_cast<int>(min(int64_t{8}, p.R - r0));  // of the eight (may be less than 0)
        const int64_t cols_in = p.C - c0;
        T v;
        if constexpr (kStaged<DT, ALIGNED>) {
            ptx::cp_async_wait<0>();
#pragma unroll
            for (int i = 0; i < 8; ++i) v.load16(i, staged + 16 * (i * kThreads + tid), true);
            if (tile + step < tiles) fetch(tile + step);
        } else {
            const unsigned char *x = p.x + b * p.x_batch + r0 * p.x_ld + c0 * blocks::elt_bytes<DT>;
            const uintptr_t end = (reinterpret_cast<uintptr_t>(x + 7 * p.x_ld) & ~uintptr_t{15}) + T::kUnitBytes;
            if (!ALIGNED && rows_in >= 8 && cols_in >= 8 &&
                (reinterpret_cast<uintptr_t>(x) & ~uintptr_t{15}) >= p.first && end <= p.last) {
                v.load_units(x, p.x_ld);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if constexpr (ALIGNED)
                        v.load16(i, x + i * p.x_ld, i < rows_in && cols_in > 0);
                    else
                        v.load(i, x + i * p.x_ld, i < rows_in ? cols_in : 0, p.first, p.last);
            }
        }
        float tile_inv = 1.f;
        if (p.square) {
            uint32_t a = v.u[0][0];
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int k = 0; k < kW; ++k) a = T::larger(a, v.u[i][k]);
            a = __reduce_max_sync(0xffffffffu, T::widest(T::magnitudes(a)));
            if (lane == 0) tile_max[parity][tid >> 5] = a;  // (the other may still be read)
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kWarps; ++w) a = max(a, tile_max[parity][w]);
            const float scale = blocks::scale_of(a, tile_inv);
            if (tid == 0) {
                if (ROWS) p.scale[(b * p.rt + tr) * p.ct + tc] = scale;
                if (TRANS) p.scale_t[(b * p.ct + tc) * p.rt + tr] = scale;
            }
        } else if constexpr (TRANS) {
            uint32_t *mine = col_max[tid >> 5] + kW * cg;  // of the warp's 16 rows
#pragma unroll
            for (int k = 0; k < kW; ++k) {
                uint32_t a = v.u[0][k];
#pragma unroll
                for (int i = 1; i < 8; ++i) a = T::larger(a, v.u[i][k]);
                a = T::larger(a, __shfl_xor_sync(0xffffffffu, a, 16));
                if (lane < 16) mine[k] = T::magnitudes(a);
            }
        }
        if constexpr (ROWS) {
            unsigned char *q = p.q + b * p.q_batch + r0 * p.q_ld;
            float mine = tile_inv;  // of row lane % 8 of the eight
            if (!p.square) {
                // the eight rows' maxima over the 16 lanes: each step, a lane gives away half of
                // its rows and takes the other half's values (8 exchanges instead of 32)
                uint32_t m[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    m[i] = v.u[i][0];
#pragma unroll
                    for (int k = 1; k < kW; ++k) m[i] = T::larger(m[i], v.u[i][k]);
                }
#pragma unroll
                for (int d = 4; d > 0; d /= 2)
#pragma unroll
                    for (int i = 0; i < d; ++i) {
                        const bool upper = lane & d;
                        const uint32_t keep = upper ? m[i + d] : m[i], give = upper ? m[i] : m[i + d];
                        m[i] = T::larger(keep, __shfl_xor_sync(0xffffffffu, give, d));
                    }
                m[0] = T::magnitudes(T::larger(m[0], __shfl_xor_sync(0xffffffffu, m[0], 8)));
                // (the two divisions cost more than the values' own arithmetic: one row a lane)
                const float scale = blocks::scale_of(T::widest(m[0]), mine);
                if (cg < 8 && r0 + cg < p.R) p.scale[(b * p.R + r0 + cg) * p.ct + tc] = scale;
            }
            const bool wide = p.q_vec && cols_in >= 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint64_t inv = both(__shfl_sync(0xffffffffu, mine, (lane & 16) + i));
                float f[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) unpack2(mul2(v.pair(i, k), inv), f[2 * k], f[2 * k + 1]);
                const uint32_t lo = blocks::pack_e4m3x4(f[0], f[1], f[2], f[3]);
                const uint32_t hi = blocks::pack_e4m3x4(f[4], f[5], f[6], f[7]);
                if (i < rows_in) {
                    unsigned char *row = q + i * p.q_ld + c0;
                    if (wide) {
                        *reinterpret_cast<uint2 *>(row) = make_uint2(lo, hi);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (j < cols_in) row[j] = static_cast<unsigned char>((j < 4 ? lo : hi) >> (8 * (j & 3)));
                    }
                }
            }
        }
        if constexpr (TRANS) {
            uint64_t invs[4];  // of the eight columns
            if (!p.square) {
                __syncthreads();  // col_max is complete
                if (tid < kB) {   // a column a thread
                    uint32_t a = 0;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        if constexpr (T::k16)
                            a = max(a, static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(col_max[w])[tid]));
                        else
                            a = max(a, col_max[w][tid]);
                    }
                    float inv;
                    const float scale = blocks::scale_of(T::widest(a), inv);
                    const int64_t col = static_cast<int64_t>(tc) * kB + tid;
                    if (col < p.C) p.scale_t[(b * p.C + col) * p.rt + tr] = scale;
                    col_inv[tid] = inv;
                }
                __syncthreads();
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
                    const ulonglong2 f = *reinterpret_cast<const ulonglong2 *>(col_inv + 8 * cg + 2 * k);
                    invs[k] = f.x, invs[k + 1] = f.y;
                }
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) invs[k] = both(tile_inv);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float e[8], o[8];  // columns 2 k and 2 k + 1
#pragma unroll
                for (int i = 0; i < 8; ++i) unpack2(mul2(v.pair(i, k), invs[k]), e[i], o[i]);
                unsigned char *to = tq + (8 * cg + 2 * k) * kB + 8 * (rg ^ cg);
                *reinterpret_cast<uint2 *>(to) =
                    make_uint2(blocks::pack_e4m3x4(e[0], e[1], e[2], e[3]), blocks::pack_e4m3x4(e[4], e[5], e[6], e[7]));
                *reinterpret_cast<uint2 *>(to + kB) =
                    make_uint2(blocks::pack_e4m3x4(o[0], o[1], o[2], o[3]), blocks::pack_e4m3x4(o[4], o[5], o[6], o[7]));
            }
            __syncthreads();
            // 16 rows a thread, eight threads a column, every 32nd column
            const int c = tid >> 3, u = tid & 7;
            const int64_t r = static_cast<int64_t>(tr) * kB + 16 * u, col = static_cast<int64_t>(tc) * kB + c;
            const int left = static_cast<int>(min(int64_t{16}, p.R - r));
            if (left <= 0) continue;
            unsigned char *to = p.qt + b * p.qt_batch + col * p.qt_ld + r;
            const bool wide = p.qt_vec && left == 16;
#pragma unroll
            for (int i = 0; i < kB * kB / 16 / kThreads; ++i) {
                if (col + 32 * i >= p.C) break;
                const unsigned char *from = tq + (c + 32 * i) * kB;
                const int swizzle = (c >> 3) + 4 * i;
                const uint2 lo = *reinterpret_cast<const uint2 *>(from + 8 * ((2 * u) ^ swizzle));
                const uint2 hi = *reinterpret_cast<const uint2 *>(from + 8 * ((2 * u + 1) ^ swizzle));
                if (wide) {
                    *reinterpret_cast<uint4 *>(to) = make_uint4(lo.x, lo.y, hi.x, hi.y);
                } else {
                    const uint32_t w[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        if (k < left) to[k] = static_cast<unsigned char>(w[k / 4] >> (8 * (k & 3)));
                }
                to += 32 * p.qt_ld;
            }
        }
    }
}

using Kernel = void (*)(const Params);
template <int DT, bool ALIGNED>
Kernel kernel_of(bool rows, bool trans) {
    if (!trans) return quant_kernel<DT, ALIGNED, true, false>;
    return rows ? quant_kernel<DT, ALIGNED, true, true> : quant_kernel<DT, ALIGNED, false, true>;
}
Kernel kernel_of(int dt, bool vec, bool rows, bool trans) {
    switch (dt) {
        case VLMCE_F32:
            return vec ? kernel_of<VLMCE_F32, true>(rows, trans) : kernel_of<VLMCE_F32, false>(rows, trans);
        case VLMCE_F16:
            return vec ? kernel_of<VLMCE_F16, true>(rows, trans) : kernel_of<VLMCE_F16, false>(rows, trans);
        default:
            return vec ? kernel_of<VLMCE_BF16, true>(rows, trans) : kernel_of<VLMCE_BF16, false>(rows, trans);
    }
}

// The kernels that stage tiles, their shared memory, once per device.
cudaError_t opt_in(int device) {
    static std::mutex mu;
    static bool done[64] = {};
    std::lock_guard<std::mutex> lock(mu);
    cudaError_t e = cudaSuccess;
    if (!done[device]) {
        for (const int dt : {VLMCE_BF16, VLMCE_F16})
            for (const int out : {1, 2, 3})
                if (e == cudaSuccess)
                    e = cudaFuncSetAttribute(kernel_of(dt, true, out & 1, out & 2),
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, kStage);
        done[device] = e == cudaSuccess;
    }
    return e;
}

}  // namespace
}  // namespace quant
}  // namespace vlmce

extern "C" vlmce_status quantize_blocks(const void *x, int32_t dtype, int64_t batch, int64_t R,
                                        int64_t C, int64_t x_stride, int64_t x_batch_stride,
                                        int32_t square, void *q, int64_t q_stride, float *scale,
                                        void *qt, int64_t qt_stride, float *scale_t,
                                        vlmce_stream_t stream) {
    using namespace vlmce;
    using namespace vlmce::quant;
    if (dtype != VLMCE_F32 && dtype != VLMCE_BF16 && dtype != VLMCE_F16)
        return VLMCE_ERR_UNSUPPORTED_DTYPE;
    const int elt = dtype == VLMCE_F32 ? 4 : 2;
    if (batch < 0 || R < 0 || C < 1 || x_stride < C || (!q && !qt) || (q && q_stride < C) ||
        (qt && qt_stride < R) || (q != nullptr) != (scale != nullptr) ||
        (qt != nullptr) != (scale_t != nullptr))
        return VLMCE_ERR_INVALID_ARG;
    if (batch == 0 || R == 0) return VLMCE_OK;
    if (!x || (batch > 1 && x_batch_stride < (R - 1) * x_stride + C)) return VLMCE_ERR_INVALID_ARG;
    constexpr int64_t kMax = int64_t(1) << 40;  // elements a stride may span
    if (R > INT32_MAX || C > INT32_MAX || batch > INT32_MAX || x_stride > kMax / R ||
        q_stride > kMax / R || qt_stride > kMax / C || x_batch_stride > kMax / batch ||
        (q && R * q_stride > kMax / batch) || (qt && C * qt_stride > kMax / batch))
        return VLMCE_ERR_TOO_LARGE;
    const int64_t rt = (R + kB - 1) / kB, ct = (C + kB - 1) / kB;
    if (rt * ct > INT32_MAX / batch) return VLMCE_ERR_TOO_LARGE;
    if (!aligned(x, static_cast<uintptr_t>(elt)) || !aligned(scale, 4) || !aligned(scale_t, 4))
        return VLMCE_ERR_MISALIGNED;
    // the matrices as one run of memory each
    struct Span {
        const void *p;
        int64_t bytes;
    };
    const Span in{x, ((batch - 1) * x_batch_stride + (R - 1) * x_stride + C) * elt};
    const int64_t blocks_of = batch * (square ? rt * ct : R * ct), blocks_t = batch * (square ? rt * ct : C * rt);
    const Span out[4] = {{q, batch * R * q_stride - (q_stride - C)}, {scale, 4 * blocks_of},
                         {qt, batch * C * qt_stride - (qt_stride - R)}, {scale_t, 4 * blocks_t}};
    auto meet = [](const Span &a, const Span &b) {
        return rows_overlap({a.p, 1, a.bytes, a.bytes}, {b.p, 1, b.bytes, b.bytes});
    };
    for (int i = 0; i < 4; ++i) {
        if (meet(out[i], in)) return VLMCE_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (meet(out[i], out[j])) return VLMCE_ERR_INVALID_ARG;
    }
    DeviceInfo dev;
    const vlmce_status st = current_device(&dev);
    if (st != VLMCE_OK) return st;
    Params p = {};
    p.x = static_cast<const unsigned char *>(x);
    p.q = static_cast<unsigned char *>(q);
    p.qt = static_cast<unsigned char *>(qt);
    p.scale = scale;
    p.scale_t = scale_t;
    p.x_ld = x_stride * elt;
    p.x_batch = batch > 1 ? x_batch_stride * elt : 0;
    p.q_ld = q_stride;
    p.q_batch = R * q_stride;
    p.qt_ld = qt_stride;
    p.qt_batch = C * qt_stride;
    p.R = R;
    p.C = C;
    p.batch = static_cast<int>(batch);
    p.rt = static_cast<int>(rt);
    p.ct = static_cast<int>(ct);
    p.square = square != 0;
    p.q_vec = aligned(q, 8) && q_stride % 8 == 0 && (batch == 1 || p.q_batch % 8 == 0);
    p.qt_vec = aligned(qt, 16) && qt_stride % 16 == 0;
    p.first = reinterpret_cast<uintptr_t>(x);
    p.last = p.first + static_cast<uintptr_t>(in.bytes);
    const bool vec = C % 8 == 0 && aligned(x, 16) && p.x_ld % 16 == 0 && p.x_batch % 16 == 0;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    const Kernel kernel = kernel_of(dtype, vec, q != nullptr, qt != nullptr);
    const int64_t tiles = batch * rt * ct;
    const bool staged = vec && dtype != VLMCE_F32;
    const int64_t at_once = std::min<int64_t>(tiles, kCtas<VLMCE_BF16> * dev.sm_count);
    const int64_t ctas = !staged ? tiles : square ? std::max(at_once, (tiles + kSquareRun - 1) / kSquareRun) : at_once;
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
    cfg.dynamicSmemBytes = staged ? kStage : 0;
    if (staged) {
        const cudaError_t e = opt_in(dev.device);
        if (e != cudaSuccess) return launch_status(e, "quantize_blocks");
    }
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return launch_status(
        cudaLaunchKernelEx(&cfg, kernel, static_cast<const Params>(p)), "quantize_blocks");
}
