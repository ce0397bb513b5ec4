// rmsnorm.cu -- root-mean-square norm of rows with the residual's addition,
// forward (output in the input type, or in e4m3 with one scale per row) and
// backward.
//
//   forward   s = x + residual,  rstd = (mean_j s_j^2 + eps)^-1/2,
//             y = s rstd (w + offset)
//   e4m3      scale = max_j |y_j| / 448,  q = e4m3(y / scale)
//   backward  a_j = dy_j (w_j + offset),  xhat = s rstd,
//             dx = rstd (a - xhat mean_j(a_j xhat_j)) + dresidual
//             dw_j = sum_t dy_j xhat_j
//
// All in fp32, each output rounded once; y is formed from the unrounded sum s.
// For e4m3 the row's sum of squares and max |s (w + offset)| come from one
// reduction: rstd cancels in y / scale = s (w + offset) 448 / max|s (w + offset)|.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <mutex>
#include <set>
#include <utility>

#include "act.cuh"
#include "colsum.cuh"
#include "host_util.h"
#include "ptx_async.cuh"
#include "rows_host.h"
#include "vlmce.h"

namespace vlmce {
namespace rms {
namespace {

template <int DT>
struct Elt {
    static constexpr int kBytes = DT == VLMCE_F32 ? 4 : 2;
    static constexpr int kPer16 = 16 / kBytes;
};

// E consecutive elements at element index i of a row (E = 16 bytes' worth, or 1).
template <int DT, int E>
__device__ __forceinline__ void load_e(const void *row, int i, float (&v)[E]) {
    if constexpr (E == 1) {
        if constexpr (DT == VLMCE_F32)
            v[0] = static_cast<const float *>(row)[i];
        else
            v[0] = act::from16(static_cast<const uint16_t *>(row)[i], DT == VLMCE_F16);
    } else if constexpr (DT == VLMCE_F32) {
        const float4 u = *reinterpret_cast<const float4 *>(static_cast<const float *>(row) + i);
        v[0] = u.x;
        v[1] = u.y;
        v[2] = u.z;
        v[3] = u.w;
    } else {
        const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(row) + i);
        act::unpack16x2(u.x, v[0], v[1], DT == VLMCE_F16);
        act::unpack16x2(u.y, v[2], v[3], DT == VLMCE_F16);
        act::unpack16x2(u.z, v[4], v[5], DT == VLMCE_F16);
        act::unpack16x2(u.w, v[6], v[7], DT == VLMCE_F16);
    }
}
template <int DT, int E>
__device__ __forceinline__ void store_e(void *row, int i, const float (&v)[E]) {
    if constexpr (E == 1) {
        if constexpr (DT == VLMCE_F32)
            static_cast<float *>(row)[i] = v[0];
        else
            static_cast<uint16_t *>(row)[i] = act::to16(v[0], DT == VLMCE_F16);
    } else if constexpr (DT == VLMCE_F32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(row) + i) =
            make_float4(v[0], v[1], v[2], v[3]);
    } else {
        constexpr bool f16 = DT == VLMCE_F16;
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(row) + i) =
            make_uint4(act::pack16x2(v[0], v[1], f16), act::pack16x2(v[2], v[3], f16),
                       act::pack16x2(v[4], v[5], f16), act::pack16x2(v[6], v[7], f16));
    }
}
template <int E>
__device__ __forceinline__ void store_e4m3(unsigned char *row, int i, const float (&v)[E]) {
    if constexpr (E == 1) {
        row[i] = __nv_cvt_float_to_fp8(v[0], __NV_SATFINITE, __NV_E4M3);
    } else {
        uint32_t u[E / 4];
#pragma unroll
        for (int j = 0; j < E / 4; ++j)
            u[j] = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * j], v[4 * j + 1]), __NV_SATFINITE,
                                            __NV_E4M3) |
                   static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(
                       make_float2(v[4 * j + 2], v[4 * j + 3]), __NV_SATFINITE, __NV_E4M3))
                       << 16;
        if constexpr (E == 8)
            *reinterpret_cast<uint2 *>(row + i) = make_uint2(u[0], u[1]);
        else
            *reinterpret_cast<uint32_t *>(row + i) = u[0];
    }
}
// The weight has the rows' type or fp32.
template <int DT, int E>
__device__ __forceinline__ void load_w(const void *w, bool f32, int i, float offset,
                                       float (&v)[E]) {
    if (DT == VLMCE_F32 || !f32) {
        load_e<DT, E>(w, i, v);
    } else if constexpr (E == 8) {
        float a[4], b[4];
        load_e<VLMCE_F32, 4>(w, i, a);
        load_e<VLMCE_F32, 4>(w, i + 4, b);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = a[j];
            v[4 + j] = b[j];
        }
    } else {
        load_e<VLMCE_F32, E>(w, i, v);
    }
#pragma unroll
    for (int j = 0; j < E; ++j) v[j] += offset;
}

// Granules at a row's ends (the ring kernels' SHIFT): elements i .. i + E of which
// only those in [0, H) belong to the row.
template <int E>
__device__ __forceinline__ bool at_end(int i, int H) {
    return i < 0 || i + E > H;
}
template <int E>
__device__ __forceinline__ void clear_outside(int i, int H, float (&v)[E]) {
    if (at_end<E>(i, H)) {
#pragma unroll
        for (int j = 0; j < E; ++j)
            if (i + j < 0 || i + j >= H) v[j] = 0.f;
    }
}
template <int DT, int E, bool E4M3>
__device__ __forceinline__ void store_inside(unsigned char *row, int i, int H,
                                             const float (&v)[E]) {
    if (!at_end<E>(i, H)) {
        if constexpr (E4M3)
            store_e4m3<E>(row, i, v);
        else
            store_e<DT, E>(row, i, v);
        return;
    }
#pragma unroll
    for (int j = 0; j < E; ++j)
        if (i + j >= 0 && i + j < H) {
            const float one[1] = {v[j]};
            if constexpr (E4M3)
                store_e4m3<1>(row, i + j, one);
            else
                store_e<DT, 1>(row, i + j, one);
        }
}
// Weights i .. i + E at any alignment, zeros outside the row.
template <int DT, int E>
__device__ __forceinline__ void load_w_inside(const void *w, bool f32, int i, int H, float offset,
                                              float (&v)[E]) {
#pragma unroll
    for (int j = 0; j < E; ++j) {
        float one[1] = {0.f};
        if (i + j >= 0 && i + j < H) load_w<DT, 1>(w, f32, i + j, offset, one);
        v[j] = one[0];
    }
}

// Sum of a (and, with MAX, the maximum of m >= 0) over the block, in every
// thread.  sh: [2][32].
template <bool MAX>
__device__ __forceinline__ void warp_sum_max(float &a, float &m) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, off);
        if constexpr (MAX) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    }
}
template <bool MAX>
__device__ __forceinline__ void block_sum_max(float &a, float &m, float (*sh)[32]) {
    warp_sum_max<MAX>(a, m);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) {
        sh[0][warp] = a;
        if constexpr (MAX) sh[1][warp] = m;
    }
    __syncthreads();
    a = lane < warps ? sh[0][lane] : 0.f;
    if constexpr (MAX) m = lane < warps ? sh[1][lane] : 0.f;
    warp_sum_max<MAX>(a, m);
}

// ------------------------------------------------------------ forward
struct FwdParams {
    const unsigned char *x, *residual;
    const void *weight;
    unsigned char *y, *sum;
    float *rstd, *scale;
    int64_t T;
    int H;
    int64_t x_ld, residual_ld, y_ld, sum_ld;  // bytes
    float eps, offset;
    int w_f32;
};

// One CTA per row (few rows: latency-bound, 1.9 us for one row of 4096 bf16 in a
// stream of such calls); thread i holds the row's elements (i + k blockDim) E .. + E
// for k < NG in registers (fp32 sums), so memory is read once.  NG = 0: rows
// too wide for that; the sums are read again for the second pass.
template <int DT, int E, int NG, bool QUANT>
__global__ void __launch_bounds__(1024) fwd_kernel(const FwdParams p) {
    __shared__ float sh[2][32];
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int64_t row = blockIdx.x;
    const unsigned char *x = p.x + row * p.x_ld;
    const unsigned char *res = p.residual ? p.residual + row * p.residual_ld : nullptr;
    unsigned char *sum = p.sum ? p.sum + row * p.sum_ld : nullptr;
    unsigned char *y = p.y + row * p.y_ld;
    constexpr int kHold = NG > 0 ? NG : 1;
    float v[kHold][E];
    float ss = 0.f, mx = 0.f;
    auto sum_at = [&](int i, float (&s)[E]) {
        load_e<DT, E>(x, i, s);
        if (res) {
            float r[E];
            load_e<DT, E>(res, i, r);
#pragma unroll
            for (int j = 0; j < E; ++j) s[j] += r[j];
        }
    };
    auto fold = [&](int i, const float (&s)[E]) {
#pragma unroll
        for (int j = 0; j < E; ++j) ss = fmaf(s[j], s[j], ss);
        if constexpr (QUANT) {
            float w[E];
            load_w<DT, E>(p.weight, p.w_f32 != 0, i, p.offset, w);
#pragma unroll
            for (int j = 0; j < E; ++j) mx = fmaxf(mx, fabsf(s[j] * w[j]));
        }
    };
    const int step = static_cast<int>(blockDim.x) * E;
    const int i0 = static_cast<int>(threadIdx.x) * E;
    if constexpr (NG > 0) {
        // (a thread without a k-th element loads the row's last one, so that no
        // branch keeps the loads apart)
#pragma unroll
        for (int k = 0; k < NG; ++k) sum_at(min(i0 + k * step, p.H - E), v[k]);
#pragma unroll
        for (int k = 0; k < NG; ++k)
            if (i0 + k * step < p.H) {
                fold(i0 + k * step, v[k]);
                if (sum) store_e<DT, E>(sum, i0 + k * step, v[k]);
            }
    } else {
        for (int i = i0; i < p.H; i += step) {
            sum_at(i, v[0]);
            fold(i, v[0]);
        }
    }
    block_sum_max<QUANT>(ss, mx, sh);
    const float rstd = __frsqrt_rn(ss / static_cast<float>(p.H) + p.eps);
    mx = fmaxf(mx, 1e-30f);
    if (threadIdx.x == 0) {
        if (p.rstd) p.rstd[row] = rstd;
        if constexpr (QUANT) p.scale[row] = rstd * mx / 448.f;
    }
    const float mul = QUANT ? 448.f / mx : rstd;
    auto emit = [&](int i, const float (&s)[E]) {
        float w[E], o[E];
        load_w<DT, E>(p.weight, p.w_f32 != 0, i, p.offset, w);
        if constexpr (QUANT) {
#pragma unroll
            for (int j = 0; j < E; ++j) o[j] = s[j] * w[j] * mul;
            store_e4m3<E>(y, i, o);
        } else {
#pragma unroll
            for (int j = 0; j < E; ++j) o[j] = s[j] * mul * w[j];
            store_e<DT, E>(y, i, o);
        }
    };
    if constexpr (NG > 0) {
#pragma unroll
        for (int k = 0; k < NG; ++k)
            if (i0 + k * step < p.H) emit(i0 + k * step, v[k]);
    } else {
        for (int i = i0; i < p.H; i += step) {
            sum_at(i, v[0]);
            if (sum) store_e<DT, E>(sum, i, v[0]);
            emit(i, v[0]);
        }
    }
}

// Many rows: CTAs stay and take rows blockIdx.x, + gridDim.x, ...  A thread owns
// the same kOwn granules of every row, with their weights in registers, and
// keeps the granules of the next kAhead - 1 rows on their way into its own slots
// of shared memory, so loads never wait for a row's reduction and stores.  At
// least two CTAs share an SM: one works while the other meets at its barrier.
// HBM-bound: 8192 x 6656 bf16 to e4m3 60.5 us = 6.3 TB/s (93 % of the measured copy
// rate; 74 us with one CTA per row), 8192 x 8192 bf16 88 us (90 %).
constexpr int kOwn = 2;
constexpr int kRingThreads = 512;  // most threads of a CTA
constexpr int kBwdAhead = 2;

// SHIFT: rows whose first element is not on a 16-byte boundary.  Granules are those
// of the memory, so the row's first element is element `shift` of its first granule;
// all arrays have the same shift in a row, and the grid's size is a multiple of E, so a
// CTA's rows all have it too (its weights stay where they are).  A granule at a row's
// start also reads the end of the row before, which is left out of everything.
// 8192 x 6661 bf16 77 us (147 element by element), to e4m3 66 us (131).
template <int DT, bool QUANT, int kFwdAhead, bool SHIFT>
__global__ void __launch_bounds__(kRingThreads, 2) fwd_ring_kernel(const FwdParams p) {
    constexpr int E = Elt<DT>::kPer16;
    extern __shared__ __align__(16) unsigned char ring[];  // [kFwdAhead][2][kOwn][threads][16]
    __shared__ float sh[2][2][32];
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    int at[kOwn];
    bool in[kOwn];
    float w[kOwn][E];
    const int shift =
        SHIFT ? static_cast<int>(blockIdx.x * (p.x_ld / Elt<DT>::kBytes) % E) : 0;
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
        at[k] = static_cast<int>(k * blockDim.x + threadIdx.x) * E - shift;
        in[k] = at[k] < p.H;
        if constexpr (SHIFT)
            load_w_inside<DT, E>(p.weight, p.w_f32 != 0, at[k], p.H, p.offset, w[k]);
        else if (in[k])
            load_w<DT, E>(p.weight, p.w_f32 != 0, at[k], p.offset, w[k]);
    }
    auto copy = [&](unsigned char *dst, const unsigned char *row, int i) {
        const unsigned char *src = row + i * Elt<DT>::kBytes;
        if constexpr (SHIFT)
            ptx::cp_async16_first(ptx::smem_addr(dst), src, min(E, p.H - i) * Elt<DT>::kBytes);
        else
            ptx::cp_async16(ptx::smem_addr(dst), src);
    };
    auto slot = [&](int s, int which, int k) {
        return ring + 16 * (((s * 2 + which) * kOwn + k) * blockDim.x + threadIdx.x);
    };
    auto fetch = [&](int64_t row, int s) {
        if (row < p.T) {
#pragma unroll
            for (int k = 0; k < kOwn; ++k)
                if (in[k]) {
                    copy(slot(s, 0, k), p.x + row * p.x_ld, at[k]);
                    if (p.residual) copy(slot(s, 1, k), p.residual + row * p.residual_ld, at[k]);
                }
        }
        ptx::cp_async_commit();
    };
    const int64_t step = gridDim.x;
    for (int n = 0; n < kFwdAhead - 1; ++n) fetch(blockIdx.x + n * step, n);
    int s = 0, flip = 0;
    for (int64_t row = blockIdx.x; row < p.T; row += step, flip ^= 1) {
        fetch(row + (kFwdAhead - 1) * step, s == 0 ? kFwdAhead - 1 : s - 1);
        ptx::cp_async_wait<kFwdAhead - 1>();
        float v[kOwn][E];
        float ss = 0.f, mx = 0.f;
#pragma unroll
        for (int k = 0; k < kOwn; ++k)
            if (in[k]) {
                load_e<DT, E>(slot(s, 0, k), 0, v[k]);
                if (p.residual) {
                    float r[E];
                    load_e<DT, E>(slot(s, 1, k), 0, r);
#pragma unroll
                    for (int j = 0; j < E; ++j) v[k][j] += r[j];
                }
                if constexpr (SHIFT) clear_outside<E>(at[k], p.H, v[k]);
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    ss = fmaf(v[k][j], v[k][j], ss);
                    if constexpr (QUANT) mx = fmaxf(mx, fabsf(v[k][j] * w[k][j]));
                }
                if (p.sum) {
                    if constexpr (SHIFT)
                        store_inside<DT, E, false>(p.sum + row * p.sum_ld, at[k], p.H, v[k]);
                    else
                        store_e<DT, E>(p.sum + row * p.sum_ld, at[k], v[k]);
                }
            }
        block_sum_max<QUANT>(ss, mx, sh[flip]);  // two buffers: one barrier a row
        const float rstd = __frsqrt_rn(ss / static_cast<float>(p.H) + p.eps);
        mx = fmaxf(mx, 1e-30f);
        if (threadIdx.x == 0) {
            if (p.rstd) p.rstd[row] = rstd;
            if constexpr (QUANT) p.scale[row] = rstd * mx / 448.f;
        }
        const float mul = QUANT ? 448.f / mx : rstd;
#pragma unroll
        for (int k = 0; k < kOwn; ++k)
            if (in[k]) {
#pragma unroll
                for (int j = 0; j < E; ++j)
                    v[k][j] = QUANT ? v[k][j] * w[k][j] * mul : v[k][j] * mul * w[k][j];
                if constexpr (SHIFT)
                    store_inside<DT, E, QUANT>(p.y + row * p.y_ld, at[k], p.H, v[k]);
                else if constexpr (QUANT)
                    store_e4m3<E>(p.y + row * p.y_ld, at[k], v[k]);
                else
                    store_e<DT, E>(p.y + row * p.y_ld, at[k], v[k]);
            }
        if (++s == kFwdAhead) s = 0;
    }
}

// ------------------------------------------------------------ backward
// A thread's columns i .. i + E of a CTA's partial dw, in whole 16 bytes (in single
// floats, 8 apart in a warp, they took 600 x 4096 bf16 from 9.1 to 16.7 us).
template <int E>
__device__ __forceinline__ void store_part(float *part, int i, const float (&dw)[E]) {
    if constexpr (E == 1) {
        part[i] = dw[0];
    } else {
#pragma unroll
        for (int j = 0; j < E; j += 4)
            *reinterpret_cast<float4 *>(part + i + j) =
                make_float4(dw[j], dw[j + 1], dw[j + 2], dw[j + 3]);
    }
}

struct BwdParams {
    const unsigned char *dy, *x, *dres;
    const void *weight;
    const float *rstd;
    unsigned char *dx;
    float *part;       // [CTAs][H] partial dw, or null
    float *dot;        // wide rows: [T] mean_j(a_j xhat_j)
    int64_t T;
    int H;
    int64_t dy_ld, x_ld, dres_ld, dx_ld;  // bytes
    float offset;
    int w_f32;
    int groups;        // ring kernel: rows a CTA works on at once
};

// Each CTA takes rows blockIdx.x, + gridDim.x, ...; a thread owns the same
// columns in all of them, so dw accumulates in registers.
template <int DT, int E, int NG>
__global__ void __launch_bounds__(1024) bwd_kernel(const BwdParams p) {
    __shared__ float sh[2][2][32];
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int step = static_cast<int>(blockDim.x) * E;
    const int i0 = static_cast<int>(threadIdx.x) * E;
    float dw[NG][E];
#pragma unroll
    for (int k = 0; k < NG; ++k)
#pragma unroll
        for (int j = 0; j < E; ++j) dw[k][j] = 0.f;
    int flip = 0;
    for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x, flip ^= 1) {
        const unsigned char *dy = p.dy + row * p.dy_ld, *x = p.x + row * p.x_ld;
        const float rstd = p.rstd[row];
        float a[NG][E], h[NG][E];
        float c = 0.f, unused = 0.f;
#pragma unroll
        for (int k = 0; k < NG; ++k) {  // (as in fwd_kernel)
            const int i = min(i0 + k * step, p.H - E);
            load_e<DT, E>(dy, i, a[k]);
            load_e<DT, E>(x, i, h[k]);
        }
#pragma unroll
        for (int k = 0; k < NG; ++k) {
            const int i = i0 + k * step;
            if (i < p.H) {
                float w[E];
                load_w<DT, E>(p.weight, p.w_f32 != 0, i, p.offset, w);
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    h[k][j] *= rstd;
                    dw[k][j] = fmaf(a[k][j], h[k][j], dw[k][j]);
                    a[k][j] *= w[j];
                    c = fmaf(a[k][j], h[k][j], c);
                }
            }
        }
        block_sum_max<false>(c, unused, sh[flip]);  // two buffers: one barrier a row
        c /= static_cast<float>(p.H);
#pragma unroll
        for (int k = 0; k < NG; ++k) {
            const int i = i0 + k * step;
            if (i < p.H) {
                float r[E];
#pragma unroll
                for (int j = 0; j < E; ++j) r[j] = 0.f;
                if (p.dres) load_e<DT, E>(p.dres + row * p.dres_ld, i, r);
#pragma unroll
                for (int j = 0; j < E; ++j) r[j] = fmaf(rstd, a[k][j] - h[k][j] * c, r[j]);
                store_e<DT, E>(p.dx + row * p.dx_ld, i, r);
            }
        }
    }
    if (p.part) {
        float *part = p.part + static_cast<int64_t>(blockIdx.x) * p.H;
#pragma unroll
        for (int k = 0; k < NG; ++k)
            if (i0 + k * step < p.H) store_part<E>(part, i0 + k * step, dw[k]);
    }
}

// The same with the ring of fwd_ring_kernel, read a second time after a row's
// reduction instead of held in registers.  With MULTI a CTA works on `groups` short
// rows at once, each with its own threads and named barrier, and adds up their dw at
// the end, so that two CTAs per SM leave few partial rows (its weights are in shared
// memory: in registers they would spill).  HBM-bound for long rows: 8192 x
// 6656 bf16 67 us (70 with the sum of the partial rows; 118 with one row per CTA
// loaded at a time), 8192 x 8192 83 us (95 %); short rows are bound by a row's chain
// of reduction and stores (8192 x 2048 30 us, 67 %).  SHIFT as above: 8192 x 6661 83 us
// (225 element by element).
template <int DT, bool MULTI, bool SHIFT>
__global__ void __launch_bounds__(kRingThreads, 2) bwd_ring_kernel(const BwdParams p) {
    constexpr int E = Elt<DT>::kPer16;
    extern __shared__ __align__(16) unsigned char ring[];  // [kBwdAhead][3][kOwn][threads][16]
    __shared__ float sh[2][kRingThreads / 32];
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int groups = MULTI ? p.groups : 1;
    const int gt = MULTI ? static_cast<int>(blockDim.x) / groups : static_cast<int>(blockDim.x);
    const int gw = gt >> 5;
    const int group = MULTI ? static_cast<int>(threadIdx.x) / gt : 0;
    const int tg = static_cast<int>(threadIdx.x) - group * gt;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * groups + group;
    const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
    int at[kOwn];
    bool in[kOwn];
    float w[kOwn][E], dw[kOwn][E];
    const int shift = SHIFT ? static_cast<int>(first * (p.x_ld / Elt<DT>::kBytes) % E) : 0;
    auto load = [&](int i, float offset, float (&v)[E]) {
        if constexpr (SHIFT)
            load_w_inside<DT, E>(p.weight, p.w_f32 != 0, i, p.H, offset, v);
        else
            load_w<DT, E>(p.weight, p.w_f32 != 0, i, offset, v);
    };
    auto w_slot = [&](int k) {  // MULTI: weights of the rows' type
        return ring + 16 * ((kBwdAhead * 3 * kOwn + k) * blockDim.x + threadIdx.x);
    };
    auto weights = [&](int k, float (&v)[E]) {
        if (DT != VLMCE_F32 && p.w_f32 != 0) {
            load(at[k], p.offset, v);
        } else {
            load_e<DT, E>(w_slot(k), 0, v);
#pragma unroll
            for (int j = 0; j < E; ++j) v[j] += p.offset;
        }
    };
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
        at[k] = (k * gt + tg) * E - shift;
        in[k] = at[k] < p.H;
        if (in[k]) {
            load(at[k], MULTI ? 0.f : p.offset, w[k]);
            if constexpr (MULTI) store_e<DT, E>(w_slot(k), 0, w[k]);
        }
#pragma unroll
        for (int j = 0; j < E; ++j) dw[k][j] = 0.f;
    }
    auto slot = [&](int s, int which, int k) {
        return ring + 16 * (((s * 3 + which) * kOwn + k) * blockDim.x + threadIdx.x);
    };
    auto copy = [&](unsigned char *dst, const unsigned char *row, int i) {
        const unsigned char *src = row + i * Elt<DT>::kBytes;
        if constexpr (SHIFT)
            ptx::cp_async16_first(ptx::smem_addr(dst), src, min(E, p.H - i) * Elt<DT>::kBytes);
        else
            ptx::cp_async16(ptx::smem_addr(dst), src);
    };
    auto fetch = [&](int64_t row, int s) {
        if (row < p.T) {
#pragma unroll
            for (int k = 0; k < kOwn; ++k)
                if (in[k]) {
                    copy(slot(s, 0, k), p.dy + row * p.dy_ld, at[k]);
                    copy(slot(s, 1, k), p.x + row * p.x_ld, at[k]);
                    if (p.dres) copy(slot(s, 2, k), p.dres + row * p.dres_ld, at[k]);
                }
        }
        ptx::cp_async_commit();
    };
    const float inv_h = 1.f / static_cast<float>(p.H);
    for (int n = 0; n < kBwdAhead - 1; ++n) fetch(first + n * step, n);
    float rstd = 0.f, next = first < p.T ? p.rstd[first] : 0.f;
    int s = 0, flip = 0;
    for (int64_t row = first; row < p.T; row += step, flip ^= 1) {
        rstd = next;
        if (row + step < p.T) next = p.rstd[row + step];
        fetch(row + (kBwdAhead - 1) * step, s == 0 ? kBwdAhead - 1 : s - 1);
        ptx::cp_async_wait<kBwdAhead - 1>();
        float c = 0.f, unused = 0.f;
#pragma unroll
        for (int k = 0; k < kOwn; ++k)
            if (in[k]) {
                float d[E], h[E];
                load_e<DT, E>(slot(s, 0, k), 0, d);
                load_e<DT, E>(slot(s, 1, k), 0, h);
                if constexpr (MULTI) weights(k, w[k]);
                if constexpr (SHIFT) {
                    clear_outside<E>(at[k], p.H, d);
                    clear_outside<E>(at[k], p.H, h);
                }
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    const float g = d[j] * (h[j] * rstd);
                    dw[k][j] += g;
                    c = fmaf(g, w[k][j], c);
                }
            }
        // sum over the group's warps; two buffers, so one barrier a row
        warp_sum_max<false>(c, unused);
        if (gw > 1) {
            if (lane == 0) sh[flip][warp] = c;
            if (MULTI)
                asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(gt) : "memory");
            else
                __syncthreads();
            c = lane < gw ? sh[flip][group * gw + lane] : 0.f;
            warp_sum_max<false>(c, unused);
        }
        c *= inv_h;
#pragma unroll
        for (int k = 0; k < kOwn; ++k)
            if (in[k]) {
                float d[E], h[E], r[E];
                load_e<DT, E>(slot(s, 0, k), 0, d);
                load_e<DT, E>(slot(s, 1, k), 0, h);
                if constexpr (MULTI) weights(k, w[k]);
#pragma unroll
                for (int j = 0; j < E; ++j) r[j] = 0.f;
                if (p.dres) load_e<DT, E>(slot(s, 2, k), 0, r);
#pragma unroll
                for (int j = 0; j < E; ++j)
                    r[j] = fmaf(rstd, fmaf(d[j], w[k][j], -(h[j] * rstd) * c), r[j]);
                if constexpr (SHIFT)
                    store_inside<DT, E, false>(p.dx + row * p.dx_ld, at[k], p.H, r);
                else
                    store_e<DT, E>(p.dx + row * p.dx_ld, at[k], r);
            }
        if (++s == kBwdAhead) s = 0;
    }
    if (!p.part) return;
    float *part = p.part + static_cast<int64_t>(blockIdx.x) * p.H;
    if constexpr (!MULTI && !SHIFT) {
#pragma unroll
        for (int k = 0; k < kOwn; ++k)
            if (in[k]) store_part<E>(part, at[k], dw[k]);
    } else {
        // [groups][kOwn gt E] floats in the ring, which no copy writes any more
        float *sum = reinterpret_cast<float *>(ring);
        const int width = kOwn * gt * E;
        ptx::cp_async_wait<0>();
        __syncthreads();
        if constexpr (SHIFT) {  // (each group's columns start elsewhere)
#pragma unroll
            for (int k = 0; k < kOwn; ++k)
#pragma unroll
                for (int j = 0; j < E; ++j)
                    if (at[k] + j >= 0 && at[k] + j < p.H)
                        sum[group * width + at[k] + j] = dw[k][j];
            __syncthreads();
            for (int i = static_cast<int>(threadIdx.x); i < p.H; i += static_cast<int>(blockDim.x)) {
                float a = sum[i];
                for (int g = 1; g < groups; ++g) a += sum[g * width + i];
                part[i] = a;
            }
            return;
        }
#pragma unroll
        for (int k = 0; k < kOwn; ++k)
            store_part<E>(sum + group * width, at[k], dw[k]);
        __syncthreads();
        for (int i = 4 * static_cast<int>(threadIdx.x); i < p.H;
             i += 4 * static_cast<int>(blockDim.x)) {
            float4 a = *reinterpret_cast<const float4 *>(sum + i);
            for (int g = 1; g < groups; ++g) {
                const float4 o = *reinterpret_cast<const float4 *>(sum + g * width + i);
                a.x += o.x;
                a.y += o.y;
                a.z += o.z;
                a.w += o.w;
            }
            *reinterpret_cast<float4 *>(part + i) = a;
        }
    }
}

// Rows too wide for one CTA's registers, and element by element from 4097 elements on
// (16 elements of four arrays per thread spill: 4096 x 6661 bf16 167 us, so: 117): the
// rows' mean(a xhat), then dx and the partial dw by column segments.
template <int DT, int E>
__global__ void __launch_bounds__(512) dot_kernel(const BwdParams p) {
    __shared__ float sh[2][32];
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int64_t row = blockIdx.x;
    const float rstd = p.rstd[row];
    float c = 0.f, unused = 0.f;
    for (int i = static_cast<int>(threadIdx.x) * E; i < p.H; i += static_cast<int>(blockDim.x) * E) {
        float d[E], h[E], w[E];
        load_e<DT, E>(p.dy + row * p.dy_ld, i, d);
        load_e<DT, E>(p.x + row * p.x_ld, i, h);
        load_w<DT, E>(p.weight, p.w_f32 != 0, i, p.offset, w);
#pragma unroll
        for (int j = 0; j < E; ++j) c = fmaf(d[j] * w[j], h[j] * rstd, c);
    }
    block_sum_max<false>(c, unused, sh);
    if (threadIdx.x == 0) p.dot[row] = c / static_cast<float>(p.H);
}
template <int DT, int E>
__global__ void __launch_bounds__(512) segment_kernel(const BwdParams p) {
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int i = static_cast<int>(blockIdx.x * blockDim.x + threadIdx.x) * E;
    if (i >= p.H) return;
    float dw[E], w[E];
    load_w<DT, E>(p.weight, p.w_f32 != 0, i, p.offset, w);
#pragma unroll
    for (int j = 0; j < E; ++j) dw[j] = 0.f;
    constexpr int R = E == 1 ? 4 : 1;  // rows in flight
    for (int64_t row0 = static_cast<int64_t>(blockIdx.y) * R; row0 < p.T;
         row0 += static_cast<int64_t>(gridDim.y) * R) {
        float d[R][E], h[R][E], r[R][E], rstd[R], c[R];
#pragma unroll
        for (int q = 0; q < R; ++q) {  // (rows past the end: the last one again)
            const int64_t row = min(row0 + q, p.T - 1);
            rstd[q] = p.rstd[row];
            c[q] = p.dot[row];
            load_e<DT, E>(p.dy + row * p.dy_ld, i, d[q]);
            load_e<DT, E>(p.x + row * p.x_ld, i, h[q]);
#pragma unroll
            for (int j = 0; j < E; ++j) r[q][j] = 0.f;
            if (p.dres) load_e<DT, E>(p.dres + row * p.dres_ld, i, r[q]);
        }
#pragma unroll
        for (int q = 0; q < R; ++q) {
            if (row0 + q < p.T) {
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    h[q][j] *= rstd[q];
                    dw[j] = fmaf(d[q][j], h[q][j], dw[j]);
                    r[q][j] = fmaf(rstd[q], d[q][j] * w[j] - h[q][j] * c[q], r[q][j]);
                }
                store_e<DT, E>(p.dx + (row0 + q) * p.dx_ld, i, r[q]);
            }
        }
    }
    if (p.part) store_part<E>(p.part + static_cast<int64_t>(blockIdx.y) * p.H, i, dw);
}

// ------------------------------------------------------------ host side
constexpr int64_t kMaxH = INT64_C(1) << 30;  // columns and the kernels' strides over them fit 32 bits
// CTAs whose partial dw the workspace holds (SMs x CTAs of one SM).
int64_t max_parts(int64_t T, int64_t H) {
    const int64_t n = 160 * std::min<int64_t>(8, std::max<int64_t>(2, 16384 / H));
    return std::min(std::max<int64_t>(T, 1), n);
}
// CTAs of `threads` threads on one SM, for about 1024 threads.
int per_sm_of(int threads) { return std::max(1, std::min(8, 1024 / threads)); }

// Dynamic shared memory of the ring kernels with `threads` threads.
size_t fwd_ring_smem(int ahead, int threads) {
    return static_cast<size_t>(ahead) * 2 * kOwn * 16 * threads;
}
size_t bwd_ring_smem(bool multi, int threads) {
    return static_cast<size_t>(kBwdAhead * 3 + multi) * kOwn * 16 * threads;
}

// Opt a kernel in to the most dynamic shared memory it is ever launched with, once
// per device.  The limit belongs to the function, not to a launch: set to each
// launch's own size, it could fall below what another thread, or a node of a captured
// graph, is about to launch with.
template <class Params>
cudaError_t opt_in(void (*k)(Params), size_t most, int device) {
    static std::mutex mu;
    static std::set<std::pair<int, void (*)(Params)>> done;
    std::lock_guard<std::mutex> lock(mu);
    if (done.count({device, k})) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(most));
    if (e == cudaSuccess) done.insert({device, k});
    return e;
}

// All kernels are launched dependent on what precedes them on the stream.
template <class Params>
cudaError_t launch(void (*k)(Params), dim3 grid, int threads, size_t smem, cudaStream_t s,
                   const Params &p) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, p);
}

int elt_of(int32_t dtype) { return dtype == VLMCE_F32 ? 4 : 2; }
bool dtype_ok(int32_t d) { return d == VLMCE_F32 || d == VLMCE_BF16 || d == VLMCE_F16; }

// Registers hold ng granules of E elements per thread with `threads` threads;
// ng = 0: the row is too wide.
struct Shape {
    int ng, threads;
};
Shape shape_of(int64_t H, int E) {
    const int64_t granules = (H + E - 1) / E;
    const int sizes[3] = {E == 1 ? 4 : 1, E == 1 ? 8 : 2, E == 1 ? 16 : 4};
    const int most[3] = {256, 512, 1024};
    for (int k = 0; k < 3; ++k)
        if (granules <= static_cast<int64_t>(sizes[k]) * most[k])
            return {sizes[k],
                    static_cast<int>(round_up((granules + sizes[k] - 1) / sizes[k], 32))};
    return {0, 512};
}

using FwdKernel = void (*)(const FwdParams);
template <int DT, bool Q>
FwdKernel fwd_pick(bool vec, int ng) {
    constexpr int E = Elt<DT>::kPer16;
    if (vec) {
        switch (ng) {
            case 1: return fwd_kernel<DT, E, 1, Q>;
            case 2: return fwd_kernel<DT, E, 2, Q>;
            case 4: return fwd_kernel<DT, E, 4, Q>;
            default: return fwd_kernel<DT, E, 0, Q>;
        }
    }
    switch (ng) {
        case 4: return fwd_kernel<DT, 1, 4, Q>;
        case 8: return fwd_kernel<DT, 1, 8, Q>;
        case 16: return fwd_kernel<DT, 1, 16, Q>;
        default: return fwd_kernel<DT, 1, 0, Q>;
    }
}
FwdKernel fwd_kernel_of(int32_t dtype, bool quant, bool vec, int ng) {
    switch (dtype) {
        case VLMCE_F32:
            return quant ? fwd_pick<VLMCE_F32, true>(vec, ng) : fwd_pick<VLMCE_F32, false>(vec, ng);
        case VLMCE_BF16:
            return quant ? fwd_pick<VLMCE_BF16, true>(vec, ng)
                         : fwd_pick<VLMCE_BF16, false>(vec, ng);
        default:
            return quant ? fwd_pick<VLMCE_F16, true>(vec, ng) : fwd_pick<VLMCE_F16, false>(vec, ng);
    }
}
// Threads of the ring kernels, kOwn granules of 16 bytes each (`shifted` rows can
// touch one more at an end); 0: the row is too wide.
int ring_threads(int64_t H, int32_t dtype, bool shifted) {
    const int64_t E = 16 / elt_of(dtype);
    const int64_t granules = shifted ? (H + 2 * E - 2) / E : H / E;
    return granules <= kOwn * kRingThreads
               ? static_cast<int>(round_up((granules + kOwn - 1) / kOwn, 32))
               : 0;
}
template <bool Q, int A, bool S>
FwdKernel fwd_ring_typed(int32_t dtype) {
    switch (dtype) {
        case VLMCE_F32: return fwd_ring_kernel<VLMCE_F32, Q, A, S>;
        case VLMCE_BF16: return fwd_ring_kernel<VLMCE_BF16, Q, A, S>;
        default: return fwd_ring_kernel<VLMCE_F16, Q, A, S>;
    }
}
template <bool S>
FwdKernel fwd_ring_of(int32_t dtype, bool quant, int ahead) {
    if (ahead == 2)
        return quant ? fwd_ring_typed<true, 2, S>(dtype) : fwd_ring_typed<false, 2, S>(dtype);
    return quant ? fwd_ring_typed<true, 3, S>(dtype) : fwd_ring_typed<false, 3, S>(dtype);
}
using BwdKernel = void (*)(const BwdParams);
template <bool MULTI, bool S>
BwdKernel bwd_ring_typed(int32_t dtype) {
    switch (dtype) {
        case VLMCE_F32: return bwd_ring_kernel<VLMCE_F32, MULTI, S>;
        case VLMCE_BF16: return bwd_ring_kernel<VLMCE_BF16, MULTI, S>;
        default: return bwd_ring_kernel<VLMCE_F16, MULTI, S>;
    }
}
BwdKernel bwd_ring_of(int32_t dtype, bool multi, bool shifted) {
    if (shifted) return multi ? bwd_ring_typed<true, true>(dtype) : bwd_ring_typed<false, true>(dtype);
    return multi ? bwd_ring_typed<true, false>(dtype) : bwd_ring_typed<false, false>(dtype);
}
template <int DT>
BwdKernel bwd_pick(bool vec, int ng) {
    constexpr int E = Elt<DT>::kPer16;
    if (vec) {
        switch (ng) {
            case 1: return bwd_kernel<DT, E, 1>;
            case 2: return bwd_kernel<DT, E, 2>;
            default: return bwd_kernel<DT, E, 4>;
        }
    }
    switch (ng) {
        case 4: return bwd_kernel<DT, 1, 4>;
        case 8: return bwd_kernel<DT, 1, 8>;
        default: return bwd_kernel<DT, 1, 16>;
    }
}
BwdKernel bwd_kernel_of(int32_t dtype, bool vec, int ng) {
    switch (dtype) {
        case VLMCE_F32: return bwd_pick<VLMCE_F32>(vec, ng);
        case VLMCE_BF16: return bwd_pick<VLMCE_BF16>(vec, ng);
        default: return bwd_pick<VLMCE_F16>(vec, ng);
    }
}
template <int DT>
void wide_pick(bool vec, BwdKernel *dot, BwdKernel *seg) {
    constexpr int E = Elt<DT>::kPer16;
    *dot = vec ? dot_kernel<DT, E> : dot_kernel<DT, 1>;
    *seg = vec ? segment_kernel<DT, E> : segment_kernel<DT, 1>;
}

// A [T, H] argument: stride in elements of elt bytes.
vlmce_status check_rows(const void *p, int64_t T, int64_t H, int64_t ld, int elt) {
    if (ld < H) return VLMCE_ERR_INVALID_ARG;
    if (ld > (INT64_MAX / 8) / elt / std::max<int64_t>(T, 1)) return VLMCE_ERR_TOO_LARGE;
    if (T > 0 && !p) return VLMCE_ERR_INVALID_ARG;
    if (!aligned(p, static_cast<uintptr_t>(elt))) return VLMCE_ERR_MISALIGNED;
    return VLMCE_OK;
}
bool overlap(const void *a, int64_t a_ld, int a_elt, const void *b, int64_t b_ld, int b_elt,
             int64_t T, int64_t H) {
    return rows_overlap({a, T, H * a_elt, a_ld * a_elt}, {b, T, H * b_elt, b_ld * b_elt});
}

}  // namespace
}  // namespace rms
}  // namespace vlmce

extern "C" vlmce_status rmsnorm_fwd(const void *x, int64_t x_stride, const void *residual,
                                    int64_t residual_stride, const void *weight,
                                    int32_t weight_dtype, int32_t dtype, int64_t T, int64_t H,
                                    float eps, float weight_offset, void *y, int64_t y_stride,
                                    int32_t y_dtype, void *residual_out,
                                    int64_t residual_out_stride, float *rstd, float *scale,
                                    vlmce_stream_t stream) {
    using namespace vlmce;
    using namespace vlmce::rms;
    if (!dtype_ok(dtype) || (weight_dtype != dtype && weight_dtype != VLMCE_F32) ||
        (y_dtype != dtype && y_dtype != VLMCE_E4M3))
        return VLMCE_ERR_UNSUPPORTED_DTYPE;
    const bool quant = y_dtype == VLMCE_E4M3;
    const int elt = elt_of(dtype), yelt = quant ? 1 : elt;
    if (T < 0 || H < 1 || !(eps >= 0.f) || !std::isfinite(eps) || !std::isfinite(weight_offset) ||
        !weight || (T > 0 && quant != (scale != nullptr)))
        return VLMCE_ERR_INVALID_ARG;
    if (H > kMaxH || T > INT32_MAX) return VLMCE_ERR_TOO_LARGE;
    vlmce_status st = check_rows(x, T, H, x_stride, elt);
    if (st == VLMCE_OK) st = check_rows(y, T, H, y_stride, yelt);
    if (st == VLMCE_OK && residual) st = check_rows(residual, T, H, residual_stride, elt);
    if (st == VLMCE_OK && residual_out)
        st = check_rows(residual_out, T, H, residual_out_stride, elt);
    if (st != VLMCE_OK) return st;
    if (!aligned(weight, weight_dtype == VLMCE_F32 ? 4 : 2) || !aligned(rstd, 4) ||
        !aligned(scale, 4))
        return VLMCE_ERR_MISALIGNED;
    auto same = [&](const void *a, int64_t a_ld, const void *b, int64_t b_ld) {
        return a == b && (a_ld == b_ld || T <= 1);
    };
    if (overlap(y, y_stride, yelt, x, x_stride, elt, T, H) ||
        overlap(y, y_stride, yelt, residual, residual_stride, elt, T, H) ||
        overlap(y, y_stride, yelt, residual_out, residual_out_stride, elt, T, H) ||
        (overlap(residual_out, residual_out_stride, elt, x, x_stride, elt, T, H) &&
         !same(residual_out, residual_out_stride, x, x_stride)) ||
        (overlap(residual_out, residual_out_stride, elt, residual, residual_stride, elt, T, H) &&
         !same(residual_out, residual_out_stride, residual, residual_stride)))
        return VLMCE_ERR_INVALID_ARG;
    if (T == 0) return VLMCE_OK;
    DeviceInfo dev;
    st = current_device(&dev);
    if (st != VLMCE_OK) return st;
    const int E = 16 / elt;
    const bool vec = H % E == 0 && x_stride % E == 0 && aligned(x, 16) && y_stride % E == 0 &&
                     aligned(y, static_cast<uintptr_t>(E * yelt)) && aligned(weight, 16) &&
                     (!residual || (residual_stride % E == 0 && aligned(residual, 16))) &&
                     (!residual_out || (residual_out_stride % E == 0 && aligned(residual_out, 16)));
    const Shape sh = shape_of(H, vec ? E : 1);
    FwdParams p = {};
    p.x = static_cast<const unsigned char *>(x);
    p.residual = static_cast<const unsigned char *>(residual);
    p.weight = weight;
    p.y = static_cast<unsigned char *>(y);
    p.sum = static_cast<unsigned char *>(residual_out);
    p.rstd = rstd;
    p.scale = scale;
    p.T = T;
    p.H = static_cast<int>(H);
    p.x_ld = x_stride * elt;
    p.residual_ld = residual_stride * elt;
    p.y_ld = y_stride * yelt;
    p.sum_ld = residual_out_stride * elt;
    p.eps = eps;
    p.offset = weight_offset;
    p.w_f32 = weight_dtype == VLMCE_F32;
    cudaStream_t st_ = reinterpret_cast<cudaStream_t>(stream);
    // rows at any alignment, the same in all arrays
    auto like_x = [&](const void *q, int64_t ld, int bytes) {
        return !q || (ld % E == x_stride % E && aligned(q, static_cast<uintptr_t>(bytes)));
    };
    const bool shifted = !vec && aligned(x, 16) && like_x(y, y_stride, E * yelt) &&
                         like_x(residual, residual_stride, 16) &&
                         like_x(residual_out, residual_out_stride, 16);
    const int rt = vec || shifted ? ring_threads(H, dtype, shifted) : 0;
    if (rt > 0) {
        const int per_sm = per_sm_of(rt);
        const int64_t ctas = static_cast<int64_t>(dev.sm_count) * per_sm / (shifted ? E : 1) *
                             (shifted ? E : 1);
        // rows ahead: long 16-bit rows fill the memory system with one row ahead
        // (8192 x 6656 bf16 to e4m3: 59 us, two rows ahead 65), others need two
        // (8192 x 1024 bf16: 11.7 against 15.7; 4096 x 4096 fp32: 45.8 against 48)
        const int ahead = elt == 2 && H >= 4096 ? 2 : 3;
        // rows enough for that; one CTA per row has the lower latency, but goes element by
        // element through shifted rows (1200 x 2001 bf16 5.2 us, the ring 4.8; 8192 x
        // 1001 19.7 and 14.8; 8192 x 701 14.5 and 15.0)
        if (ctas > 0 && (shifted ? H > 768 && 2 * T >= ctas : T >= 3 * ctas)) {
            const FwdKernel k = shifted ? fwd_ring_of<true>(dtype, quant, ahead)
                                        : fwd_ring_of<false>(dtype, quant, ahead);
            cudaError_t e = opt_in(k, fwd_ring_smem(ahead, kRingThreads), dev.device);
            if (e == cudaSuccess)
                e = launch(k, dim3(static_cast<unsigned>(ctas), 1, 1), rt,
                           fwd_ring_smem(ahead, rt), st_, p);
            return launch_status(e, "rmsnorm_fwd");
        }
    }
    return launch_status(launch(fwd_kernel_of(dtype, quant, vec, sh.ng),
                                dim3(static_cast<unsigned>(T), 1, 1), sh.threads, 0, st_, p),
                         "rmsnorm_fwd");
}

extern "C" size_t vlmce_rmsnorm_bwd_workspace_bytes(int64_t T, int64_t H) {
    using namespace vlmce;
    using namespace vlmce::rms;
    if (T < 0 || H < 1 || H > kMaxH || T > INT32_MAX) return 0;
    return static_cast<size_t>(round_up(4 * H * max_parts(T, H), 256) + round_up(4 * T, 256));
}

extern "C" vlmce_status rmsnorm_bwd(const void *dy, int64_t dy_stride, const void *x,
                                    int64_t x_stride, const void *weight, int32_t weight_dtype,
                                    const float *rstd, const void *dresidual,
                                    int64_t dresidual_stride, int32_t dtype, int64_t T, int64_t H,
                                    float weight_offset, void *dx, int64_t dx_stride,
                                    float *dweight, int32_t accumulate_dweight, void *workspace,
                                    size_t workspace_bytes, vlmce_stream_t stream) {
    using namespace vlmce;
    using namespace vlmce::rms;
    if (!dtype_ok(dtype) || (weight_dtype != dtype && weight_dtype != VLMCE_F32))
        return VLMCE_ERR_UNSUPPORTED_DTYPE;
    const int elt = elt_of(dtype);
    if (T < 0 || H < 1 || !std::isfinite(weight_offset) || !weight || (T > 0 && !rstd))
        return VLMCE_ERR_INVALID_ARG;
    if (H > kMaxH || T > INT32_MAX) return VLMCE_ERR_TOO_LARGE;
    vlmce_status st = check_rows(dy, T, H, dy_stride, elt);
    if (st == VLMCE_OK) st = check_rows(x, T, H, x_stride, elt);
    if (st == VLMCE_OK) st = check_rows(dx, T, H, dx_stride, elt);
    if (st == VLMCE_OK && dresidual) st = check_rows(dresidual, T, H, dresidual_stride, elt);
    if (st != VLMCE_OK) return st;
    if (!aligned(weight, weight_dtype == VLMCE_F32 ? 4 : 2) || !aligned(rstd, 4) ||
        !aligned(dweight, 4))
        return VLMCE_ERR_MISALIGNED;
    auto clash = [&](const void *b, int64_t b_ld) {
        return overlap(dx, dx_stride, elt, b, b_ld, elt, T, H) &&
               !(dx == b && (dx_stride == b_ld || T <= 1));
    };
    if (overlap(dx, dx_stride, elt, x, x_stride, elt, T, H) || clash(dy, dy_stride) ||
        clash(dresidual, dresidual_stride))
        return VLMCE_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < vlmce_rmsnorm_bwd_workspace_bytes(T, H))
        return VLMCE_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned(workspace, 256)) return VLMCE_ERR_MISALIGNED;
    DeviceInfo dev;
    st = current_device(&dev);
    if (st != VLMCE_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0) {
        cudaError_t e = cudaSuccess;
        if (dweight && !accumulate_dweight)
            e = cudaMemsetAsync(dweight, 0, static_cast<size_t>(4 * H), s);
        return launch_status(e, "rmsnorm_bwd");
    }
    const int E = 16 / elt;
    const bool vec = H % E == 0 && x_stride % E == 0 && aligned(x, 16) && dy_stride % E == 0 &&
                     aligned(dy, 16) && dx_stride % E == 0 && aligned(dx, 16) &&
                     aligned(weight, 16) &&
                     (!dresidual || (dresidual_stride % E == 0 && aligned(dresidual, 16)));
    const Shape sh = shape_of(H, vec ? E : 1);
    const int64_t parts_max = max_parts(T, H);
    BwdParams p = {};
    p.dy = static_cast<const unsigned char *>(dy);
    p.x = static_cast<const unsigned char *>(x);
    p.dres = static_cast<const unsigned char *>(dresidual);
    p.weight = weight;
    p.rstd = rstd;
    p.dx = static_cast<unsigned char *>(dx);
    p.part = dweight ? static_cast<float *>(workspace) : nullptr;
    p.dot = reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) +
                                      round_up(4 * H * parts_max, 256));
    p.T = T;
    p.H = static_cast<int>(H);
    p.dy_ld = dy_stride * elt;
    p.x_ld = x_stride * elt;
    p.dres_ld = dresidual_stride * elt;
    p.dx_ld = dx_stride * elt;
    p.offset = weight_offset;
    p.w_f32 = weight_dtype == VLMCE_F32;
    int64_t parts;
    auto like_x = [&](const void *q, int64_t ld) {
        return !q || (ld % E == x_stride % E && aligned(q, 16));
    };
    const bool shifted = !vec && aligned(x, 16) && like_x(dy, dy_stride) && like_x(dx, dx_stride) &&
                         like_x(dresidual, dresidual_stride);
    const int rt = vec || shifted ? ring_threads(H, dtype, shifted) : 0;
    // rows of up to 128 threads share a CTA, two CTAs per SM; longer ones have their
    // own, 1024 threads per SM
    p.groups = rt > 0 && rt <= 128 ? std::min(15, kRingThreads / rt) : 1;
    const int64_t full = static_cast<int64_t>(dev.sm_count) * (rt > 128 ? per_sm_of(rt) : 2);
    const int64_t unit = shifted ? E : 1;
    const int64_t ring_ctas =
        std::min(full, (T + p.groups - 1) / p.groups) / unit * unit;
    // Rows enough to run ahead (us, the ring and bwd_kernel).  Rows that share a CTA
    // leave fewer partial rows, so theirs may be fewer: 1200 x 1024 bf16 8.2 and 9.3,
    // 600 x 1024 7.5 and 6.0; longer ones 600 x 6656 10.4 and 11.2, 300 x 6656 7.7 and
    // 8.0, 1200 x 2048 8.9 and 7.8; shifted 8192 x 1001 26 and 49, 1200 x 1001 12.5
    // and 8.6.
    const int64_t needed = rt <= 64 && !shifted ? full * p.groups / 4 : full * p.groups;
    cudaError_t e;
    if (rt > 0 && ring_ctas > 0 && T >= needed && ring_ctas <= parts_max) {
        parts = ring_ctas;
        const int threads = p.groups * rt;
        const bool multi = p.groups > 1;
        const BwdKernel k = bwd_ring_of(dtype, multi, shifted);
        e = opt_in(k, bwd_ring_smem(multi, kRingThreads), dev.device);
        if (e == cudaSuccess)
            e = launch(k, dim3(static_cast<unsigned>(parts), 1, 1), threads,
                       bwd_ring_smem(multi, threads), s, p);
    } else if (sh.ng > 0 && sh.ng < 16) {
        parts = std::min<int64_t>(parts_max, static_cast<int64_t>(dev.sm_count) *
                                                 std::max(2, per_sm_of(sh.threads)));
        e = launch(bwd_kernel_of(dtype, vec, sh.ng), dim3(static_cast<unsigned>(parts), 1, 1),
                   sh.threads, 0, s, p);
    } else {
        BwdKernel dot, seg;
        if (dtype == VLMCE_F32)
            wide_pick<VLMCE_F32>(vec, &dot, &seg);
        else if (dtype == VLMCE_BF16)
            wide_pick<VLMCE_BF16>(vec, &dot, &seg);
        else
            wide_pick<VLMCE_F16>(vec, &dot, &seg);
        e = launch(dot, dim3(static_cast<unsigned>(T), 1, 1), 512, 0, s, p);
        st = launch_status(e, "rmsnorm_bwd");
        if (st != VLMCE_OK) return st;
        const int64_t per = 512 * (vec ? E : 1);
        const int64_t gx = (H + per - 1) / per;
        parts = std::min<int64_t>(parts_max,
                                  std::max<int64_t>(1, static_cast<int64_t>(dev.sm_count) * 4 / gx));
        e = launch(seg, dim3(static_cast<unsigned>(gx), static_cast<unsigned>(parts), 1), 512, 0, s,
                   p);
    }
    st = launch_status(e, "rmsnorm_bwd");
    if (st != VLMCE_OK || !dweight) return st;
    const colsum::Params d = {p.part, dweight, H, static_cast<int>(parts), accumulate_dweight};
    return launch_status(launch(colsum::kernel<colsum::kWarps>, dim3(colsum::blocks(H), 1, 1),
                                32 * colsum::kWarps, 0, s, d),
                         "rmsnorm_bwd");
}
