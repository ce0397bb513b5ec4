// linear.cu -- entry points of the linear layer (bias, activation, residual in
// the product's epilogue) and of the gated layer (both projections, activation
// and product in one kernel), forward and backward.
//
// Backward, with dz the gradient of the pre-activations:
//   linear   dz = dy act'(z)
//   gated    dz = (dy u act'(g) | dy act(g))
//   dx = dz W,  dW = dz^T x,  db = sum_t dz
// dz is formed in fp32 by one elementwise pass and rounded once to the
// operands' 16-bit type, which the tensor cores need (its range too: fp16 ends at
// 65504); db is summed from the fp32 values.  The two products run as one launch of
// the pair kernel, or dx on the small kernel and dW after it (mm.cu).
// Without an activation dz is dy itself and the pass is left out (unless dy's
// rows are not 16-byte aligned, or db is wanted, which reads dy only).
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>

#include "act.cuh"
#include "colsum.cuh"
#include "host_util.h"
#include "mm_types.h"
#include "rows_host.h"
#include "vlmce.h"

namespace vlmce {
namespace linear {
namespace {

// ------------------------------------------------------------ dz and db
constexpr int kDzWarps = 8;
constexpr int kMaxRowChunks = 64;  // partial sums of db

struct DzParams {
    const uint16_t *dy, *pre;
    uint16_t *dz;   // may be null (db only)
    float *part;    // [row chunks][N] partial sums of dz's columns, may be null
    int64_t dy_ld, pre_ld, dz_ld;
    int64_t T, N;
    int64_t rows_per_chunk;
    int f16;
};

template <int V>
__device__ __forceinline__ void load_v(const uint16_t *p, float (&v)[V], bool f16) {
    if constexpr (V == 8) {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        act::unpack16x2(u.x, v[0], v[1], f16);
        act::unpack16x2(u.y, v[2], v[3], f16);
        act::unpack16x2(u.z, v[4], v[5], f16);
        act::unpack16x2(u.w, v[6], v[7], f16);
    } else {
        v[0] = act::from16(*p, f16);
    }
}
template <int V>
__device__ __forceinline__ void store_v(uint16_t *p, const float (&v)[V], bool f16) {
    if constexpr (V == 8)
        *reinterpret_cast<uint4 *>(p) =
            make_uint4(act::pack16x2(v[0], v[1], f16), act::pack16x2(v[2], v[3], f16),
                       act::pack16x2(v[4], v[5], f16), act::pack16x2(v[6], v[7], f16));
    else
        *p = act::to16(v[0], f16);
}

// One warp: 32 V consecutive columns of a row; a block's 8 warps take every
// 8th row of its chunk, element by element several rows at once.  HBM-bound: T = 4096,
// n = 16384 gated bf16 99 us = 6.8 TB/s.
template <int ACT, bool GATED, int V>
__global__ void __launch_bounds__(32 * kDzWarps) dz_kernel(const DzParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int64_t col = (static_cast<int64_t>(blockIdx.x) * 32 + lane) * V;
    const int64_t r0 = blockIdx.y * p.rows_per_chunk;
    const int64_t r1 = min(p.T, r0 + p.rows_per_chunk);
    const bool f16 = p.f16 != 0;
    float sum[V];
#pragma unroll
    for (int j = 0; j < V; ++j) sum[j] = 0.f;
    if (col < p.N) {
        constexpr int R = V == 1 ? 4 : 1;  // rows in flight
        for (int64_t first = r0 + warp; first < r1; first += kDzWarps * R) {
            float d[R][V], g[R][V], u[R][V];
#pragma unroll
            for (int q = 0; q < R; ++q) {  // (past the end: the last row again)
                const int64_t r = R == 1 ? first : min(first + q * kDzWarps, r1 - 1);
                load_v<V>(p.dy + r * p.dy_ld + col, d[q], f16);
                if constexpr (ACT != VLMCE_ACT_NONE)
                    load_v<V>(p.pre + r * p.pre_ld + col, g[q], f16);
                if constexpr (GATED) load_v<V>(p.pre + r * p.pre_ld + p.N + col, u[q], f16);
            }
#pragma unroll
            for (int q = 0; q < R; ++q) {
                const int64_t r = first + q * kDzWarps;
                if (R > 1 && r >= r1) break;
                if constexpr (ACT != VLMCE_ACT_NONE) {
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        float f, df;
                        act::fwd_bwd<ACT>(g[q][j], f, df);
                        if constexpr (GATED) {
                            g[q][j] = d[q][j] * f;
                            d[q][j] *= u[q][j] * df;
                        } else {
                            d[q][j] *= df;
                        }
                    }
                }
                if constexpr (GATED) {
                    store_v<V>(p.dz + r * p.dz_ld + col, d[q], f16);
                    store_v<V>(p.dz + r * p.dz_ld + p.N + col, g[q], f16);
                } else {
                    if (p.dz) store_v<V>(p.dz + r * p.dz_ld + col, d[q], f16);
#pragma unroll
                    for (int j = 0; j < V; ++j) sum[j] += d[q][j];
                }
            }
        }
    }
    if constexpr (!GATED) {
        if (p.part) {
            __shared__ float s[kDzWarps][32 * V];
#pragma unroll
            for (int j = 0; j < V; ++j) s[warp][lane * V + j] = sum[j];
            __syncthreads();
            for (int c = threadIdx.x; c < 32 * V; c += 32 * kDzWarps) {
                const int64_t n = static_cast<int64_t>(blockIdx.x) * 32 * V + c;
                if (n >= p.N) continue;
                float a = 0.f;
#pragma unroll
                for (int w = 0; w < kDzWarps; ++w) a += s[w][c];
                p.part[blockIdx.y * p.N + n] = a;
            }
        }
    }
}

using DzKernel = void (*)(const DzParams);
template <int ACT>
DzKernel dz_pick(bool gated, bool vec) {
    if constexpr (ACT != VLMCE_ACT_NONE)
        if (gated) return vec ? dz_kernel<ACT, true, 8> : dz_kernel<ACT, true, 1>;
    return vec ? dz_kernel<ACT, false, 8> : dz_kernel<ACT, false, 1>;
}
DzKernel dz_kernel_of(int act, bool gated, bool vec) {
    switch (act) {
        case VLMCE_ACT_SILU: return dz_pick<VLMCE_ACT_SILU>(gated, vec);
        case VLMCE_ACT_GELU: return dz_pick<VLMCE_ACT_GELU>(gated, vec);
        case VLMCE_ACT_GELU_TANH: return dz_pick<VLMCE_ACT_GELU_TANH>(gated, vec);
        case VLMCE_ACT_RELU: return dz_pick<VLMCE_ACT_RELU>(gated, vec);
        default: return dz_pick<VLMCE_ACT_NONE>(gated, vec);
    }
}

// A launch dependent on what precedes it on the stream.
template <class... Params, class... Args>
cudaError_t launch(void (*k)(Params...), dim3 grid, int threads, cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, args...);
}

// ------------------------------------------------------------ checks
constexpr int64_t kMaxDim = INT32_MAX - 1024;

struct Buf {
    const void *p;
    int64_t rows, cols, ld;
    int elt;
    RowsOf bytes() const { return {p, rows, cols * elt, ld * elt}; }
};
bool overlap(const Buf &a, const Buf &b) { return rows_overlap(a.bytes(), b.bytes()); }
bool same(const Buf &a, const Buf &b) { return a.p == b.p && (a.ld == b.ld || a.rows <= 1); }
// rows * ld elements are addressable
bool fits(int64_t rows, int64_t ld, int elt) {
    return ld <= (INT64_MAX / 8) / elt && (rows < 1 || ld <= (INT64_MAX / 8) / elt / rows);
}
bool act_ok(int32_t act, bool gated) {
    return act >= (gated ? VLMCE_ACT_SILU : VLMCE_ACT_NONE) && act <= VLMCE_ACT_RELU;
}
// An operand of the tensor cores: [rows, K] K-major.
vlmce_status check_operand(const void *p, int64_t rows, int64_t K, int64_t ld, int elt) {
    if (ld < K || ld * elt % 16 != 0) return VLMCE_ERR_INVALID_ARG;
    if (!fits(rows, ld, elt) || ld * elt >= (int64_t(1) << 40)) return VLMCE_ERR_TOO_LARGE;
    if (rows > 0 && !p) return VLMCE_ERR_INVALID_ARG;
    if (!aligned(p, 16)) return VLMCE_ERR_MISALIGNED;
    return VLMCE_OK;
}
vlmce_status check16(const void *p, int64_t rows, int64_t cols, int64_t ld) {
    if (ld < cols) return VLMCE_ERR_INVALID_ARG;
    if (!fits(rows, ld, 2)) return VLMCE_ERR_TOO_LARGE;
    if (!aligned(p, 2)) return VLMCE_ERR_MISALIGNED;
    return VLMCE_OK;
}

struct FwdArgs {
    const void *x;
    int64_t x_stride;
    const float *x_scale;
    const void *weight;
    int64_t weight_stride;
    const float *weight_scale;
    int32_t dtype, out_dtype;
    const void *bias, *residual;
    int64_t residual_stride;
    int64_t T, N, K;
    int32_t act;
    void *y;
    int64_t y_stride;
    void *preact;
    int64_t preact_stride;
    int32_t *dev_err;
    bool gated;
    cudaStream_t stream;
};

// the products' tiles are numbered in 32 bits
bool fwd_sizes_ok(int64_t T, int64_t N, int64_t K) {
    return T <= kMaxDim && N <= kMaxDim / 2 && K <= kMaxDim &&
           T / 256 + 1 <= INT32_MAX / 16 / (N / 128 + 1);
}

vlmce_status forward(const FwdArgs &a, const char *where) {
    const bool fp8 = a.dtype == VLMCE_E4M3;
    if (!fp8 && a.dtype != VLMCE_BF16 && a.dtype != VLMCE_F16) return VLMCE_ERR_UNSUPPORTED_DTYPE;
    if (a.out_dtype != VLMCE_BF16 && a.out_dtype != VLMCE_F16) return VLMCE_ERR_UNSUPPORTED_DTYPE;
    if (!fp8 && a.out_dtype != a.dtype) return VLMCE_ERR_UNSUPPORTED_DTYPE;
    const int elt = fp8 ? 1 : 2;
    if (a.T < 0 || a.N < 1 || a.K < 1 || a.K * elt % 16 != 0 || !act_ok(a.act, a.gated))
        return VLMCE_ERR_INVALID_ARG;
    if (!fwd_sizes_ok(a.T, a.N, a.K)) return VLMCE_ERR_TOO_LARGE;
    const int64_t rows = a.gated ? 2 * a.N : a.N;
    vlmce_status st = check_operand(a.x, a.T, a.K, a.x_stride, elt);
    if (st == VLMCE_OK) st = check_operand(a.weight, rows, a.K, a.weight_stride, elt);
    if (st != VLMCE_OK) return st;
    if (fp8 ? !a.weight_scale || (a.T > 0 && !a.x_scale) : a.x_scale || a.weight_scale)
        return VLMCE_ERR_INVALID_ARG;
    if (a.T > 0 && !a.y) return VLMCE_ERR_INVALID_ARG;
    st = check16(a.y, a.T, a.N, a.y_stride);
    if (st == VLMCE_OK && a.preact) st = check16(a.preact, a.T, rows, a.preact_stride);
    if (st == VLMCE_OK && a.residual) st = check16(a.residual, a.T, a.N, a.residual_stride);
    if (st != VLMCE_OK) return st;
    if (!aligned(a.bias, 2) || !aligned(a.x_scale, 4) || !aligned(a.weight_scale, 4) ||
        !aligned(a.dev_err, 4))
        return VLMCE_ERR_MISALIGNED;
    const Buf y{a.y, a.T, a.N, a.y_stride, 2}, z{a.preact, a.T, rows, a.preact_stride, 2},
        x{a.x, a.T, a.K, a.x_stride, elt}, w{a.weight, rows, a.K, a.weight_stride, elt},
        r{a.residual, a.T, a.N, a.residual_stride, 2};
    if (overlap(y, x) || overlap(y, w) || overlap(y, z) || overlap(z, x) || overlap(z, w) ||
        overlap(z, r) || (overlap(y, r) && !same(y, r)))
        return VLMCE_ERR_INVALID_ARG;
    if (a.T == 0) return VLMCE_OK;
    DeviceInfo dev;
    st = current_device(&dev);
    if (st != VLMCE_OK) return st;

    mm::Fwd f = {};
    f.x = a.x;
    f.w = a.weight;
    f.x_ld = a.x_stride;
    f.w_ld = a.weight_stride;
    f.T = a.T;
    f.N = a.N;
    f.K = a.K;
    f.gated = a.gated;
    f.dtype = a.dtype;
    f.err = a.dev_err;
    mm::Epi &e = f.e;
    e.y = static_cast<uint16_t *>(a.y);
    e.y_ld = a.y_stride;
    e.preact = static_cast<uint16_t *>(a.preact);
    e.preact_ld = a.preact_stride;
    e.bias = static_cast<const uint16_t *>(a.bias);
    e.residual = static_cast<const uint16_t *>(a.residual);
    e.residual_ld = a.residual_stride;
    e.xs = a.x_scale;
    e.ws = a.weight_scale;
    e.act = a.act;
    e.f16 = a.out_dtype == VLMCE_F16;
    e.y_vec = mm::vec_of(a.y, a.y_stride, a.N);
    if (e.preact) {
        e.preact_vec = mm::vec_of(e.preact, a.preact_stride, a.N);
        e.preact_up_vec = mm::vec_of(e.preact + a.N, a.preact_stride, a.N);
    }
    return launch_status(mm::forward(f, a.stream), where);
}

// ------------------------------------------------------------ backward
struct BwdArgs {
    const void *dy;
    int64_t dy_stride;
    const void *x;
    int64_t x_stride;
    const void *weight;
    int64_t weight_stride;
    const void *preact;
    int64_t preact_stride;
    int32_t dtype;
    int64_t T, N, K;
    int32_t act;
    void *dx;
    int64_t dx_stride;
    void *dweight;
    int32_t dweight_dtype;
    float *dbias;
    int32_t accumulate;
    int32_t *dev_err;
    void *workspace;
    size_t workspace_bytes;
    bool gated;
    cudaStream_t stream;
};

int64_t dz_ld_of(int64_t rows) { return round_up(rows, 8); }
int64_t part_bytes(int64_t N) { return round_up(4 * kMaxRowChunks * N, 256); }
bool bwd_sizes_ok(int64_t T, int64_t N, int64_t K) {
    return T >= 0 && N >= 1 && K >= 1 && T <= kMaxDim && N <= kMaxDim / 2 && K <= kMaxDim &&
           (T / 256 + 1 + N / 128 + 1) <= INT32_MAX / 32 / (K / 256 + 1);
}
// dz [T, rows rounded to 8] and, for a linear layer, the partial sums of db.
size_t bwd_workspace(int64_t T, int64_t N, int64_t K, bool gated) {
    if (!bwd_sizes_ok(T, N, K)) return 0;
    const int64_t ld = dz_ld_of(gated ? 2 * N : N);
    return static_cast<size_t>(round_up(2 * T * ld, 256) + (gated ? 0 : part_bytes(N)));
}

vlmce_status backward(const BwdArgs &a, const char *where) {
    if (a.dtype != VLMCE_BF16 && a.dtype != VLMCE_F16) return VLMCE_ERR_UNSUPPORTED_DTYPE;
    if (a.dweight && a.dweight_dtype != VLMCE_F32 && a.dweight_dtype != a.dtype)
        return VLMCE_ERR_UNSUPPORTED_DTYPE;
    if (a.T < 0 || a.N < 1 || a.K < 1 || a.K % 8 != 0 || !act_ok(a.act, a.gated))
        return VLMCE_ERR_INVALID_ARG;
    if (!bwd_sizes_ok(a.T, a.N, a.K)) return VLMCE_ERR_TOO_LARGE;
    const int64_t rows = a.gated ? 2 * a.N : a.N;
    const bool need_pre = a.act != VLMCE_ACT_NONE;
    if (!a.dx && !a.dweight && !a.dbias && a.T > 0) return VLMCE_ERR_INVALID_ARG;
    if (a.accumulate && a.dweight && a.dweight_dtype != VLMCE_F32) return VLMCE_ERR_INVALID_ARG;
    vlmce_status st = VLMCE_OK;
    if (a.dweight) st = check_operand(a.x, a.T, a.K, a.x_stride, 2);
    if (st == VLMCE_OK && a.dx) st = check_operand(a.weight, rows, a.K, a.weight_stride, 2);
    if (st != VLMCE_OK) return st;
    if (a.T > 0 && (!a.dy || (need_pre && !a.preact))) return VLMCE_ERR_INVALID_ARG;
    st = check16(a.dy, a.T, a.N, a.dy_stride);
    if (st == VLMCE_OK && need_pre) st = check16(a.preact, a.T, rows, a.preact_stride);
    if (st == VLMCE_OK && a.dx) st = check16(a.dx, a.T, a.K, a.dx_stride);
    if (st != VLMCE_OK) return st;
    if ((a.dx && (!aligned(a.dx, 16) || a.dx_stride % 8 != 0)) || !aligned(a.dweight, 16) ||
        !aligned(a.dbias, 4) || !aligned(a.dev_err, 4))
        return VLMCE_ERR_MISALIGNED;
    const Buf dy{a.dy, a.T, a.N, a.dy_stride, 2},
        z{need_pre ? a.preact : nullptr, a.T, rows, a.preact_stride, 2},
        x{a.dweight ? a.x : nullptr, a.T, a.K, a.x_stride, 2},
        w{a.dx ? a.weight : nullptr, rows, a.K, a.weight_stride, 2},
        dx{a.dx, a.T, a.K, a.dx_stride, 2},
        dw{a.dweight, rows, a.K, a.K, a.dweight_dtype == VLMCE_F32 ? 4 : 2};
    if (overlap(dx, dy) || overlap(dx, z) || overlap(dx, x) || overlap(dx, w) || overlap(dx, dw) ||
        overlap(dw, dy) || overlap(dw, z) || overlap(dw, x) || overlap(dw, w))
        return VLMCE_ERR_INVALID_ARG;
    // without an activation dz is dy, where the tensor cores can read its rows
    const bool as_is = !need_pre && a.dy_stride % 8 == 0 && aligned(a.dy, 16) &&
                       a.dy_stride * 2 < (int64_t(1) << 40);
    const bool products = a.dx || a.dweight;
    if (a.workspace ? a.workspace_bytes < bwd_workspace(a.T, a.N, a.K, a.gated)
                    : a.dbias || (products && !as_is))
        return VLMCE_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned(a.workspace, 256)) return VLMCE_ERR_MISALIGNED;
    DeviceInfo dev;
    st = current_device(&dev);
    if (st != VLMCE_OK) return st;
    cudaError_t e = cudaSuccess;
    if (a.T == 0) {
        if (!a.accumulate && a.dweight)
            e = cudaMemsetAsync(a.dweight, 0, static_cast<size_t>(rows * a.K * dw.elt), a.stream);
        if (e == cudaSuccess && !a.accumulate && a.dbias)
            e = cudaMemsetAsync(a.dbias, 0, static_cast<size_t>(4 * a.N), a.stream);
        return launch_status(e, where);
    }

    unsigned char *ws = static_cast<unsigned char *>(a.workspace);
    uint16_t *dz = reinterpret_cast<uint16_t *>(ws);
    int64_t dz_ld = dz_ld_of(rows);
    float *part = reinterpret_cast<float *>(ws + round_up(2 * a.T * dz_ld, 256));
    if (a.dbias || (products && !as_is)) {
        DzParams p = {};
        p.dy = static_cast<const uint16_t *>(a.dy);
        p.pre = static_cast<const uint16_t *>(a.preact);
        p.dz = products && !as_is ? dz : nullptr;
        p.part = a.dbias ? part : nullptr;
        p.dy_ld = a.dy_stride;
        p.pre_ld = a.preact_stride;
        p.dz_ld = dz_ld;
        p.T = a.T;
        p.N = a.N;
        p.f16 = a.dtype == VLMCE_F16;
        const bool vec = a.N % 8 == 0 && a.dy_stride % 8 == 0 && aligned(a.dy, 16) &&
                         (!need_pre || (a.preact_stride % 8 == 0 && aligned(a.preact, 16)));
        const int64_t per_block = 32 * (vec ? 8 : 1);
        const int64_t gx = (a.N + per_block - 1) / per_block;
        int64_t chunks = (static_cast<int64_t>(dev.sm_count) * 16 + gx - 1) / gx;
        chunks = std::min({chunks, (a.T + kDzWarps - 1) / kDzWarps, int64_t(kMaxRowChunks)});
        p.rows_per_chunk = (a.T + chunks - 1) / chunks;
        chunks = (a.T + p.rows_per_chunk - 1) / p.rows_per_chunk;
        st = launch_status(launch(dz_kernel_of(a.act, a.gated, vec),
                                  dim3(static_cast<unsigned>(gx), static_cast<unsigned>(chunks), 1),
                                  32 * kDzWarps, a.stream, static_cast<const DzParams>(p)),
                           where);
        if (st != VLMCE_OK) return st;
        if (a.dbias) {
            const colsum::Params d = {part, a.dbias, a.N, static_cast<int>(chunks), a.accumulate};
            st = launch_status(launch(colsum::kernel<colsum::kWarps>,
                                      dim3(colsum::blocks(a.N), 1, 1), 32 * colsum::kWarps,
                                      a.stream, d),
                               where);
            if (st != VLMCE_OK) return st;
        }
    }
    if (!products) return VLMCE_OK;
    const uint16_t *g = dz;
    if (as_is) {
        g = static_cast<const uint16_t *>(a.dy);
        dz_ld = a.dy_stride;
    }
    mm::Bwd b = {};
    b.dz = g;
    b.x = a.x;
    b.w = a.weight;
    b.dz_ld = dz_ld;
    b.x_ld = a.x_stride;
    b.w_ld = a.weight_stride;
    b.T = a.T;
    b.rows = rows;
    b.K = a.K;
    b.f16 = a.dtype == VLMCE_F16;
    b.dx = a.dx;
    b.dx_ld = a.dx_stride;
    b.dw = a.dweight;
    b.dw_f32 = a.dweight_dtype == VLMCE_F32;
    b.accumulate = a.accumulate;
    b.err = a.dev_err;
    return launch_status(mm::backward(b, a.stream), where);
}

}  // namespace
}  // namespace linear
}  // namespace vlmce

extern "C" vlmce_status linear_fwd(const void *x, int64_t x_stride, const float *x_scale,
                                   const void *weight, int64_t weight_stride,
                                   const float *weight_scale, int32_t dtype, const void *bias,
                                   const void *residual, int64_t residual_stride,
                                   int32_t out_dtype, int64_t T, int64_t N, int64_t K, int32_t act,
                                   void *y, int64_t y_stride, void *preact, int64_t preact_stride,
                                   int32_t *dev_err, vlmce_stream_t stream) {
    vlmce::linear::FwdArgs a = {x, x_stride, x_scale, weight, weight_stride, weight_scale, dtype,
                                out_dtype, bias, residual, residual_stride, T, N, K, act, y,
                                y_stride, preact, preact_stride, dev_err, false,
                                reinterpret_cast<cudaStream_t>(stream)};
    return vlmce::linear::forward(a, "linear_fwd");
}

extern "C" vlmce_status glu_fwd(const void *x, int64_t x_stride, const float *x_scale,
                                const void *weight, int64_t weight_stride,
                                const float *weight_scale, int32_t dtype, int32_t out_dtype,
                                int64_t T, int64_t n, int64_t K, int32_t act, void *y,
                                int64_t y_stride, void *preact, int64_t preact_stride,
                                int32_t *dev_err, vlmce_stream_t stream) {
    vlmce::linear::FwdArgs a = {x, x_stride, x_scale, weight, weight_stride, weight_scale, dtype,
                                out_dtype, nullptr, nullptr, n, T, n, K, act, y, y_stride, preact,
                                preact_stride, dev_err, true,
                                reinterpret_cast<cudaStream_t>(stream)};
    return vlmce::linear::forward(a, "glu_fwd");
}

extern "C" size_t vlmce_linear_bwd_workspace_bytes(int64_t T, int64_t N, int64_t K) {
    return vlmce::linear::bwd_workspace(T, N, K, false);
}
extern "C" size_t vlmce_glu_bwd_workspace_bytes(int64_t T, int64_t n, int64_t K) {
    return vlmce::linear::bwd_workspace(T, n, K, true);
}

extern "C" vlmce_status linear_bwd(const void *dy, int64_t dy_stride, const void *x,
                                   int64_t x_stride, const void *weight, int64_t weight_stride,
                                   const void *preact, int64_t preact_stride, int32_t dtype,
                                   int64_t T, int64_t N, int64_t K, int32_t act, void *dx,
                                   int64_t dx_stride, void *dweight, int32_t dweight_dtype,
                                   float *dbias, int32_t accumulate, int32_t *dev_err,
                                   void *workspace, size_t workspace_bytes,
                                   vlmce_stream_t stream) {
    vlmce::linear::BwdArgs a = {dy, dy_stride, x, x_stride, weight, weight_stride, preact,
                                preact_stride, dtype, T, N, K, act, dx, dx_stride, dweight,
                                dweight_dtype, dbias, accumulate, dev_err, workspace,
                                workspace_bytes, false, reinterpret_cast<cudaStream_t>(stream)};
    return vlmce::linear::backward(a, "linear_bwd");
}

extern "C" vlmce_status glu_bwd(const void *dy, int64_t dy_stride, const void *x, int64_t x_stride,
                                const void *weight, int64_t weight_stride, const void *preact,
                                int64_t preact_stride, int32_t dtype, int64_t T, int64_t n,
                                int64_t K, int32_t act, void *dx, int64_t dx_stride, void *dweight,
                                int32_t dweight_dtype, int32_t accumulate, int32_t *dev_err,
                                void *workspace, size_t workspace_bytes, vlmce_stream_t stream) {
    vlmce::linear::BwdArgs a = {dy, dy_stride, x, x_stride, weight, weight_stride, preact,
                                preact_stride, dtype, T, n, K, act, dx, dx_stride, dweight,
                                dweight_dtype, nullptr, accumulate, dev_err, workspace,
                                workspace_bytes, true, reinterpret_cast<cudaStream_t>(stream)};
    return vlmce::linear::backward(a, "glu_bwd");
}

extern "C" vlmce_status vlmce_linear_describe_plan(int32_t gated, int32_t backward, int64_t T,
                                                   int64_t N, int64_t K, int32_t dtype,
                                                   int32_t *out) {
    using namespace vlmce;
    const bool fp8 = dtype == VLMCE_E4M3;
    if ((!fp8 || backward) && dtype != VLMCE_BF16 && dtype != VLMCE_F16)
        return VLMCE_ERR_UNSUPPORTED_DTYPE;
    if (!out || T < 1 || N < 1 || K < 1 || K % (fp8 ? 16 : 8) != 0) return VLMCE_ERR_INVALID_ARG;
    if (!linear::fwd_sizes_ok(T, N, K) || (backward && !linear::bwd_sizes_ok(T, N, K)))
        return VLMCE_ERR_TOO_LARGE;
    DeviceInfo dev;
    const vlmce_status st = current_device(&dev);
    if (st != VLMCE_OK) return st;
    for (int i = 0; i < 8; ++i) out[i] = 0;
    cudaError_t e;
    if (backward) {
        mm::Bwd b = {};
        b.T = T;
        b.rows = gated ? 2 * N : N;
        b.K = K;
        b.f16 = dtype == VLMCE_F16;
        b.dw = out;  // dx and dweight; nothing is written
        e = mm::describe(b, out);
    } else {
        mm::Fwd f = {};
        f.T = T;
        f.N = N;
        f.K = K;
        f.gated = gated != 0;
        f.dtype = dtype;
        e = mm::describe(f, out);
    }
    return launch_status(e, "vlmce_linear_describe_plan");
}
