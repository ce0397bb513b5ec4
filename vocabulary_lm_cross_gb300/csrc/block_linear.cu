// block_linear.cu -- entry points of the products of e4m3 operands with one scale per
// block of 128, dense and by experts: argument checks (mm_block.cu runs them).
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>

#include "host_util.h"
#include "mm_block_types.h"
#include "rows_host.h"
#include "vlmce.h"

namespace vlmce {
namespace mmb {
namespace {

struct Mat {
    const void *p;
    int64_t rows, cols, ld;
    int elt;
};
bool overlap(const Mat &a, const Mat &b) {
    return rows_overlap({a.p, a.rows, a.cols * a.elt, a.ld * a.elt},
                        {b.p, b.rows, b.cols * b.elt, b.ld * b.elt});
}
vlmce_status check(const Mat &m) {
    if (m.ld < m.cols || (m.rows > 0 && !m.p)) return VLMCE_ERR_INVALID_ARG;
    if (m.ld > (int64_t(1) << 60) / m.elt / std::max<int64_t>(m.rows, 1)) return VLMCE_ERR_TOO_LARGE;
    if (!aligned(m.p, static_cast<uintptr_t>(m.elt))) return VLMCE_ERR_MISALIGNED;
    return VLMCE_OK;
}
// An operand of the tensor cores: its rows in whole 16-byte units.
vlmce_status check_operand(const Mat &m) {
    const vlmce_status st = check(m);
    if (st != VLMCE_OK) return st;
    if (m.ld % 16 != 0) return VLMCE_ERR_INVALID_ARG;
    if (m.ld >= (int64_t(1) << 40)) return VLMCE_ERR_TOO_LARGE;
    return aligned(m.p, 16) ? VLMCE_OK : VLMCE_ERR_MISALIGNED;
}
int64_t blocks_of(int64_t n) { return n / 128 + (n % 128 != 0); }

// The tiles are numbered in 32 bits, also where a cluster of eight shares one.
vlmce_status sizes(int64_t T, int64_t N, int64_t K, int64_t groups) {
    if (T < 0 || N < 1 || K < 1 || groups < 1) return VLMCE_ERR_INVALID_ARG;
    if (groups > VLMCE_MOE_MAX_EXPERTS || T > INT32_MAX - 256 || N > (INT32_MAX - 256) / groups ||
        K > INT32_MAX - 256 || T / 16 + groups + 1 > INT32_MAX / 16 / (N / 128 + 1))
        return VLMCE_ERR_TOO_LARGE;
    return VLMCE_OK;
}
bool block_ok(int32_t block) { return block == 1 || block == 128; }

}  // namespace
}  // namespace mmb
}  // namespace vlmce

extern "C" vlmce_status block_linear_fwd(const void *x, int64_t x_stride, const float *x_scale,
                                         int64_t x_scale_stride, const void *weight,
                                         int64_t weight_stride, const float *weight_scale,
                                         int64_t weight_scale_stride, int32_t weight_block,
                                         const int32_t *offsets, int64_t E, const void *residual,
                                         int64_t residual_stride, int32_t out_dtype, int64_t T,
                                         int64_t N, int64_t K, void *y, int64_t y_stride,
                                         int32_t *dev_err, vlmce_stream_t stream) {
    using namespace vlmce;
    using namespace vlmce::mmb;
    if (out_dtype != VLMCE_BF16 && out_dtype != VLMCE_F16) return VLMCE_ERR_UNSUPPORTED_DTYPE;
    if (!block_ok(weight_block) || (!offsets && E != 1)) return VLMCE_ERR_INVALID_ARG;
    vlmce_status st = sizes(T, N, K, E);
    if (st != VLMCE_OK) return st;
    const int64_t nb = blocks_of(K), wb = weight_block == 1 ? N : blocks_of(N);
    const Mat a{x, T, K, x_stride, 1}, w{weight, E * N, K, weight_stride, 1},
        as{x_scale, T, nb, x_scale_stride, 4}, ws{weight_scale, E * wb, nb, weight_scale_stride, 4},
        r{residual, residual ? T : 0, N, residual_stride, 2}, o{y, T, N, y_stride, 2},
        off{offsets, offsets ? 1 : 0, E + 1, E + 1, 4};
    st = check_operand(a);
    if (st == VLMCE_OK) st = check_operand(w);
    if (st == VLMCE_OK) st = check(as);
    if (st == VLMCE_OK) st = check(ws);
    if (st == VLMCE_OK && residual) st = check(r);
    if (st == VLMCE_OK) st = check(o);
    if (st != VLMCE_OK) return st;
    if (!aligned(offsets, 4) || !aligned(dev_err, 4)) return VLMCE_ERR_MISALIGNED;
    if (overlap(o, a) || overlap(o, w) || overlap(o, as) || overlap(o, ws) || overlap(o, off) ||
        (overlap(o, r) && !(y == residual && (y_stride == residual_stride || T <= 1))))
        return VLMCE_ERR_INVALID_ARG;
    if (T == 0) return VLMCE_OK;
    DeviceInfo dev;
    st = current_device(&dev);
    if (st != VLMCE_OK) return st;
    Fwd f = {};
    f.x = x;
    f.w = weight;
    f.x_ld = x_stride;
    f.w_ld = weight_stride;
    f.xs = x_scale;
    f.ws = weight_scale;
    f.xs_ld = x_scale_stride;
    f.ws_ld = weight_scale_stride;
    f.block = weight_block;
    f.offsets = offsets;
    f.groups = E;
    f.T = T;
    f.N = N;
    f.K = K;
    f.residual = static_cast<const uint16_t *>(residual);
    f.residual_ld = residual_stride;
    f.y = static_cast<uint16_t *>(y);
    f.y_ld = y_stride;
    f.f16 = out_dtype == VLMCE_F16;
    f.err = dev_err;
    return launch_status(forward(f, reinterpret_cast<cudaStream_t>(stream)), "block_linear_fwd");
}

extern "C" vlmce_status block_linear_dweight(const void *dyt, int64_t dyt_stride,
                                             const float *dyt_scale, int64_t dyt_scale_stride,
                                             const void *xt, int64_t xt_stride, const float *xt_scale,
                                             int64_t xt_scale_stride, const int32_t *offsets,
                                             int64_t E, int64_t R, int64_t N, int64_t K,
                                             void *dweight, int32_t dweight_dtype,
                                             int32_t accumulate, int32_t *dev_err,
                                             vlmce_stream_t stream) {
    using namespace vlmce;
    using namespace vlmce::mmb;
    if (dweight_dtype != VLMCE_F32 && dweight_dtype != VLMCE_BF16 && dweight_dtype != VLMCE_F16)
        return VLMCE_ERR_UNSUPPORTED_DTYPE;
    if (!offsets && E != 1) return VLMCE_ERR_INVALID_ARG;
    vlmce_status st = sizes(R, N, K, E);
    if (st != VLMCE_OK) return st;
    if (K / 256 + 1 > INT32_MAX / 16 / E / (N / 256 + 1)) return VLMCE_ERR_TOO_LARGE;
    if (accumulate && dweight_dtype != VLMCE_F32) return VLMCE_ERR_INVALID_ARG;
    const int64_t nb = blocks_of(R);
    const int elt = dweight_dtype == VLMCE_F32 ? 4 : 2;
    const int64_t some = R > 0 ? 1 : 0;  // without rows nothing is read
    const Mat a{dyt, some * N, R, dyt_stride, 1}, b{xt, some * K, R, xt_stride, 1},
        as{dyt_scale, some * N, nb, dyt_scale_stride, 4}, bs{xt_scale, some * K, nb, xt_scale_stride, 4},
        o{dweight, E * N, K, K, elt}, off{offsets, offsets ? 1 : 0, E + 1, E + 1, 4};
    st = check(o);
    if (st == VLMCE_OK && some) st = check_operand(a);
    if (st == VLMCE_OK && some) st = check_operand(b);
    if (st == VLMCE_OK && some) st = check(as);
    if (st == VLMCE_OK && some) st = check(bs);
    if (st != VLMCE_OK) return st;
    if (!aligned(offsets, 4) || !aligned(dev_err, 4)) return VLMCE_ERR_MISALIGNED;
    if (overlap(o, a) || overlap(o, b) || overlap(o, as) || overlap(o, bs) || overlap(o, off))
        return VLMCE_ERR_INVALID_ARG;
    DeviceInfo dev;
    st = current_device(&dev);
    if (st != VLMCE_OK) return st;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (R == 0) {
        cudaError_t e = cudaSuccess;
        if (!accumulate) e = cudaMemsetAsync(dweight, 0, static_cast<size_t>(E * N * K * elt), s);
        return launch_status(e, "block_linear_dweight");
    }
    Dw d = {};
    d.dyt = dyt;
    d.xt = xt;
    d.dyt_ld = dyt_stride;
    d.xt_ld = xt_stride;
    d.dyts = dyt_scale;
    d.xts = xt_scale;
    d.dyts_ld = dyt_scale_stride;
    d.xts_ld = xt_scale_stride;
    d.offsets = offsets;
    d.groups = E;
    d.R = R;
    d.N = N;
    d.K = K;
    d.dw = dweight;
    d.dtype = dweight_dtype;
    d.accumulate = accumulate != 0;
    d.err = dev_err;
    return launch_status(mmb::dweight(d, s), "block_linear_dweight");
}

extern "C" vlmce_status vlmce_block_linear_describe_plan(int64_t T, int64_t N, int64_t K, int64_t E,
                                                         int32_t grouped, int32_t *out) {
    using namespace vlmce;
    using namespace vlmce::mmb;
    if (!out || T < 1 || (!grouped && E != 1)) return VLMCE_ERR_INVALID_ARG;
    vlmce_status st = sizes(T, N, K, E);
    if (st != VLMCE_OK) return st;
    DeviceInfo dev;
    st = current_device(&dev);
    if (st != VLMCE_OK) return st;
    Fwd f = {};
    f.T = T;
    f.N = N;
    f.K = K;
    f.groups = E;
    f.block = 128;
    f.offsets = grouped ? out : nullptr;  // not read
    return launch_status(describe(f, out), "vlmce_block_linear_describe_plan");
}
