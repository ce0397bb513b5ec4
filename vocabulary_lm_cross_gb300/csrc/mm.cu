// mm.cu -- host side of the linear and gated layers' forward products: tensor
// maps, tile and split choice, launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "gemm_launch.h"
#include "host_util.h"
#include "mm_large.cuh"
#include "mm_small.cuh"

namespace vlmce {
namespace mm {
namespace {

constexpr int kMaxDevices = 64;

bool operand_map(CUtensorMap *m, const void *base, int32_t dtype, int64_t rows, int64_t K,
                 int64_t ld, int box_rows) {
    const int elt = dtype == VLMCE_E4M3 ? 1 : 2;
    const CUtensorMapDataType type = dtype == VLMCE_E4M3  ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : dtype == VLMCE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                          : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return gemm::make_tile_map(m, base, type, elt, K, rows, ld, 128 / elt, box_rows);
}

int chunks_of(const Fwd &f) {
    const int64_t bytes = f.K * (f.dtype == VLMCE_E4M3 ? 1 : 2);
    return static_cast<int>((bytes + 127) / 128);
}

using LargeKernel = void (*)(const CUtensorMap, const CUtensorMap, const LargeParams);
using SmallKernel = void (*)(const CUtensorMap, const CUtensorMap, const SmallParams);

LargeKernel large_kernel(bool gated, bool fp8) {
    if (gated) return fp8 ? mm_large_kernel<true, true> : mm_large_kernel<true, false>;
    return fp8 ? mm_large_kernel<false, true> : mm_large_kernel<false, false>;
}
SmallKernel small_kernel(bool gated, bool fp8) {
    if (gated) return fp8 ? mm_small_kernel<true, true> : mm_small_kernel<true, false>;
    return fp8 ? mm_small_kernel<false, true> : mm_small_kernel<false, false>;
}

// Opt in to the kernels' dynamic shared memory (once per device) and count
// the CTA pairs of the large kernels that fit at once.
cudaError_t setup(int *pairs) {
    static std::mutex mu;
    static int cached[kMaxDevices] = {};
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    if (device < 0 || device >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (cached[device] == 0) {
        int least = 0;
        for (int k = 0; k < 4; ++k) {
            LargeKernel lk = large_kernel(k & 1, k & 2);
            e = cudaFuncSetAttribute(lk, cudaFuncAttributeMaxDynamicSharedMemorySize, kLargeSmem);
            if (e != cudaSuccess) return e;
            e = cudaFuncSetAttribute(small_kernel(k & 1, k & 2),
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
            if (e != cudaSuccess) return e;
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 2;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.gridDim = dim3(2, 1, 1);
            cfg.blockDim = dim3(kLargeThreads, 1, 1);
            cfg.dynamicSmemBytes = kLargeSmem;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int n = 0;
            e = cudaOccupancyMaxActiveClusters(&n, lk, &cfg);
            if (e != cudaSuccess) return e;
            if (n < 1) return cudaErrorInvalidConfiguration;
            least = k == 0 ? n : std::min(least, n);
        }
        cached[device] = least;
    }
    *pairs = cached[device];
    return cudaSuccess;
}

}  // namespace

cudaError_t forward_large(const Fwd &f, cudaStream_t s) {
    int pairs = 0;
    cudaError_t e = setup(&pairs);
    if (e != cudaSuccess) return e;
    CUtensorMap mx, mw;
    const int64_t rows = f.gated ? 2 * f.N : f.N;
    if (!operand_map(&mx, f.x, f.dtype, f.T, f.K, f.x_ld, kHalfRows) ||
        !operand_map(&mw, f.w, f.dtype, rows, f.K, f.w_ld, kHalfRows))
        return cudaErrorInvalidValue;
    LargeParams p = {};
    p.T = static_cast<int>(f.T);
    p.N = static_cast<int>(f.N);
    p.up_row = static_cast<int>(f.N);
    p.chunks = chunks_of(f);
    p.mt = static_cast<int>((f.T + kPairM - 1) / kPairM);
    p.nt = static_cast<int>(f.gated ? (f.N + 127) / 128 : (f.N + 255) / 256);
    const int64_t tiles = static_cast<int64_t>(p.mt) * p.nt;
    if (tiles * kGroupM > INT32_MAX) return cudaErrorInvalidConfiguration;
    p.tiles = static_cast<int>(tiles);
    p.e = f.e;
    p.err = f.err;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(2 * std::min(p.tiles, pairs), 1, 1);
    cfg.blockDim = dim3(kLargeThreads, 1, 1);
    cfg.dynamicSmemBytes = kLargeSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, large_kernel(f.gated != 0, f.dtype == VLMCE_E4M3), mx, mw,
                              static_cast<const LargeParams>(p));
}

cudaError_t forward_small(const Fwd &f, int sm_count, cudaStream_t s) {
    int pairs = 0;
    cudaError_t e = setup(&pairs);
    if (e != cudaSuccess) return e;
    const int kw = f.gated ? 2 : 1;
    SmallParams p = {};
    p.T = static_cast<int>(f.T);
    p.N = static_cast<int>(f.N);
    p.up_row = static_cast<int>(f.N);
    p.chunks = chunks_of(f);
    const int64_t token_tiles = (f.T + 255) / 256;
    p.bn = static_cast<int>(round_up((f.T + token_tiles - 1) / token_tiles, 16));
    const int64_t ty = (f.T + p.bn - 1) / p.bn;
    const int64_t mt = (f.N + 127) / 128;
    int cols = 32;
    while (cols < kw * p.bn) cols *= 2;
    p.tmem_cols = cols;
    const int per_sm = cols > 256 ? 1 : 2;
    // K split over a cluster while the CTAs fit in one wave and each keeps
    // several chunks of K
    p.split = 1;
    while (p.split < kMaxSplit && mt * ty * p.split * 2 <= static_cast<int64_t>(sm_count) * per_sm &&
           p.chunks >= 8 * p.split)
        p.split *= 2;
    const int stage = kw * kWTileBytes + p.bn * 128;
    const int budget = 233472 / per_sm - kSmemReserved;
    const int want = (p.chunks + p.split - 1) / p.split;
    p.stages = std::min({(budget - 1024 - kSmallTail) / stage, kMaxSmallStages, want});
    const int ring = p.stages * stage;
    p.red_tokens = std::min(p.bn, ring / (kw * 512) / 16 * 16);
    int smem = 1024 + ring + kSmallTail;
    smem = std::max({smem, cols * kSmemPerTmemCol - kSmemReserved, kSmallSmemMin});
    p.e = f.e;
    p.err = f.err;
    if (ty > 65535 || mt * p.split > INT32_MAX) return cudaErrorInvalidConfiguration;

    CUtensorMap mx, mw;
    const int64_t rows = f.gated ? 2 * f.N : f.N;
    if (!operand_map(&mx, f.x, f.dtype, f.T, f.K, f.x_ld, p.bn) ||
        !operand_map(&mw, f.w, f.dtype, rows, f.K, f.w_ld, 128))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(p.split);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(mt * p.split), static_cast<unsigned>(ty), 1);
    cfg.blockDim = dim3(kSmallThreads, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, small_kernel(f.gated != 0, f.dtype == VLMCE_E4M3), mw, mx,
                              static_cast<const SmallParams>(p));
}

cudaError_t forward(const Fwd &f, int sm_count, cudaStream_t s) {
    const int64_t tiles =
        ((f.T + 255) / 256) * (f.gated ? (f.N + 127) / 128 : (f.N + 255) / 256);
    if (f.T <= 256 || tiles < sm_count / 2) return forward_small(f, sm_count, s);
    return forward_large(f, s);
}

}  // namespace mm
}  // namespace vlmce
