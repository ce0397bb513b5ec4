// mm.cu -- host side of the linear and gated layers' products: tensor maps,
// tile and split choice, launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "device_errors.h"
#include "gemm_launch.h"
#include "host_util.h"
#include "mm_grad.cuh"
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

// A 16-bit (or fp32) output [rows, cols], stored in boxes of 128 bytes x 32 rows: its
// columns in whole granules of 16 bytes, since a store would fill the last one (Out in
// mm_pair.cuh; the fp32 ones, a weight's K columns, are whole).
bool output_map(CUtensorMap *m, const void *base, bool f32, int64_t rows, int64_t cols,
                int64_t ld) {
    return gemm::make_tile_map(
        m, base, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
        f32 ? 4 : 2, cols & ~int64_t{7}, rows, ld, f32 ? 32 : 64, 32);
}

int chunks_of(const Fwd &f) {
    const int64_t bytes = f.K * (f.dtype == VLMCE_E4M3 ? 1 : 2);
    return static_cast<int>((bytes + 127) / 128);
}

using LargeKernel = void (*)(const LargeMaps, const LargeParams);
using SmallKernel = void (*)(const CUtensorMap, const CUtensorMap, const SmallParams);

LargeKernel large_kernel(bool gated, bool fp8, bool add) {
    if (gated) return fp8 ? mm_large_kernel<true, true, false> : mm_large_kernel<true, false, false>;
    if (add) return fp8 ? mm_large_kernel<false, true, true> : mm_large_kernel<false, false, true>;
    return fp8 ? mm_large_kernel<false, true, false> : mm_large_kernel<false, false, false>;
}
SmallKernel small_kernel(bool gated, bool fp8, bool w_mn) {
    if (w_mn) return mm_small_kernel<false, false, true>;
    if (gated) return fp8 ? mm_small_kernel<true, true, false> : mm_small_kernel<true, false, false>;
    return fp8 ? mm_small_kernel<false, true, false> : mm_small_kernel<false, false, false>;
}

// Clusters of `csize` CTAs, launched dependent on what precedes them.
void launch_attributes(cudaLaunchAttribute (&attr)[2], unsigned csize) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = csize;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
}

// Per device: the CTA pairs of the large kernels, and the clusters of 1 ..
// kMaxSplit small CTAs with one (or two) CTAs' shared memory per SM, that fit
// at once (SMs of a GPC that cannot complete a cluster stay idle); and the word that
// takes the errors of calls without one of their own.
struct Capacity {
    int pairs = 0;
    int small[2][kMaxSplit];
    int *errors = nullptr;
};
// no small CTA beside a kernel that holds all TMEM columns (mm_small.cuh)
static_assert(gemm::kSmemBytes + kSmallSmemMin + 2 * kSmemReserved > kSmSmem, "GEMM engine");
static_assert(kPairSmem + kSmallSmemMin + 2 * kSmemReserved > kSmSmem, "pair kernels");
constexpr int small_budget(int per_sm) { return kSmSmem / per_sm - kSmemReserved; }

// Stands for the small kernels in occupancy queries, which count a kernel that
// allocates TMEM as one CTA per SM whatever it takes (several do share one).
// Never launched.
__global__ void __launch_bounds__(kSmallBound, 2) small_shape_kernel() {}

template <class Kernel>
cudaError_t clusters_of(Kernel k, int csize, int threads, int smem, int *n) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    launch_attributes(attr, static_cast<unsigned>(csize));
    cfg.gridDim = dim3(static_cast<unsigned>(csize), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaOccupancyMaxActiveClusters(n, k, &cfg);
    return e == cudaSuccess && *n < 1 ? cudaErrorInvalidConfiguration : e;
}

// Opt in to the kernels' dynamic shared memory and query the capacities, once
// per device.
cudaError_t setup(Capacity *out) {
    static std::mutex mu;
    static Capacity cached[kMaxDevices];
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    if (device < 0 || device >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (cached[device].pairs == 0) {
        Capacity c;
        e = device_error_word(&c.errors);
        if (e != cudaSuccess) return e;
        for (int k = 0; k < 5; ++k) {
            e = cudaFuncSetAttribute(small_kernel(k & 1, k & 2, k & 4),
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, small_budget(1));
            if (e != cudaSuccess) return e;
        }
        for (int k = 0; k < 8; ++k) {
            const LargeKernel lk = large_kernel(k & 1, k & 2, k & 4);
            e = cudaFuncSetAttribute(lk, cudaFuncAttributeMaxDynamicSharedMemorySize, kPairSmem);
            int n = 0;
            if (e == cudaSuccess) e = clusters_of(lk, 2, kPairThreads, kPairSmem, &n);
            if (e != cudaSuccess) return e;
            c.pairs = k == 0 ? n : std::min(c.pairs, n);
        }
        e = cudaFuncSetAttribute(mm_grad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kPairSmem);
        int n = 0;
        if (e == cudaSuccess) e = clusters_of(mm_grad_kernel, 2, kPairThreads, kPairSmem, &n);
        if (e != cudaSuccess) return e;
        c.pairs = std::min(c.pairs, n);
        e = cudaFuncSetAttribute(small_shape_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 small_budget(1));
        if (e != cudaSuccess) return e;
        for (int per_sm = 1; per_sm <= 2; ++per_sm)
            for (int split = 1; split <= kMaxSplit; ++split) {
                e = clusters_of(small_shape_kernel, split, kSmallThreads,
                                small_budget(per_sm), &c.small[per_sm - 1][split - 1]);
                if (e != cudaSuccess) return e;
            }
        cached[device] = c;
    }
    *out = cached[device];
    return cudaSuccess;
}

// How a product is run: pair tiles, or bn tokens x 128 weight rows per CTA
// with K split over `split` CTAs.
struct Plan {
    bool large;
    int narrow;     // large: tiles of 128 weight rows
    int bn, split, stages, per_stage, tmem_cols, smem;
    int part_offset, red_tokens;  // SmallParams
    int per_sm;       // small: CTAs of an SM that the estimate counts on
    double clocks;  // estimate
};

// Estimates in SM clocks at 1.9 GHz, fitted to a sweep on GB300 of every bn,
// split and per_stage over 27 products (T = 1 .. 2000, K = 512 .. 16384, N =
// 100 .. 12288, both types, linear and gated): the chosen plan is within 2 % of
// the fastest on average, 11 % at worst.  A stage of a small CTA costs the
// larger of its MMAs (128 x bn: bn / 2 clocks each at the tensor cores' rate,
// or the shared-memory reads of both operands) and its way from L2, shared by
// the CTAs of an SM; it is free again a fetch latency, a transfer and its MMAs
// later.  The weight comes from HBM at 6.8 TB/s at best.  A narrow pair tile's chunk
// costs 3/4 of a wide one's for half the products, so narrow tiles are for few of them
// (us, narrow and wide: T 512, K 4096, N 4096 bf16 20.9 and 24.2; T 256, K 8192, N 8192
// 36.0 and 44.2; T 1024, K 4096, N 4096 36.0 and 25.1).
constexpr double kHbmBytesPerClock = 3570., kL2BytesPerClock = 76.;
constexpr double kFetch = 900., kPerStage = 260., kPerCta = 6900., kSplitSync = 1300.;
constexpr double kOut = 25., kOutSplit = 40.;   // epilogue, per token of an accumulator
constexpr double kPairChunk = 640., kNarrowChunk = 480., kPairCta = 7900.;

double hbm_clocks(const Fwd &f) {
    return static_cast<double>(f.N) * (f.gated ? 2 : 1) * f.K *
           (f.dtype == VLMCE_E4M3 ? 1 : 2) / kHbmBytesPerClock;
}

bool small_plan(const Fwd &f, const Capacity &cap, int64_t ty, int split, int per_stage,
                Plan *out) {
    const int kw = f.gated ? 2 : 1;
    const int chunks = chunks_of(f);
    Plan p = {};
    p.bn = static_cast<int>(round_up((f.T + ty - 1) / ty, 16));
    if (p.bn > 256 || split * per_stage > chunks) return false;
    p.split = split;
    p.per_stage = per_stage;
    const int64_t clusters = (f.N + 127) / 128 * ((f.T + p.bn - 1) / p.bn);
    p.tmem_cols = 32;
    while (p.tmem_cols < kw * p.bn) p.tmem_cols *= 2;
    const int per_sm = p.tmem_cols > 256 || clusters <= cap.small[0][split - 1] ? 1 : 2;
    p.per_sm = per_sm;
    const double waves = static_cast<double>(clusters) / cap.small[per_sm - 1][split - 1];
    const double rounds = per_sm == 1 ? std::ceil(waves) : waves > 1. ? waves + 0.3 : 1.;
    const int stage = per_stage * (kw * kWTileBytes + p.bn * 128);
    const int steps = ((chunks + split - 1) / split + per_stage - 1) / per_stage;
    // the split's exchange: up to 16 KB of its own (T = 8, K = N = 1024 5.3 -> 4.6 us;
    // more would cost the ring: T = 64, K = 16384 24.8 -> 25.9)
    int part = split > 1 ? static_cast<int>(round_up(p.bn / 4, split)) * 4 * kw * 512 : 0;
    if (part > 16384) part = 0;
    p.stages = std::min(
        {(small_budget(per_sm) - 1040 - kSmallTail - part) / stage, kMaxSmallStages, steps});
    if (p.stages < 1) return false;
    p.part_offset = part > 0 ? static_cast<int>(round_up(p.stages * stage + kSmallTail, 16)) : 0;
    p.red_tokens = p.bn;  // in the ring: as many tokens at a time as it holds
    while (part == 0 &&
           (p.red_tokens / 4 + split - 1) / split * 4 * split * kw * 512 > p.stages * stage)
        p.red_tokens -= 16;
    p.smem = std::max({1024 + p.stages * stage + kSmallTail + (part > 0 ? part + 16 : 0),
                       p.tmem_cols * kSmemPerTmemCol - kSmemReserved, kSmallSmemMin});
    const double mma = per_stage * kw * 4 * std::max(p.bn / 2., 32. + p.bn / 4.);
    const double load = stage / kL2BytesPerClock;
    const double step =
        std::max(per_sm * std::max(mma, load), (kFetch + load + mma) / p.stages) + kPerStage;
    const double main = rounds * steps * step, hbm = hbm_clocks(f);
    const double epilogue =
        per_sm * kw * p.bn * (split > 1 ? kOutSplit : kOut) + (split > 1 ? kSplitSync : 0.);
    p.clocks = std::sqrt(std::hypot(main * main, hbm * hbm)) + rounds * (kPerCta + epilogue);
    *out = p;
    return true;
}

Plan choose(const Fwd &f, const Capacity &cap) {
    Plan best = {};
    for (int narrow = 0; narrow < 2; ++narrow) {
        const int64_t width = (f.gated ? 128 : 256) >> narrow;
        const int64_t tiles = ((f.T + 255) / 256) * ((f.N + width - 1) / width);
        const double main = static_cast<double>((tiles + cap.pairs - 1) / cap.pairs) *
                            chunks_of(f) * (narrow ? kNarrowChunk : kPairChunk);
        const double clocks = std::hypot(main, 0.6 * hbm_clocks(f)) + kPairCta;
        if (narrow == 0 || clocks < best.clocks) {
            best.large = true;
            best.narrow = narrow;
            best.clocks = clocks;
        }
    }
    const int64_t t0 = (f.T + 255) / 256;
    if (t0 > 16) return best;  // enough tokens for the pair tiles
    for (int64_t ty = t0; ty < t0 + 5; ++ty)
        for (int split = 1; split <= kMaxSplit; ++split)
            for (int per_stage = 1; per_stage <= 2; ++per_stage) {
                Plan p;
                if (small_plan(f, cap, ty, split, per_stage, &p) && p.clocks < best.clocks)
                    best = p;
            }
    return best;
}

// choose() for the sizes a host thread met last (a decoder's few layer shapes;
// the search takes several microseconds).
Plan plan_of(const Fwd &f, const Capacity &cap) {
    struct Entry {
        int64_t T = -1, N, K;
        int gated, pairs;
        int32_t dtype;
        Plan plan;
    };
    constexpr int kEntries = 64;
    static thread_local Entry entries[kEntries];
    const uint64_t h = static_cast<uint64_t>(f.T) * 0x9E3779B97F4A7C15ull ^
                       static_cast<uint64_t>(f.N) * 0xC2B2AE3D27D4EB4Full ^
                       static_cast<uint64_t>(f.K) * 0x165667B19E3779F9ull ^
                       static_cast<uint64_t>(f.dtype * 2 + f.gated);
    Entry &e = entries[(h ^ h >> 29) % kEntries];
    if (e.T != f.T || e.N != f.N || e.K != f.K || e.gated != f.gated || e.dtype != f.dtype ||
        e.pairs != cap.pairs) {
        e.plan = choose(f, cap);
        e.T = f.T;
        e.N = f.N;
        e.K = f.K;
        e.gated = f.gated;
        e.dtype = f.dtype;
        e.pairs = cap.pairs;
    }
    return e.plan;
}

// Pair kernels: CTAs to launch, and how the pairs share the tiles (Tiles in
// mm_pair.cuh).  Dealt out, T = 16, K = 4096, N = 16384's dW takes 38.7 us (45.6 by
// launch control); T = 4096, K = 6656, 2n = 32768 forward is 4 % slower that way.
unsigned pair_grid(int64_t tiles, int chunks, const Capacity &cap, int *dealt) {
    *dealt = chunks < 32 ? static_cast<int>(tiles) : 0;
    return static_cast<unsigned>(2 * (*dealt > 0 ? std::min<int64_t>(tiles, cap.pairs) : tiles));
}

cudaError_t forward_large(const Fwd &f, const Capacity &cap, int narrow, cudaStream_t s) {
    LargeMaps maps = {};
    const int64_t rows = f.gated ? 2 * f.N : f.N;
    const Epi &e = f.e;
    bool ok = operand_map(&maps.x, f.x, f.dtype, f.T, f.K, f.x_ld, kHalfRows) &&
              operand_map(&maps.w, f.w, f.dtype, rows, f.K, f.w_ld, kHalfRows >> narrow);
    if (e.y_vec >= 16) ok = ok && output_map(&maps.y, e.y, false, f.T, f.N, e.y_ld);
    if (e.preact && e.preact_vec >= 16)
        ok = ok && output_map(&maps.z, e.preact, false, f.T, f.N, e.preact_ld);
    if (f.gated && e.preact && e.preact_up_vec >= 16)
        ok = ok && output_map(&maps.z_up, e.preact + f.N, false, f.T, f.N, e.preact_ld);
    if (!ok) return cudaErrorInvalidValue;
    LargeParams p = {};
    p.T = static_cast<int>(f.T);
    p.N = static_cast<int>(f.N);
    p.up_row = static_cast<int>(f.N);
    p.chunks = chunks_of(f);
    p.mt = static_cast<int>((f.T + kPairM - 1) / kPairM);
    p.narrow = narrow;
    const int64_t width = (f.gated ? 128 : 256) >> narrow;
    p.nt = static_cast<int>((f.N + width - 1) / width);
    const int64_t tiles = static_cast<int64_t>(p.mt) * p.nt;
    if (tiles * kGroupM > INT32_MAX) return cudaErrorInvalidConfiguration;
    const unsigned grid = pair_grid(tiles, p.chunks, cap, &p.dealt);
    p.e = f.e;
    p.err = f.err ? f.err : cap.errors;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    launch_attributes(attr, 2);
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(kPairThreads, 1, 1);
    cfg.dynamicSmemBytes = kPairSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, large_kernel(f.gated != 0, f.dtype == VLMCE_E4M3, f.e.residual), maps,
                              static_cast<const LargeParams>(p));
}

cudaError_t forward_small(const Fwd &f, const Capacity &cap, const Plan &plan, cudaStream_t s) {
    SmallParams p = {};
    p.T = static_cast<int>(f.T);
    p.N = static_cast<int>(f.N);
    p.up_row = static_cast<int>(f.N);
    p.chunks = chunks_of(f);
    p.split = plan.split;
    p.bn = plan.bn;
    p.stages = plan.stages;
    p.per_stage = plan.per_stage;
    p.tmem_cols = plan.tmem_cols;
    const int64_t ty = (f.T + p.bn - 1) / p.bn;
    const int64_t mt = (f.N + 127) / 128;
    p.red_tokens = plan.red_tokens;
    p.part_offset = plan.part_offset;
    p.e = f.e;
    p.err = f.err ? f.err : cap.errors;
    if (ty > 65535 || mt * p.split > INT32_MAX) return cudaErrorInvalidConfiguration;

    CUtensorMap mx, mw;
    const int64_t rows = f.gated ? 2 * f.N : f.N;
    const bool w_ok =
        f.w_mn ? gemm::make_operand_map(&mw, f.w, true, f.N, f.K, f.w_ld, f.dtype == VLMCE_F16)
               : operand_map(&mw, f.w, f.dtype, rows, f.K, f.w_ld, 128);
    if (!w_ok || !operand_map(&mx, f.x, f.dtype, f.T, f.K, f.x_ld, p.bn))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    launch_attributes(attr, static_cast<unsigned>(p.split));
    cfg.gridDim = dim3(static_cast<unsigned>(mt * p.split), static_cast<unsigned>(ty), 1);
    cfg.blockDim = dim3(kSmallThreads, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(plan.smem);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, small_kernel(f.gated != 0, f.dtype == VLMCE_E4M3, f.w_mn != 0), mw, mx,
                              static_cast<const SmallParams>(p));
}

}  // namespace

cudaError_t forward(const Fwd &f, cudaStream_t s) {
    Capacity cap;
    const cudaError_t e = setup(&cap);
    if (e != cudaSuccess) return e;
    const Plan plan = plan_of(f, cap);
    return plan.large ? forward_large(f, cap, plan.narrow, s) : forward_small(f, cap, plan, s);
}

namespace {

// Estimates of backward()'s launches in SM clocks: dW after dx, and both in one
// launch.  A dW tile of few chunks takes its epilogue's time; a dx tile's walk along
// W's rows alone goes faster than beside 75 others.  Fitted to both ways' times at 68
// sizes (T = 16 .. 2048, K = 512 .. 8192, N = 512 .. 12288): 0.4 % over the faster one
// on average, 11 % at worst.
constexpr double kDwTile = 5000., kDwChunk = 450., kDwLaunch = 9500.;
constexpr double kDxChunk = 509., kJointLaunch = 13000.;

double dw_tile_clocks(const Bwd &b) {
    const double chunks = static_cast<double>((b.T + 63) / 64);
    return std::max(kPairChunk * chunks, kDwTile + kDwChunk * chunks);
}
double dw_tiles(const Bwd &b) {
    return static_cast<double>((b.rows + 255) / 256) * static_cast<double>((b.K + 255) / 256);
}
double dw_clocks(const Bwd &b, const Capacity &cap) {
    return std::ceil(dw_tiles(b) / cap.pairs) * dw_tile_clocks(b) + kDwLaunch;
}
double joint_clocks(const Bwd &b, const Capacity &cap) {
    const double chunks = static_cast<double>((b.rows + 63) / 64);
    const double tiles =
        static_cast<double>((b.T + 255) / 256) * static_cast<double>((b.K + 255) / 256);
    return std::max(kDxChunk * chunks, (tiles * kPairChunk * chunks +
                                        dw_tiles(b) * dw_tile_clocks(b)) / cap.pairs) +
           kJointLaunch;
}

// dx = dz W as a product of the small kernel (W's rows are its K).
Fwd dx_product(const Bwd &b) {
    Fwd f = {};
    f.x = b.dz;
    f.w = b.w;
    f.x_ld = b.dz_ld;
    f.w_ld = b.w_ld;
    f.T = b.T;
    f.N = b.K;
    f.K = b.rows;
    f.w_mn = 1;
    f.dtype = b.f16 ? VLMCE_F16 : VLMCE_BF16;
    f.e.y = static_cast<uint16_t *>(b.dx);
    f.e.y_ld = b.dx_ld;
    f.e.f16 = b.f16;
    f.err = b.err;
    return f;
}
// dx alone for few tokens takes the small kernel, which spreads the weight over all SMs:
// T = 16, K = 4096, N = 16384 24 us (73 us in pair tiles).  Beside dW that costs a
// launch; it pays where one pair tile's walk along W's rows would last longer (the same
// sizes: 71 against 83 us; T = 256: 100 against 87).
bool dx_goes_small(const Bwd &b, const Plan &plan, const Capacity &cap) {
    return !plan.large && (!b.dw || plan.clocks < joint_clocks(b, cap) - dw_clocks(b, cap));
}

}  // namespace

cudaError_t backward(const Bwd &b, cudaStream_t s) {
    Capacity cap;
    const cudaError_t e = setup(&cap);
    if (e != cudaSuccess) return e;
    bool dx = b.dx != nullptr;
    if (dx) {
        const Fwd f = dx_product(b);
        const Plan plan = plan_of(f, cap);
        if (dx_goes_small(b, plan, cap)) {
            const cudaError_t es = forward_small(f, cap, plan, s);
            if (es != cudaSuccess || !b.dw) return es;
            dx = false;
        }
    }
    GradMaps maps;
    GradParams p = {};
    p.f16 = b.f16;
    p.err = b.err ? b.err : cap.errors;
    const bool f16 = b.f16 != 0;
    int64_t tiles = 0;
    bool ok = true;
    auto add = [&](const void *a, bool a_mn, int64_t a_ld, const void *w, int64_t w_ld, int64_t M,
                   int64_t K, void *C, int64_t ld, int f32, int accumulate) {
        GradProblem &q = p.p[p.nprob];
        ok = ok && gemm::make_operand_map(&maps.a[p.nprob], a, a_mn, M, K, a_ld, f16) &&
             gemm::make_operand_map(&maps.b[p.nprob], w, true, b.K, K, w_ld, f16) &&
             output_map(&maps.c[p.nprob], C, f32 != 0, M, b.K, ld);
        q.M = static_cast<int>(M);
        q.N = static_cast<int>(b.K);
        q.chunks = static_cast<int>((K + 63) / 64);
        q.a_mn = a_mn;
        q.b_mn = 1;
        q.mt = static_cast<int>((M + 255) / 256);
        q.nt = static_cast<int>((b.K + 255) / 256);
        q.tile0 = static_cast<int>(tiles);
        q.f32 = f32;
        q.accumulate = accumulate;
        q.C = C;
        q.ld = ld;
        tiles += static_cast<int64_t>(q.mt) * q.nt;
        ++p.nprob;
    };
    const bool dx_first = b.rows >= b.T;  // longer tiles first
    for (int i = 0; i < 2; ++i) {
        if ((i == 0) == dx_first) {
            if (dx)
                add(b.dz, false, b.dz_ld, b.w, b.w_ld, b.T, b.rows, b.dx, b.dx_ld, 0, 0);
        } else if (b.dw) {
            add(b.dz, true, b.dz_ld, b.x, b.x_ld, b.rows, b.T, b.dw, b.K, b.dw_f32, b.accumulate);
        }
    }
    if (!ok) return cudaErrorInvalidValue;
    const unsigned grid = pair_grid(tiles, p.p[0].chunks, cap, &p.dealt);  // the longest
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    launch_attributes(attr, 2);
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(kPairThreads, 1, 1);
    cfg.dynamicSmemBytes = kPairSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, mm_grad_kernel, maps, static_cast<const GradParams>(p));
}

namespace {

// Tiles of a pair kernel's launch, and whether they are dealt out.
void describe_pairs(int64_t tiles, int chunks, const Capacity &cap, int32_t *out) {
    int dealt = 0;
    pair_grid(tiles, chunks, cap, &dealt);
    out[4] = static_cast<int32_t>(std::min<int64_t>(tiles, INT32_MAX));
    out[5] = dealt > 0;
}
void describe_tile(const Plan &p, bool gated, int32_t *out) {
    out[0] = !p.large;
    out[1] = p.large ? (gated ? 128 : 256) >> p.narrow : 128;
    out[2] = p.large ? kPairM : p.bn;
    out[3] = p.large ? 1 : p.split;
    out[6] = p.large ? 1 : p.per_sm;
    out[7] = p.large || p.split == 1 || p.part_offset > 0 ? 0 : (p.bn + p.red_tokens - 1) / p.red_tokens;
}

}  // namespace

cudaError_t describe(const Fwd &f, int32_t *out) {
    Capacity cap;
    const cudaError_t e = setup(&cap);
    if (e != cudaSuccess) return e;
    const Plan p = plan_of(f, cap);
    describe_tile(p, f.gated != 0, out);
    const int64_t tiles = (f.T + out[2] - 1) / out[2] * ((f.N + out[1] - 1) / out[1]);
    if (p.large)
        describe_pairs(tiles, chunks_of(f), cap, out);
    else
        out[4] = static_cast<int32_t>(std::min<int64_t>(tiles, INT32_MAX));
    return cudaSuccess;
}

cudaError_t describe(const Bwd &b, int32_t *out) {
    Capacity cap;
    const cudaError_t e = setup(&cap);
    if (e != cudaSuccess) return e;
    const Fwd f = dx_product(b);
    Plan p = plan_of(f, cap);
    const bool small = dx_goes_small(b, p, cap);
    if (!small) {  // dx in wide pair tiles, dW's launch
        p.large = true;
        p.narrow = 0;
    }
    describe_tile(p, false, out);
    const int64_t across = (b.K + 255) / 256;
    const int64_t dx_tiles = small ? 0 : (b.T + 255) / 256 * across;
    const int64_t deep = small ? b.T : std::max(b.T, b.rows);
    describe_pairs(dx_tiles + (b.rows + 255) / 256 * across, static_cast<int>((deep + 63) / 64), cap,
                   out);
    return cudaSuccess;
}

}  // namespace mm
}  // namespace vlmce
