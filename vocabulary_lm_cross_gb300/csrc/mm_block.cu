// mm_block.cu -- host side of the products with block scales: tensor maps, the choice of
// kernel and tiles, launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <mutex>

#include "device_errors.h"
#include "gemm_launch.h"
#include "host_util.h"
#include "mm_block_pair.cuh"
#include "mm_block_small.cuh"
#include "mm_types.h"

namespace vlmce {
namespace mmb {
namespace {

constexpr int kMaxDevices = 64;
constexpr int kBns[4] = {16, 32, 64, 128};  // rows of x in a small tile
// Shared memory of an SM (228 KB, 1 KB of it reserved per resident CTA) and, so that a
// CTA that waits for TMEM columns never waits on one that waits for it, the least a CTA of
// single-CTA kernels takes for its columns (mm_small.cuh) and beside the pair kernels.
constexpr int kSmSmem = 233472, kSmemReserved = 1024, kSmemPerTmemCol = 456;
constexpr int kSmallSmemMax = kSmSmem - kSmemReserved;
constexpr int kMaxPerSm = 2;  // CTAs of single-CTA kernels
// The least shared memory of a CTA where so many are to share an SM, and one more is not.
constexpr int least_smem(int per_sm) { return kSmSmem / (per_sm + 1) - kSmemReserved + 16; }
static_assert(gemm::kSmemBytes + least_smem(kMaxPerSm) + 2 * kSmemReserved > kSmSmem, "GEMM engine");
static_assert(mm::kPairSmem + least_smem(kMaxPerSm) + 2 * kSmemReserved > kSmSmem, "pair kernels");
static_assert(kSmemPerTmemCol * 512 >= kSmSmem, "TMEM would run out first");

using SmallKernel = void (*)(const CUtensorMap, const CUtensorMap, const SmallParams);
using PairKernel = void (*)(const PairMaps, const PairParams);

SmallKernel small_kernel(int bn, bool residual) {
    switch (bn) {
        case 16: return residual ? mm_block_small_kernel<8, true> : mm_block_small_kernel<8, false>;
        case 32: return residual ? mm_block_small_kernel<16, true> : mm_block_small_kernel<16, false>;
        case 64: return residual ? mm_block_small_kernel<32, true> : mm_block_small_kernel<32, false>;
        default: return residual ? mm_block_small_kernel<64, true> : mm_block_small_kernel<64, false>;
    }
}
PairKernel pair_kernel(bool dw, bool b_rows) {
    if (dw) return mm_block_pair_kernel<true, true>;
    return b_rows ? mm_block_pair_kernel<false, true> : mm_block_pair_kernel<false, false>;
}

void launch_attributes(cudaLaunchAttribute (&attr)[2], unsigned csize) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = csize;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
}

// Per device: the kernels' shared memory is opted in to, the CTA pairs that fit at once, the
// clusters of single CTAs (one or two of them on an SM), the SMs, and the word for errors of
// calls without one of their own.
struct Capacity {
    int pairs = 0, sms = 0;
    int clusters[2][kMaxSplit + 1] = {};
    int *errors = nullptr;
};
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
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&c.sms, cudaDevAttrMultiProcessorCount, device);
        if (e != cudaSuccess) return e;
        for (const int bn : kBns)
            for (int res = 0; res < 2; ++res) {
                e = cudaFuncSetAttribute(small_kernel(bn, res), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kSmallSmemMax);
                if (e != cudaSuccess) return e;
            }
        for (int k = 0; k < 3; ++k) {
            const PairKernel pk = pair_kernel(k == 2, k == 1);
            e = cudaFuncSetAttribute(pk, cudaFuncAttributeMaxDynamicSharedMemorySize, mm::kPairSmem);
            if (e != cudaSuccess) return e;
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute attr[2];
            launch_attributes(attr, 2);
            cfg.gridDim = dim3(2, 1, 1);
            cfg.blockDim = dim3(kPairThreads, 1, 1);
            cfg.dynamicSmemBytes = mm::kPairSmem;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int n = 0;
            e = cudaOccupancyMaxActiveClusters(&n, pk, &cfg);
            if (e == cudaSuccess && n < 1) e = cudaErrorInvalidConfiguration;
            if (e != cudaSuccess) return e;
            c.pairs = k == 0 ? n : std::min(c.pairs, n);
        }
        int *one = c.clusters[0], *two = c.clusters[1];
        one[1] = c.sms;
        for (int split = 2; split <= kMaxSplit; ++split) {
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute attr[2];
            launch_attributes(attr, static_cast<unsigned>(split));
            cfg.gridDim = dim3(static_cast<unsigned>(split), 1, 1);
            cfg.blockDim = dim3(kSmallThreads, 1, 1);
            cfg.dynamicSmemBytes = kSmallSmemMax;
            cfg.attrs = attr;
            cfg.numAttrs = 2;
            e = cudaOccupancyMaxActiveClusters(&one[split], small_kernel(128, false), &cfg);
            if (e != cudaSuccess) return e;
        }
        // Two CTAs on an SM: as half as many alone (the runtime's answer counts one for kernels
        // with tensor memory).
        for (int split = 2; split <= kMaxSplit; ++split) {
            const int half = (split + 1) / 2;
            two[split] = one[half] * 2 * half / split;
        }
        cached[device] = c;
    }
    *out = cached[device];
    return cudaSuccess;
}

bool e4m3_map(CUtensorMap *m, const void *p, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
    return gemm::make_tile_map(m, p, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, cols, rows, ld, 128, box_rows);
}

// How a forward product is run.
struct Plan {
    bool pair;
    int bn, split, per_sm, per_stage, stages;
    int part, factors, table, bar, smem;  // small: where its shared memory's parts start, and its size
    double clocks;                        // estimate
};

bool small_layout(const Fwd &f, int bn, int split, int per_sm, int per_stage, Plan *p) {
    const int chunk = kSmallWBytes + bn * 128;
    const int part = split > 1 ? (bn + split - 1) / split * split * 512 : 0;
    const int factors = kSmallFactors + kFactorBarBytes;
    const int table = static_cast<int>(round_up(table_bytes(static_cast<int>(f.groups)), 16));
    const int budget = kSmSmem / per_sm - kSmemReserved;
    const int fixed = 1024 + part + factors + table + kSmallTail;
    const int64_t chunks = (f.K + 127) / 128;
    p->pair = false;
    p->bn = bn;
    p->split = split;
    p->per_sm = per_sm;
    p->per_stage = per_stage;
    p->stages = std::min((budget - fixed) / (per_stage * chunk), kMaxStages);
    if (p->stages < 2 || split > chunks || (per_sm > 1 && bn > 2 * kSmallTwoNc)) return false;
    p->part = p->stages * per_stage * chunk;
    p->factors = p->part + part;
    p->table = p->factors + factors;
    p->bar = p->table + table;
    p->smem = std::max(p->bar + kSmallTail + 1024, kSmallBufs * bn * kSmemPerTmemCol - kSmemReserved);
    p->smem = std::max(p->smem, least_smem(per_sm));
    return true;
}

int64_t groups_used(const Fwd &f) { return f.offsets ? std::min(f.groups, f.T) : 1; }

// Estimates in SM clocks at 1.9 GHz, from sweeps on GB300 of every bn, split, per_sm and
// per_stage over 49 products (T = 1 .. 22252, dense and of 4 .. 128 experts): the chosen plan
// is within 10 % of the fastest, 1.5 % on average.  All of them had weights with a scale for
// 128 rows: a pair tile's block takes half as long again with one for each row
// (mm_block_pair.cuh), which the estimate does not know.  A block costs an SM kSmallBlock[bn] clocks
// (of a pair tile kPairBlock) and the weights come from HBM at 6.8 TB/s at best.  Where a
// group's rows are known on the device only, a group takes kGroupTail tiles more than its
// average.  Two CTAs per SM are for tiles of few rows (us with two and with one: T 512, 32
// experts, K 4096, N 4096 in tiles of 16 93 and 107, T 2048, 64 experts, N 2048 in tiles of 32
// 102 and 140), two blocks a stage wherever there are two (the latter 102 and 107).
constexpr double kHbmBytesPerClock = 3570.;
constexpr double kSmallBlock[4] = {315., 490., 820., 1270.}, kPairBlock = 1140.;
constexpr double kLoneCta = 1.35;  // one CTA on an SM that could take two
constexpr double kSmallCta = 5700., kPairCta = 9300., kSplitSync = 1240., kSplitRow = 40., kGroupTail = 0.45;

Plan choose(const Fwd &f, const Capacity &cap) {
    const int64_t used = groups_used(f);
    const double rows = static_cast<double>(f.T) / static_cast<double>(used);  // of a group
    const int64_t chunks = (f.K + 127) / 128;
    const double hbm = static_cast<double>(used) * f.N * f.K / kHbmBytesPerClock;
    auto tiles_of = [&](int step, int64_t across) {
        const double down = f.offsets ? std::max(1., rows / step + kGroupTail) * used
                                      : static_cast<double>((f.T + step - 1) / step);
        return down * static_cast<double>(across);
    };
    auto joined = [&](double own) { return std::sqrt(std::hypot(own * own, hbm * hbm)); };
    Plan best = {};
    best.pair = true;
    best.clocks = joined(std::ceil(tiles_of(256, (f.N + kPairN - 1) / kPairN) / cap.pairs) *
                         chunks * kPairBlock) + kPairCta;
    for (int i = 0; i < 4; ++i) {
        const int bn = kBns[i], per_sm = bn <= 2 * kSmallTwoNc ? kMaxPerSm : 1;
        const double tiles = tiles_of(bn, (f.N + 127) / 128);
        if (tiles > 1e6) continue;  // pair tiles
        for (int split = 1; split <= kMaxSplit && split <= chunks; ++split) {
            const double ctas = tiles * split;
            // A shared tile is a cluster's only one, so a second wave starts from nothing (T
            // 128, K 4096, N 12288 in three parts 49.6 us, whole 23.4), and fewer clusters of
            // eight fit than eighths of the SMs (T 1017, K 7664, N 108: 16 clusters of eight
            // 19.0 us, of six 11.6).
            if (split > 1 && tiles > cap.clusters[per_sm - 1][split]) continue;
            const int64_t each = (chunks + split - 1) / split;
            const int at_once = ctas <= cap.sms ? 1 : per_sm;
            const double own = std::ceil(ctas / (cap.sms * at_once)) * at_once * each * kSmallBlock[i] *
                               (at_once < per_sm ? kLoneCta : 1.);
            const double clocks = joined(own) + kSmallCta + (split > 1 ? kSplitSync + kSplitRow * bn : 0.);
            Plan p = {};
            if (clocks < best.clocks && small_layout(f, bn, split, per_sm, each >= 2 ? 2 : 1, &p)) {
                best = p;
                best.clocks = clocks;
            }
        }
    }
    return best;
}

cudaError_t forward_small(const Fwd &f, const Capacity &cap, const Plan &plan, cudaStream_t s) {
    CUtensorMap mw, mx;
    if (!e4m3_map(&mw, f.w, f.groups * f.N, f.K, f.w_ld, 128) ||
        !e4m3_map(&mx, f.x, f.T, f.K, f.x_ld, plan.bn))
        return cudaErrorInvalidValue;
    SmallParams p = {};
    p.offsets = f.offsets;
    p.xs = f.xs;
    p.ws = f.ws;
    p.xs_ld = f.xs_ld;
    p.ws_ld = f.ws_ld;
    p.residual = f.residual;
    p.residual_ld = f.residual_ld;
    p.y = f.y;
    p.y_ld = f.y_ld;
    p.T = static_cast<int>(f.T);
    p.N = static_cast<int>(f.N);
    p.groups = static_cast<int>(f.groups);
    p.block = f.block;
    p.scale_rows = static_cast<int>((f.N + f.block - 1) / f.block);
    p.nt = static_cast<int>((f.N + 127) / 128);
    p.chunks = static_cast<int>((f.K + 127) / 128);
    p.split = plan.split;
    p.stages = plan.stages;
    p.per_stage = plan.per_stage;
    p.part_offset = plan.part;
    p.factor_offset = plan.factors;
    p.table_offset = plan.table;
    p.bar_offset = plan.bar;
    p.f16 = f.f16;
    p.err = f.err ? f.err : cap.errors;
    const int64_t most = p.nt * (f.offsets ? f.T / plan.bn + groups_used(f) : (f.T + plan.bn - 1) / plan.bn);
    if (most * plan.split > INT32_MAX) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    launch_attributes(attr, static_cast<unsigned>(plan.split));
    cfg.gridDim = dim3(static_cast<unsigned>(plan.split > 1 ? most * plan.split : std::min<int64_t>(most, cap.sms * plan.per_sm)),
                       1, 1);
    cfg.blockDim = dim3(kSmallThreads, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(plan.smem);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, small_kernel(plan.bn, f.residual != nullptr), static_cast<const CUtensorMap>(mw),
                              static_cast<const CUtensorMap>(mx), static_cast<const SmallParams>(p));
}

cudaError_t launch_pair(PairKernel k, const PairMaps &maps, const PairParams &p, int64_t tiles,
                        const Capacity &cap, cudaStream_t s) {
    if (tiles > INT32_MAX / kPairGroupM) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    launch_attributes(attr, 2);
    cfg.gridDim = dim3(static_cast<unsigned>(2 * std::min<int64_t>(tiles, cap.pairs)), 1, 1);
    cfg.blockDim = dim3(kPairThreads, 1, 1);
    cfg.dynamicSmemBytes = mm::kPairSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k, maps, p);
}

// (A TMA store fills a row's last 16 bytes, so the map ends with the last whole ones.)
bool output_map(CUtensorMap *m, const void *p, int64_t rows, int64_t cols, int64_t ld) {
    return gemm::make_tile_map(m, p, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, cols & ~int64_t{7}, rows, ld, 64, 32);
}

cudaError_t forward_pair(const Fwd &f, const Capacity &cap, cudaStream_t s) {
    PairMaps maps = {};
    PairParams p = {};
    p.vec = mm::vec_of(f.y, f.y_ld, f.N);
    if (!e4m3_map(&maps.a, f.x, f.T, f.K, f.x_ld, mm::kHalfRows) ||
        !e4m3_map(&maps.b, f.w, f.groups * f.N, f.K, f.w_ld, kPairN / 2) ||
        (p.vec >= 16 && !output_map(&maps.y, f.y, f.T, f.N, f.y_ld)))
        return cudaErrorInvalidValue;
    p.offsets = f.offsets;
    p.as = f.xs;
    p.bs = f.ws;
    p.as_ld = f.xs_ld;
    p.bs_ld = f.ws_ld;
    p.residual = f.residual;
    p.residual_ld = f.residual_ld;
    p.y = f.y;
    p.y_ld = f.y_ld;
    p.T = static_cast<int>(f.T);
    p.N = static_cast<int>(f.N);
    p.groups = static_cast<int>(f.groups);
    p.scale_rows = static_cast<int>((f.N + f.block - 1) / f.block);
    p.nt = static_cast<int>((f.N + kPairN - 1) / kPairN);
    p.chunks = static_cast<int>((f.K + 127) / 128);
    p.out = f.f16 ? VLMCE_F16 : VLMCE_BF16;
    p.err = f.err ? f.err : cap.errors;
    const int64_t most = p.nt * (f.offsets ? f.T / 256 + groups_used(f) : (f.T + 255) / 256);
    return launch_pair(pair_kernel(false, f.block == 1), maps, p, most, cap, s);
}

}  // namespace

cudaError_t forward(const Fwd &f, cudaStream_t s) {
    Capacity cap;
    const cudaError_t e = setup(&cap);
    if (e != cudaSuccess) return e;
    const Plan plan = choose(f, cap);
    return plan.pair ? forward_pair(f, cap, s) : forward_small(f, cap, plan, s);
}

cudaError_t describe(const Fwd &f, int32_t *out) {
    Capacity cap;
    const cudaError_t e = setup(&cap);
    if (e != cudaSuccess) return e;
    const Plan plan = choose(f, cap);
    out[0] = plan.pair ? 0 : 1;
    out[1] = plan.pair ? 256 : plan.bn;
    out[2] = plan.pair ? 1 : plan.split;
    out[3] = plan.pair ? 1 : plan.per_stage;
    return cudaSuccess;
}

cudaError_t dweight(const Dw &d, cudaStream_t s) {
    Capacity cap;
    const cudaError_t e = setup(&cap);
    if (e != cudaSuccess) return e;
    PairMaps maps = {};
    PairParams p = {};
    const bool f32 = d.dtype == VLMCE_F32;
    p.vec = f32 ? (aligned(d.dw, 16) && d.K % 4 == 0 ? 16 : 2) : mm::vec_of(d.dw, d.K, d.K);
    if (!e4m3_map(&maps.a, d.dyt, d.N, d.R, d.dyt_ld, mm::kHalfRows) ||
        !e4m3_map(&maps.b, d.xt, d.K, d.R, d.xt_ld, kPairN / 2) ||
        (p.vec >= 16 && !(f32 ? gemm::make_stack_map(&maps.y, d.dw, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, d.K, d.N,
                                                     d.groups, d.K, 32, 32)
                              : output_map(&maps.y, d.dw, d.groups * d.N, d.K, d.K))))
        return cudaErrorInvalidValue;
    p.offsets = d.offsets;
    p.as = d.dyts;
    p.bs = d.xts;
    p.as_ld = d.dyts_ld;
    p.bs_ld = d.xts_ld;
    p.y = d.dw;
    p.y_ld = d.K;
    p.T = static_cast<int>(d.R);
    p.N = static_cast<int>(d.N);
    p.groups = static_cast<int>(d.groups);
    p.K = static_cast<int>(d.K);
    p.nt = static_cast<int>((d.K + kPairN - 1) / kPairN);
    p.mt = static_cast<int>((d.N + 255) / 256);
    p.out = d.dtype;
    p.add = d.accumulate;
    p.err = d.err ? d.err : cap.errors;
    const int64_t tiles = d.groups * p.mt * static_cast<int64_t>(p.nt);
    return launch_pair(pair_kernel(true, true), maps, p, tiles, cap, s);
}

}  // namespace mmb
}  // namespace vlmce
