// mbar_wait.cuh -- bounded waits on mbarriers, shared by the kernels that run
// as warp-specialised pipelines.  A wait that gives up (kWaitLimitNs) sets
// VLMCE_DEVERR_TIMEOUT in the device error word and the CTA's abort flag,
// after which its other waits return at once, so a launch always ends (its
// results are invalid: whoever launches a kernel passes a word that is read).
#pragma once

#include <cstdint>

#include "ptx.cuh"
#include "vlmce.h"

namespace vlmce {

constexpr unsigned long long kWaitLimitNs = 4000000000ull;

template <bool CLUSTER_ACQUIRE = false>
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int *abort,
                                         int *err, unsigned long long limit_ns = kWaitLimitNs) {
    auto try_once = [&] {
        return CLUSTER_ACQUIRE ? ptx::mbar_try_wait_cluster(bar, parity)
                               : ptx::mbar_try_wait(bar, parity);
    };
    if (try_once()) return true;
    if (*abort) return false;
    const unsigned long long t0 = ptx::globaltimer_ns();
    for (;;) {
        for (int i = 0; i < 64; ++i)
            if (try_once()) return true;
        if (*abort) return false;
        if (ptx::globaltimer_ns() - t0 > limit_ns) {
            *abort = 1;
            if (err) atomicOr(err, VLMCE_DEVERR_TIMEOUT);
            return false;
        }
    }
}
// Same, but never skipped: used where copies or MMAs may still be in flight.
__device__ __forceinline__ void drain_bar(uint32_t bar, uint32_t parity, int *err) {
    volatile int no_abort = 0;
    wait_bar(bar, parity, &no_abort, err);
}

}  // namespace vlmce
