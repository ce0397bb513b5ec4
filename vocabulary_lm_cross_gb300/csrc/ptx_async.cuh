// ptx_async.cuh -- inline-PTX wrappers for the decoder-layer kernels, next to
// those of ptx.cuh: per-thread asynchronous copies into shared memory, the two
// halves of a cluster barrier, and cluster launch control.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace vlmce {
namespace ptx {

// The two halves of cluster_sync_any: the arrival, and the wait for every thread's.
__device__ __forceinline__ void cluster_arrive_any() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait_any() {
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// 16 bytes from global to shared memory without a register in between; each
// thread's copies complete in groups (cp_async_wait<N>: all but the last N).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Same, of which only the first `bytes` are read; zeros follow them.
__device__ __forceinline__ void cp_async16_first(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// --------------------------------------------------- cluster launch control
// Ask for a cluster of this grid that has not started yet: it will not be
// launched, and the caller runs its work.  The 16-byte answer goes to `dst` and
// 16 bytes are counted on `bar`, in every CTA of the cluster at these offsets.
__device__ __forceinline__ void clc_try_cancel(uint32_t dst, uint32_t bar) {
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes"
        ".multicast::cluster::all.b128 [%0], [%1];" ::"r"(dst),
        "r"(bar)
        : "memory");
}
// blockIdx.x of the first CTA of the cluster an answer grants, or -1: none left.
__device__ __forceinline__ int clc_first_cta(uint32_t src) {
    uint32_t ok, x;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
        "ld.shared.b128 r, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "mov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, _, _, _}, r;\n\t}"
        : "=r"(ok), "=r"(x)
        : "r"(src)
        : "memory");
    return ok ? static_cast<int>(x) : -1;
}
__device__ __forceinline__ void mbar_remote_arrive_expect_tx(uint32_t remote_bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.release.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(
                     remote_bar),
                 "r"(bytes)
                 : "memory");
}

}  // namespace ptx
}  // namespace vlmce
