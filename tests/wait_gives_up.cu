// A kernel waits, for at most 50 ms, on an mbarrier that nothing arrives on, with the
// error word of calls that were given none.  The launch has to end by itself, mark its
// CTA as aborted (a second wait returns at once) and leave the bit in the word, which
// vlmce_take_device_errors reads and clears.  Prints "wait ok".
#include <cuda_runtime.h>

#include <cstdio>

#include "device_errors.h"
#include "mbar_wait.cuh"
#include "vlmce.h"

__global__ void wait_kernel(int *err, int *out) {
    __shared__ unsigned long long bar;
    __shared__ int abort;
    if (threadIdx.x != 0) return;
    abort = 0;
    const unsigned b = vlmce::ptx::smem_addr(&bar);
    vlmce::ptx::mbar_init(b, 1);
    out[0] = vlmce::wait_bar(b, 0, &abort, err, 50000000ull);
    out[1] = abort;
    const unsigned long long t0 = vlmce::ptx::globaltimer_ns();
    out[2] = vlmce::wait_bar(b, 0, &abort, err, 50000000ull);
    out[3] = vlmce::ptx::globaltimer_ns() - t0 < 25000000ull;
}

#define CHECK(c)                                                \
    do {                                                        \
        if (!(c)) {                                             \
            std::printf("failed: %s, line %d\n", #c, __LINE__); \
            return 1;                                           \
        }                                                       \
    } while (0)

int main() {
    int *word = nullptr, *out = nullptr, *taken = nullptr, h[4], t = -1;
    CHECK(vlmce::device_error_word(&word) == cudaSuccess && word);
    CHECK(cudaMalloc(&out, sizeof h) == cudaSuccess && cudaMalloc(&taken, 4) == cudaSuccess);
    auto take = [&] {
        return vlmce_take_device_errors(taken, nullptr) == VLMCE_OK &&
               cudaMemcpy(&t, taken, 4, cudaMemcpyDeviceToHost) == cudaSuccess;
    };
    CHECK(take() && t == 0);
    wait_kernel<<<1, 32>>>(word, out);
    CHECK(cudaMemcpy(h, out, sizeof h, cudaMemcpyDeviceToHost) == cudaSuccess);
    CHECK(h[0] == 0 && h[1] == 1 && h[2] == 0 && h[3] == 1);
    CHECK(take() && t == VLMCE_DEVERR_TIMEOUT);
    CHECK(take() && t == 0);
    std::printf("wait ok\n");
    return 0;
}
