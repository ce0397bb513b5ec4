// device_errors.cu -- the devices' error words and vlmce_take_device_errors.
#include "device_errors.h"

#include <mutex>

#include "host_util.h"
#include "vlmce.h"

namespace vlmce {
namespace {

__device__ int g_errors;

__global__ void take_errors_kernel(int *word, int32_t *out) { *out = atomicExch(word, 0); }

}  // namespace

cudaError_t device_error_word(int **word) {
    constexpr int kMaxDevices = 64;
    static std::mutex mu;
    static int *cached[kMaxDevices] = {};
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    if (device < 0 || device >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!cached[device]) {
        void *p = nullptr;
        e = cudaGetSymbolAddress(&p, g_errors);
        if (e != cudaSuccess) return e;
        cached[device] = static_cast<int *>(p);
    }
    *word = cached[device];
    return cudaSuccess;
}

}  // namespace vlmce

extern "C" vlmce_status vlmce_take_device_errors(int32_t *out, vlmce_stream_t stream) {
    using namespace vlmce;
    if (!out) return VLMCE_ERR_INVALID_ARG;
    if (!aligned(out, 4)) return VLMCE_ERR_MISALIGNED;
    DeviceInfo dev;
    const vlmce_status st = current_device(&dev);
    if (st != VLMCE_OK) return st;
    int *word = nullptr;
    const cudaError_t e = device_error_word(&word);
    if (e == cudaSuccess)
        take_errors_kernel<<<1, 1, 0, reinterpret_cast<cudaStream_t>(stream)>>>(word, out);
    return launch_status(e, "vlmce_take_device_errors");
}
