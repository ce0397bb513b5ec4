// device_errors.h -- where kernels leave VLMCE_DEVERR_* bits when the caller gave
// no error word: one word per device, read by vlmce_take_device_errors.
#pragma once

#include <cuda_runtime.h>

namespace vlmce {

// The current device's word.
cudaError_t device_error_word(int **word);

}  // namespace vlmce
