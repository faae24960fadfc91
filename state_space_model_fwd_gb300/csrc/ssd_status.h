// ssd_status.h -- the device status word of the library (ssd_api.cu).
#pragma once

#include <cuda_runtime.h>

namespace ssd {

// The current device's word into which kernels latch failures (bit 0: a bounded wait gave up).
cudaError_t device_status_word(unsigned **out);

}  // namespace ssd
