// What the C entry points in api.cu and api_serve.cu share.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>

#include "w4a16.h"

namespace w4a16 {

struct DeviceInfo {
    int sms;
    int* status;              // the library's error word for kernels without a workspace
    long long wait_limit_ns;  // limit of the kernels' bounded waits
};

// The status of a CUDA call, its code kept for w4a16_last_cuda_error().
w4a16_status report_cuda(cudaError_t e);
// The current device, checked to be sm_103, with every kernel's attributes set.
w4a16_status device_info(DeviceInfo* info);
// Attributes of the serving step's kernels, those over caches of 4 and 8 bits, set with the matmuls'.
cudaError_t setup_kv4();
// The library's own workspace on the current device.
w4a16_status library_workspace(void** ws, size_t* bytes);

// Layout of every workspace: error word at 0, one counter per CTA, partial sums.
constexpr size_t kWsCountersOff = 256;
constexpr int kWsMaxGrid = 1024;
constexpr size_t kWsPartialsOff = kWsCountersOff + 4 * kWsMaxGrid;

}  // namespace w4a16
