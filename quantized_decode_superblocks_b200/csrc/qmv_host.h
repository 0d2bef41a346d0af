// qmv_host.h -- host state of libqmv.so that its translation units share
// (defined in qmv_api.cu): the current device's properties, the CUDA error
// record behind QMV_ERR_CUDA, and the failure-injection hook.
#pragma once

#include <cuda_runtime.h>

namespace qmv {

struct HostDev {
    int sm_count = 0;
    int *err = nullptr;      // device address of the sticky error word
};

// The current device; QMV_OK or QMV_ERR_DEVICE.
__attribute__((visibility("hidden"))) int host_dev(HostDev &out);
// Records e for qmv_last_cuda_error; returns QMV_ERR_CUDA.
__attribute__((visibility("hidden"))) int host_cuda_fail(cudaError_t e);
// Whether the next launch is to fail (qmv_debug_fail_next_launches).
__attribute__((visibility("hidden"))) bool host_injected_failure();

}  // namespace qmv
