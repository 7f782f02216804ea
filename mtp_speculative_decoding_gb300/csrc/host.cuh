// host.cuh -- host helpers shared by the ABI's translation units (internal).
#pragma once

#include <cudaTypedefs.h>
#include <cuda_runtime.h>

namespace mtp {

// SM count of the current device (cached per device), 0 on an error
int num_sms();
// cuTensorMapEncodeTiled from the driver, resolved once; null if it cannot be had
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();
// The encoder wants a current context, which a host thread that has made no CUDA call
// yet lacks: the device's is made current then.
template <typename F>
bool encoded(F&& encode) {
    if (encode() == CUDA_SUCCESS) return true;
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && encode() == CUDA_SUCCESS;
}

}  // namespace mtp
