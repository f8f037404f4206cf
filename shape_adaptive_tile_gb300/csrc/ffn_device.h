// The device that the feed-forward operators run on.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

#include "gemm.h"
#include "registry.h"

namespace sat {
namespace ffn {

// The current device's SMs, or a status.
inline int device_sms(int* sms)
{
    static std::atomic<int> known[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return fail_with(GEMM_ERR_LAUNCH, "querying the device: %s", cudaGetErrorString(e));
    int n = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        int major = 0, minor = 0;
        e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
        if (e == cudaSuccess)
            e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
        if (e == cudaSuccess)
            e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess)
            return fail_with(GEMM_ERR_LAUNCH, "querying the device: %s", cudaGetErrorString(e));
        if (major != 10 || minor != 3)
            return fail_with(GEMM_ERR_ARCH, "device %d is compute capability %d.%d; this library is built for sm_103a only",
                             dev, major, minor);
        if (dev < 64)
            known[dev].store(n, std::memory_order_relaxed);
    }
    *sms = n;
    return GEMM_OK;
}

}  // namespace ffn
}  // namespace sat
