// Raising a kernel's dynamic shared memory limit once per device.
#pragma once

#include <atomic>

#include <cuda_runtime.h>

namespace moda {

// Raises a kernel's dynamic shared memory limit once per device (the call
// costs more than a launch). A device reset in between is noticed by the
// launch, which then fails; the attribute is set again on the next call.
struct SmemLimit {
    std::atomic<unsigned long long> done{0};
    cudaError_t raise(const void* kernel, int bytes) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const unsigned long long bit = 1ull << (dev & 63);
        if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
        return e;
    }
};

}  // namespace moda
