// Raising a kernel's dynamic shared memory limit once per context.
#pragma once

#include <atomic>

#include <cuda_runtime.h>

#include "context_id.h"

namespace moda {

// Raises a kernel's dynamic shared memory limit once per device and context
// (the call costs more than a launch). A new context, as after cudaDeviceReset,
// loads the kernel again with the default limit, so each device's entry
// remembers the context that it was raised in.
class SmemLimit {
  public:
    cudaError_t raise(const void* kernel, int bytes) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
        unsigned long long id = 0;
        if (current_context_id(&id) && raised_[dev].load(std::memory_order_acquire) == id + 1) return cudaSuccess;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        // (the context exists now even if it did not before the call)
        if (e == cudaSuccess && current_context_id(&id)) raised_[dev].store(id + 1, std::memory_order_release);
        return e;
    }

  private:
    static constexpr int kMaxDevices = 64;
    std::atomic<unsigned long long> raised_[kMaxDevices] = {};  // id + 1 of the context, 0: none
};

}  // namespace moda
