// smem_limit.h -- dynamic shared memory above 48 KB for a kernel, allowed once on each device.
#pragma once

#include <cuda_runtime_api.h>

#include <atomic>
#include <cstdint>

namespace mm {

// The limit holds for the device that is current when it is set, so what has been done is kept by device (a bit each;
// the library takes ordinals below 64) and only if it succeeded: a failure is tried again by the next call.
class SmemLimit {
    std::atomic<uint64_t> done_{0};

public:
    cudaError_t allow(const void *kernel, int bytes) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const uint64_t bit = (uint64_t)1 << (dev & 63);
        if (done_.load(std::memory_order_relaxed) & bit) return cudaSuccess;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess) done_.fetch_or(bit, std::memory_order_relaxed);
        return e;
    }
};

}  // namespace mm
