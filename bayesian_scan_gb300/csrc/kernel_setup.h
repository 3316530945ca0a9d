// kernel_setup.h -- a kernel's dynamic shared memory, set up once per device.
#pragma once
#include <cuda_runtime.h>

#include <mutex>
#include <set>
#include <utility>

namespace kdn {

// Raises the limit of `kernel` on the current device to `bytes` (the same for
// every call with this kernel).
inline cudaError_t allow_smem(const void* kernel, size_t bytes) {
    static std::mutex lock;
    static std::set<std::pair<int, const void*>> done;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    try {   // no exception leaves a C entry point
        const std::lock_guard<std::mutex> hold(lock);
        if (done.count({dev, kernel})) return cudaSuccess;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
        if (e == cudaSuccess) done.insert({dev, kernel});
    } catch (...) {
        return cudaErrorMemoryAllocation;
    }
    return e;
}

}  // namespace kdn
