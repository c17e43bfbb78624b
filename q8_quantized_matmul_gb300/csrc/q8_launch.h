// q8_launch.h -- what the launchers set once per kernel and device.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace q8 {

// The devices that a kernel has been allowed its dynamic shared memory on: the attribute belongs to the kernel on
// one device, and a process may use several.
struct SmemAllowed {
    std::atomic<uint64_t> devices{0};
};

// Lets `kernel` be launched with up to `bytes` of dynamic shared memory on the current device; asks the runtime the
// first time there only (a device beyond 63: every time).
inline cudaError_t allow_smem(SmemAllowed &done, const void *kernel, size_t bytes) {
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev >= 0 && dev < 64 ? (uint64_t)1 << dev : 0;
    if (done.devices.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done.devices.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

}  // namespace q8
