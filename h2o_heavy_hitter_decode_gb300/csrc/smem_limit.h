// smem_limit.h — a kernel's limit of dynamic shared memory (host code).
#pragma once

#include <cuda_runtime_api.h>

#include <atomic>
#include <mutex>

namespace h2o {
namespace blk {

// A kernel's limit of dynamic shared memory, raised for each device to the
// most that any launch so far has wanted and never lowered: what is wanted
// depends on the cache, and host threads with caches of their own launch the
// same kernel.  The call costs a microsecond, so a launch that needs no more
// than an earlier one makes none; the lock keeps one thread's smaller limit
// from replacing another's larger one between its setting and its record.
struct SmemLimit {
  static constexpr int kDevices = 64;
  std::atomic<int> bytes[kDevices] = {};
  std::mutex raising;
  cudaError_t raise(const void *kernel, int want) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
    if (bytes[dev].load(std::memory_order_acquire) >= want) return cudaSuccess;
    std::lock_guard<std::mutex> lock(raising);
    if (bytes[dev].load(std::memory_order_relaxed) >= want) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, want);
    if (e == cudaSuccess) bytes[dev].store(want, std::memory_order_release);
    return e;
  }
};

}  // namespace blk
}  // namespace h2o
