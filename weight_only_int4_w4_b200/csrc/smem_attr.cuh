// smem_attr.cuh -- the attribute that dynamic shared memory above 48 KiB needs.  Host code only.
#pragma once

#include <cuda_runtime_api.h>

#include <atomic>
#include <mutex>

namespace w4 {

// Dynamic shared memory above 48 KiB needs a per-function attribute on every
// device; setting it is a driver call, so it is made once per (function, device)
// and size, tracked in `set` (one slot per device ordinal).  Sizes only grow: with
// two threads at it, a smaller size set last would fail every launch of the larger
// one, which `set` says is in force.
constexpr int kAttrDevices = 64;
inline cudaError_t ensure_smem_attr(const void *func, int bytes, std::atomic<int> (&set)[kAttrDevices]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < kAttrDevices && set[dev].load(std::memory_order_relaxed) >= bytes) return cudaSuccess;
  static std::mutex lock;
  std::lock_guard<std::mutex> hold(lock);
  if (dev >= 0 && dev < kAttrDevices && set[dev].load(std::memory_order_relaxed) >= bytes) return cudaSuccess;
  e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev >= 0 && dev < kAttrDevices) set[dev].store(bytes, std::memory_order_relaxed);
  return e;
}

}  // namespace w4
