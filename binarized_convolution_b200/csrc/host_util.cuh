// Host helpers shared by the entry points' translation units; internal.
#pragma once

#include <cuda_runtime.h>

#include <stdint.h>

#include <atomic>

#include "bconv.h"

namespace bconv {

// Makes a device current for a scope and puts the previous one back.
struct DeviceGuard {
  int prev = -1;
  bool ok = true;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) {
      ok = false;
      return;
    }
    if (prev != dev && cudaSetDevice(dev) != cudaSuccess) ok = false;
  }
  ~DeviceGuard() {
    int cur = -1;
    if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
  }
};

inline bconv_status_t from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return BCONV_OK;
  if (e == cudaErrorMemoryAllocation) return BCONV_ERR_OOM;
  if (e == cudaErrorNoDevice || e == cudaErrorInsufficientDriver) return BCONV_ERR_NO_DEVICE;
  return BCONV_ERR_CUDA;
}

// Lets the current device run Kern with `bytes` (a constant of the call site) of dynamic shared memory; asked of the
// runtime once per device.
template <auto Kern>
cudaError_t allow_smem(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t{1} << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

}  // namespace bconv
