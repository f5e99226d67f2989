// Host helpers shared by the entry points' translation units; internal.
#pragma once

#include <cuda_runtime.h>

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

}  // namespace bconv
