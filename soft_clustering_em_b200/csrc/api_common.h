// api_common.h -- what the translation units of the C ABI share.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "gmm.h"

namespace scem {

// Status after enqueuing n kernels (counted for gmm_launch_count).
gmm_status api_launched(int n);
// SM count of the current device.
gmm_status api_device_sms(int* sms);
// Nanoseconds after which a device-side wait gives up (gmm_set_wait_budget).
uint64_t api_wait_budget();

// A launch that may start while the kernel before it in the stream ends: the kernel waits
// (grid_dependency_wait) in every block before it touches memory, or, to go on beside the kernel
// before it, acquires what that one has released after such a wait, and waits at its end.
template <typename Kern, typename... Args>
gmm_status api_launch_next(Kern kern, dim3 grid, int threads, size_t smem, cudaStream_t st,
                           Args... args) {
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess)
    return api_launched(0), GMM_ERR_CUDA;
  return api_launched(1);
}

}  // namespace scem
