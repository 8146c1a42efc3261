// What the kernels of a cache of latent rows share on the host.
#pragma once

#include "kv_host.h"

namespace kvimpl {

constexpr int32_t kMaxRow = 1024;  // dims of a latent row

// KV_OK where CUDA knows every pointer and device memory is the current device's.
inline kv_status classify_here(const void* const* ptrs, int n) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  for (int i = 0; i < n; ++i) {
    cudaPointerAttributes a;
    e = cudaPointerGetAttributes(&a, ptrs[i]);
    if (e != cudaSuccess) {
      (void)cudaGetLastError();  // the query's own error is not sticky: clear it
      return cuda_fail(e);
    }
    if (a.type == cudaMemoryTypeUnregistered || (a.type == cudaMemoryTypeDevice && a.device != dev)) return KV_ERR_INVALID_ARG;
  }
  return KV_OK;
}

}  // namespace kvimpl
