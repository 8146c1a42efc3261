// A wait on a barrier that nothing arrives at: it ends by itself, and the record says so.
#include <cstdio>

#include "kv_async.cuh"
#include "kv_device.cuh"

using namespace kvimpl;

__global__ void two_waits(kv_error_record* err, int* passed) {
  __shared__ __align__(8) uint64_t barrier[2];
  __shared__ WaitState waits;
  const uint32_t bar = static_cast<uint32_t>(__cvta_generic_to_shared(barrier));
  if (threadIdx.x == 0) {
    bar_init(bar, 1);
    bar_init(bar + 8, 1);
    waits = WaitState{0, 0};
  }
  __syncthreads();
  const int warp = static_cast<int>(threadIdx.x >> 5);
  bool ok = true;
  if (warp == 1 && threadIdx.x == 32) bar_arrive(bar + 8);
  if (warp == 0) ok = __all_sync(0xFFFFFFFFu, bar_wait(bar + 8, 0u, &waits));  // arrived at: passes
  if (threadIdx.x == 0) passed[0] = ok;
  ok = __all_sync(0xFFFFFFFFu, bar_wait(bar, 0u, &waits));                      // both warps: runs out
  if ((threadIdx.x & 31u) == 0u) passed[1 + warp] = ok;
  __syncthreads();
  if (threadIdx.x == 0 && waits.ran_out()) record_wait(err);
}

int main() {
  kv_error_record* err;
  int* passed;
  if (cudaMallocManaged(&err, sizeof *err) != cudaSuccess || cudaMallocManaged(&passed, 3 * sizeof(int)) != cudaSuccess) return 2;
  *err = kv_error_record{3, ~uint64_t{5}};
  for (int i = 0; i < 3; ++i) passed[i] = -1;
  two_waits<<<1, 64>>>(err, passed);
  const cudaError_t e = cudaDeviceSynchronize();
  printf("%s %d %d %d %d %llu\n", cudaGetErrorString(e), passed[0], passed[1], passed[2], (err->oob_count & KV_ERROR_WAIT_BIT) != 0,
         static_cast<unsigned long long>(err->oob_count & ~KV_ERROR_WAIT_BIT));
  return e == cudaSuccess ? 0 : 1;
}
