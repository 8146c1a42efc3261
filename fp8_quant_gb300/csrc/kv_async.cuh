// Barriers in shared memory and TMA boxes of a paged cache.
#pragma once

#include <cuda.h>  // CUtensorMap
#include <cuda_runtime.h>

#include <cstdint>

namespace kvimpl {

// Tries of a wait, of 2 us and more each: 2 to 4 s, where no warp's work between two barriers takes a
// millisecond but on rows done key by key and page tables gone through, for which waits stand still (WaitState).
constexpr uint32_t kSpin = 1u << 20;

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Arrives and expects `bytes` more of this phase by TMA.
__device__ __forceinline__ void bar_arrive_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// Arrives when all of this thread's cp.async so far have landed.
__device__ __forceinline__ void bar_arrive_copies(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void wait_all_async() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// A box of a cache: (dim or byte, key in its page, head, page).
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t dim, int32_t key,
                                        int32_t head, int32_t page) {
  asm volatile("cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];"
               ::"r"(dst), "l"(map), "r"(bar), "r"(dim), "r"(key), "r"(head), "r"(page) : "memory");
}

__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\t"
               "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
               "selp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0u;
}

// A CTA's waits, in shared memory.
struct WaitState {
  int failed;  // a wait ran out
  int held;    // warps at work that may take any time (a row's keys one by one): tries are not counted meanwhile

  __device__ __forceinline__ bool ran_out() const { return *const_cast<const volatile int*>(&failed) != 0; }
  __device__ __forceinline__ void hold(int more) { atomicAdd(&held, more); }
};

// False when the wait ran out here or anywhere in the CTA.  kApart: the first try stands before the loop, as
// most waits end there (one prompt of 8,192 fp16 tokens 415 us, 420 without; 4-bit decode 401 and
// 410; but 4-bit chunks in the tile kernel 161 and 150, so its quantised forms do without).
template <bool kApart = true>
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, WaitState* state) {
  if (kApart && bar_try(bar, parity)) return true;
#pragma unroll 1
  for (uint32_t i = 0; i < kSpin; ++i) {
    if (bar_try(bar, parity)) return true;
    if ((i & 1023u) == 1023u) {
      if (state->ran_out()) return false;
      if (*const_cast<volatile int*>(&state->held) != 0) i = 0;
    }
  }
  *const_cast<volatile int*>(&state->failed) = 1;
  return false;
}

__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// The tensor map of a cache: rows of `row` elements of `elem_bytes` (2: 16-bit floats, 1: bytes), a box
// being `width` elements x `keys` x `heads` of one page, laid out in that order, rows of 128, 64 or
// 32 bytes in the swizzle of their length.  False where there is none: a stride that TMA does
// not take (it wants positive multiples of 16 bytes below 2^40).
bool cache_map(CUtensorMap* map, const void* cache, int elem_bytes, bool bf16, int64_t row, int64_t page_size, int64_t heads,
               int64_t pages, int64_t slot_stride, int64_t head_stride, int64_t page_stride, int width, int keys, int box_heads,
               bool swizzle);

// The tensor map of a cache of latent rows: (dim of a chunk or of the row, key of a group of eight, chunk, group of its page,
// page), boxes of `groups` groups whose keys lie as [group][chunk][key][64 elements]. With box_chunks 1 dims are the row's, so
// that those behind it are zeros. False where there is none (strides are positive multiples of 16 bytes below 2^40).
bool latent_map(CUtensorMap* map, const void* cache, int elem_bytes, bool bf16, int64_t row, int64_t page_size, int64_t pages,
                int64_t slot_stride, int64_t page_stride, int chunks, int box_chunks, int groups, bool swizzle);

}  // namespace kvimpl
