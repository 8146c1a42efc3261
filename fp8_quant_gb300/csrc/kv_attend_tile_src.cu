// The tensor-core attention kernels (kv_attend_tile.cuh) of 16-bit caches.
#include "kv_attend_tile.cuh"

namespace kvimpl {

bool tile_map(CUtensorMap* map, const void* cache, bool bf16, int head_dim, int heads, int64_t page_size, int64_t pages,
              int64_t head_stride, int64_t slot_stride, int64_t page_stride, int box) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      (void)cudaGetLastError();
      return static_cast<Encode>(nullptr);
    }
    return reinterpret_cast<Encode>(f);
  }();
  if (!encode) return false;
  if (heads == 1) head_stride = 16;  // never used, but checked
  if (pages == 1) page_stride = 16;
  const int64_t most = int64_t{1} << 40;
  for (int64_t s : {head_stride, slot_stride, page_stride})
    if (s <= 0 || s >= most || (s & 15) != 0) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(page_size), static_cast<cuuint64_t>(pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(head_stride), static_cast<cuuint64_t>(slot_stride),
                                 static_cast<cuuint64_t>(page_stride)};
  const cuuint32_t boxes[4] = {64u, 1u, static_cast<cuuint32_t>(box), 1u}, ones[4] = {1u, 1u, 1u, 1u};
  return encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void*>(cache),
                dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

kv_status tile_src(const TileParams& p, cudaStream_t stream) {
  if (p.a.bf16)
    return p.a.head_dim <= 64 ? launch_tile<KV_CACHE_SRC, 64, true>(p, stream)
                              : launch_tile<KV_CACHE_SRC, 128, true>(p, stream);
  return p.a.head_dim <= 64 ? launch_tile<KV_CACHE_SRC, 64, false>(p, stream)
                            : launch_tile<KV_CACHE_SRC, 128, false>(p, stream);
}

}  // namespace kvimpl
