// Tensor maps (kv_async.cuh).
#include "kv_async.cuh"

namespace kvimpl {

bool cache_map(CUtensorMap* map, const void* cache, int elem_bytes, bool bf16, int64_t row, int64_t page_size, int64_t heads,
               int64_t pages, int64_t slot_stride, int64_t head_stride, int64_t page_stride, int width, int keys, int box_heads,
               bool swizzle) {
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
  if (page_size == 1) slot_stride = 16;  // the stride of a dimension of one is never used, but checked
  if (heads == 1) head_stride = 16;
  if (pages == 1) page_stride = 16;
  for (int64_t s : {slot_stride, head_stride, page_stride})
    if (s <= 0 || s >= (int64_t{1} << 40) || (s & 15) != 0) return false;
  const int bytes = width * elem_bytes;
  if ((bytes & 15) != 0 || (reinterpret_cast<uintptr_t>(cache) & 15u) != 0) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(row), static_cast<cuuint64_t>(page_size), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(slot_stride), static_cast<cuuint64_t>(head_stride),
                                 static_cast<cuuint64_t>(page_stride)};
  const cuuint32_t boxes[4] = {static_cast<cuuint32_t>(width), static_cast<cuuint32_t>(keys), static_cast<cuuint32_t>(box_heads), 1u};
  const cuuint32_t ones[4] = {1u, 1u, 1u, 1u};
  const CUtensorMapSwizzle sw = !swizzle || bytes < 64 ? CU_TENSOR_MAP_SWIZZLE_NONE
                                : bytes == 64          ? CU_TENSOR_MAP_SWIZZLE_64B
                                                       : CU_TENSOR_MAP_SWIZZLE_128B;
  const CUtensorMapDataType type = elem_bytes == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : bf16          ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                   : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return encode(map, type, 4, const_cast<void*>(cache), dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace kvimpl
