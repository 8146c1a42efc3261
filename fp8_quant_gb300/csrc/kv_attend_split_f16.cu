// The key-split attention kernels (kv_attend_split.cuh) of one cache format.
#include "kv_attend_split.cuh"

namespace kvimpl {

kv_status split_f16(const SplitParams& p, bool wide, void* work, int64_t work_bytes, int64_t max_keys,
                   cudaStream_t stream) {
  return launch_split_fmt<KV_CACHE_SRC, false>(p, wide, work, work_bytes, max_keys, stream);
}

}  // namespace kvimpl
