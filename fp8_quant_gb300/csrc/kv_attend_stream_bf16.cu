// The TMA-fed attention kernels (kv_attend_stream.cuh) of one cache format.
#include "kv_attend_stream.cuh"

namespace kvimpl {

kv_status stream_bf16(const StreamParams& p, bool wide, void* work, int64_t work_bytes, int64_t max_keys,
                      cudaStream_t stream) {
  return launch_stream_fmt<KV_CACHE_SRC, true>(p, wide, work, work_bytes, max_keys, stream);
}

}  // namespace kvimpl
