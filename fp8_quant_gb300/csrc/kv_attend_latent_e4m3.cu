// The tensor-core attention kernels (kv_attend_latent_tile.cuh) of e4m3fn latent rows.
#include "kv_attend_latent_tile.cuh"

namespace kvimpl {

kv_status latent_tile_e4m3(const LatentTileParams& p, bool few, void* work, int64_t work_bytes, int64_t max_keys, cudaStream_t stream) {
  return few ? launch_latent_tile<KV_CACHE_E4M3FN, 32, false>(p, work, work_bytes, max_keys, stream)
             : launch_latent_tile<KV_CACHE_E4M3FN, 64, false>(p, work, work_bytes, max_keys, stream);
}

}  // namespace kvimpl
