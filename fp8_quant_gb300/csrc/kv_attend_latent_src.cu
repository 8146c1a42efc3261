// The tensor-core attention kernels (kv_attend_latent_tile.cuh) of 16-bit latent rows.
#include "kv_attend_latent_tile.cuh"

namespace kvimpl {

kv_status latent_tile_src(const LatentTileParams& p, bool few, void* work, int64_t work_bytes, int64_t max_keys, cudaStream_t stream) {
  if (p.l.a.bf16)
    return few ? launch_latent_tile<KV_CACHE_SRC, 32, true>(p, work, work_bytes, max_keys, stream)
               : launch_latent_tile<KV_CACHE_SRC, 64, true>(p, work, work_bytes, max_keys, stream);
  return few ? launch_latent_tile<KV_CACHE_SRC, 32, false>(p, work, work_bytes, max_keys, stream)
             : launch_latent_tile<KV_CACHE_SRC, 64, false>(p, work, work_bytes, max_keys, stream);
}

}  // namespace kvimpl
