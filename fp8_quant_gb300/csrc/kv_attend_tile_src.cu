// The tensor-core attention kernels (kv_attend_tile.cuh) of 16-bit caches.
#include "kv_attend_tile.cuh"

namespace kvimpl {

kv_status tile_src(const TileParams& p, cudaStream_t stream) {
  if (p.a.bf16)
    return p.a.head_dim <= 64 ? launch_tile<KV_CACHE_SRC, 64, true>(p, stream)
                              : launch_tile<KV_CACHE_SRC, 128, true>(p, stream);
  return p.a.head_dim <= 64 ? launch_tile<KV_CACHE_SRC, 64, false>(p, stream)
                            : launch_tile<KV_CACHE_SRC, 128, false>(p, stream);
}

}  // namespace kvimpl
