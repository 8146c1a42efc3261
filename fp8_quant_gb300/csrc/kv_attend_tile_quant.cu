// The tensor-core attention kernels (kv_attend_tile.cuh) of e4m3fn and e2m1 caches.
#include "kv_attend_tile.cuh"

namespace kvimpl {

kv_status tile_quant(const TileParams& p, kv_cache_format format, cudaStream_t stream) {
  if (format == KV_CACHE_E4M3FN)
    return p.a.head_dim <= 64 ? launch_tile<KV_CACHE_E4M3FN, 64, false>(p, stream)
                              : launch_tile<KV_CACHE_E4M3FN, 128, false>(p, stream);
  return p.a.head_dim <= 64 ? launch_tile<KV_CACHE_E2M1, 64, false>(p, stream)
                            : launch_tile<KV_CACHE_E2M1, 128, false>(p, stream);
}

}  // namespace kvimpl
