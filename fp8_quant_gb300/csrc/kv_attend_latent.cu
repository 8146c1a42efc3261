// Attention over a paged cache of latent rows (kv_attend_latent): argument
// checks, the choice of the kernel, and the general kernel.
//
//  * kv_attend_latent_tile  (kv_attend_latent_tile.cuh) row dims that are multiples of 16 up to 576, latent
//                           dims multiples of 8 up to 512, 16-byte aligned bases and strides.
//  * kv_latent_attend_rows  any dims, alignment and stride: one warp per query row
//                           and head, one key after the other.
#include <cmath>
#include <climits>

#include "kv_attend_latent_tile.cuh"

namespace kvimpl {
namespace {

template <int FMT, int ND>
__global__ void __launch_bounds__(kThreads) kv_latent_attend_rows(const __grid_constant__ LatentParams p) {
  grid_handover();
  const AttendParams& a = p.a;
  const uint64_t nwarps = static_cast<uint64_t>(gridDim.x) * warps_per_cta();
  const uint64_t units = static_cast<uint64_t>(a.num_q) * static_cast<uint64_t>(a.q_heads);
  for (uint64_t u = static_cast<uint64_t>(blockIdx.x) * warps_per_cta() + (threadIdx.x >> 5); u < units; u += nwarps) {
    const int32_t t = static_cast<int32_t>(u / static_cast<uint32_t>(a.q_heads));
    const int32_t h = static_cast<int32_t>(u - static_cast<uint64_t>(t) * a.q_heads);
    // the last sequence that begins at or before row t
    int32_t b = t;
    if (a.q_start) {
      int32_t lo = 0, hi = a.num_seqs - 1;
      while (lo < hi) {
        const int32_t mid = (lo + hi + 1) >> 1;
        if (__ldg(a.q_start + mid) <= t) lo = mid; else hi = mid - 1;
      }
      b = lo;
    }
    const AttendSeq s = attend_seq(a, b, h == 0 && (threadIdx.x & 31u) == 0);
    if (t < s.q0 || t >= s.q0 + s.nq) continue;
    attend_latent_row<FMT, ND>(p, b, s.len - s.nq + (t - s.q0), t, h, 0, p.latent);
  }
}

template <int FMT>
kv_status launch_rows_any(const LatentParams& p, cudaStream_t stream) {
  const uint64_t units = static_cast<uint64_t>(p.a.num_q) * static_cast<uint64_t>(p.a.q_heads);
  return p.a.head_dim <= 256 ? launch(kv_latent_attend_rows<FMT, 8>, units, p, stream, 0, 128)
                             : launch(kv_latent_attend_rows<FMT, 32>, units, p, stream, 0, 128);
}

}  // namespace
}  // namespace kvimpl

using namespace kvimpl;

extern "C" kv_status kv_attend_latent(const void* q, void* out, float* lse, const void* cache, const float* scales,
                                      const int32_t* page_table, int64_t table_stride, int64_t table_width,
                                      const int32_t* seq_lens, const int32_t* q_start, int32_t num_seqs,
                                      int64_t num_q_tokens, int32_t num_q_heads, int32_t row_dim, int32_t latent_dim,
                                      kv_src_dtype dtype, const kv_attend_latent_strides* s, int64_t page_size,
                                      int64_t num_pages, kv_cache_format format, float sm_scale, void* work,
                                      int64_t work_bytes, kv_error_record* d_err, kv_stream_t stream_) {
  if (num_seqs < 0 || num_q_tokens < 0) return KV_ERR_INVALID_ARG;
  if (format != KV_CACHE_SRC && format != KV_CACHE_E4M3FN) return KV_ERR_INVALID_ARG;
  if (num_seqs == 0 || num_q_tokens == 0) return KV_OK;
  if (!q || !out || !cache || !page_table || !seq_lens || !s || !d_err) return KV_ERR_INVALID_ARG;
  if (dtype != KV_SRC_F16 && dtype != KV_SRC_BF16) return KV_ERR_INVALID_ARG;
  if (num_q_heads < 1 || row_dim < 1 || latent_dim < 1 || latent_dim > row_dim || page_size < 1 || num_pages < 1 ||
      table_width < 1 || table_stride < table_width || work_bytes < 0 || !std::isfinite(sm_scale))
    return KV_ERR_INVALID_ARG;
  if (!q_start && num_q_tokens != num_seqs) return KV_ERR_INVALID_ARG;
  const bool fp8 = format == KV_CACHE_E4M3FN;
  if (fp8 && (!scales || s->scale_slot < 1)) return KV_ERR_INVALID_ARG;
  if (((u64(page_table) | u64(seq_lens) | u64(q_start) | u64(lse) | (fp8 ? u64(scales) : 0u)) & 3u) != 0 ||
      (u64(d_err) & 7u) != 0 || (work && (u64(work) & 255u) != 0))
    return KV_ERR_INVALID_ARG;
  const uint64_t q_bits = u64(q) | u64(out) | u64(s->q_token) | u64(s->q_head) | u64(s->o_token) | u64(s->o_head);
  const uint64_t c_bits = u64(cache) | u64(s->cache_page) | u64(s->cache_slot);
  if ((q_bits & 1u) != 0 || (!fp8 && (c_bits & 1u) != 0)) return KV_ERR_UNSUPPORTED;
  if (row_dim > kMaxRow || num_q_tokens >= (1 << 30) || num_q_tokens * num_q_heads >= INT_MAX - 1024 || page_size >= INT_MAX ||
      num_pages >= INT_MAX)
    return KV_ERR_UNSUPPORTED;
  {
    const void* in[10] = {q, out, page_table, seq_lens, cache, d_err};
    int n = 6;
    if (lse) in[n++] = lse;
    if (q_start) in[n++] = q_start;
    if (work && work_bytes > 0) in[n++] = work;
    if (fp8) in[n++] = scales;
    const kv_status cs = classify_here(in, n);
    if (cs != KV_OK) return cs;
  }

  LatentParams p = {};
  AttendParams& a = p.a;
  a.q = static_cast<const uint8_t*>(q);
  a.k = static_cast<const uint8_t*>(cache);
  a.out = static_cast<uint8_t*>(out);
  a.lse = lse;
  a.table = page_table;
  a.seq_lens = seq_lens;
  a.q_start = q_start;
  a.table_stride = table_stride;
  a.q_token = s->q_token; a.q_head = s->q_head;
  a.o_token = s->o_token; a.o_head = s->o_head;
  a.k_page = s->cache_page; a.k_slot = s->cache_slot;
  a.page = fast_div(static_cast<uint32_t>(page_size));
  a.group = fast_div(static_cast<uint32_t>(num_q_heads));
  a.num_pages = static_cast<int32_t>(num_pages);
  a.num_seqs = num_seqs;
  a.num_q = static_cast<int32_t>(num_q_tokens);
  a.q_heads = num_q_heads;
  a.kv_heads = 1;
  a.head_dim = row_dim;
  a.max_len = static_cast<int32_t>(table_width > (int64_t{1} << 30) / page_size ? int64_t{1} << 30 : table_width * page_size);
  a.scale_log2 = sm_scale * 1.4426950408889634f;
  a.bf16 = dtype == KV_SRC_BF16;
  a.err = d_err;
  p.scales = scales;
  p.scale_slot = s->scale_slot;
  p.latent = latent_dim;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  auto fits = [](int64_t x) { return x > INT_MIN && x < INT_MAX; };
  if (row_dim % 16 == 0 && row_dim <= 64 * kLatMaxChunks && latent_dim % 8 == 0 && latent_dim <= 512 && ((q_bits | c_bits) & 15u) == 0 &&
      fits(s->cache_page) && fits(s->cache_slot)) {
    LatentTileParams tp = {};
    tp.l = p;
    tp.page_stride = static_cast<int32_t>(s->cache_page);
    tp.slot_stride = static_cast<int32_t>(s->cache_slot);
    tp.chunks = (row_dim + 63) / 64;
    tp.ksteps = row_dim / 16;
    tp.blocks = (latent_dim + 127) / 128;
    const int64_t rows = (num_q_tokens + num_seqs - 1) / num_seqs * num_q_heads;
    const bool few = rows <= 32;
    // TMA: runs of 8, 16 or 32 keys of a page a box, with all their dims where these are whole chunks
    int groups = 4;
    while (groups > 0 && page_size % (8 * groups) != 0) groups /= 2;
    const bool whole = row_dim % 64 == 0;
    if (groups > 0 && (whole || !fp8) &&
        latent_map(&tp.map, cache, fp8 ? 1 : 2, a.bf16, row_dim, page_size, num_pages, s->cache_slot, s->cache_page, tp.chunks,
                   whole ? tp.chunks : 1, whole ? groups : 1, !fp8)) {
      tp.box = whole ? groups : 1;
      tp.box_chunks = whole ? tp.chunks : 1;
    }
    if (fp8) return latent_tile_e4m3(tp, few, work, work_bytes, a.max_len, stream);
    return latent_tile_src(tp, few, work, work_bytes, a.max_len, stream);
  }
  return fp8 ? launch_rows_any<KV_CACHE_E4M3FN>(p, stream) : launch_rows_any<KV_CACHE_SRC>(p, stream);
}
