// Attention over the paged cache (kv_attend): argument checks, the choice of
// the kernel, and the general kernel.
//
//  * kv_attend_tile   (kv_attend_tile.cuh) many query rows per sequence: head
//                     dims that are multiples of 16 up to 128, aligned as below.
//  * kv_attend_stream (kv_attend_stream.cuh) few query rows over much cache, in
//                     layouts that TMA takes.
//  * kv_attend_split  (kv_attend_split.cuh) the rest of head dims that are multiples of 16
//                     up to 256, 16-byte aligned bases and strides.
//  * kv_attend_rows   any head dim, alignment and stride: one warp per query
//                     row and head, one key after the other.
#include <algorithm>
#include <cmath>
#include <climits>

#include "kv_attend_stream.cuh"
#include "kv_attend_tile.cuh"

namespace kvimpl {
namespace {

template <int FMT, int ND>
__global__ void __launch_bounds__(kThreads) kv_attend_rows(const __grid_constant__ AttendParams p) {
  grid_handover();
  const uint64_t nwarps = static_cast<uint64_t>(gridDim.x) * warps_per_cta();
  const uint64_t units = static_cast<uint64_t>(p.num_q) * static_cast<uint64_t>(p.q_heads);
  for (uint64_t u = static_cast<uint64_t>(blockIdx.x) * warps_per_cta() + (threadIdx.x >> 5);
       u < units; u += nwarps) {
    const int32_t t = static_cast<int32_t>(u / static_cast<uint32_t>(p.q_heads));
    const int32_t h = static_cast<int32_t>(u - static_cast<uint64_t>(t) * p.q_heads);
    // the last sequence that begins at or before row t
    int32_t b = t;
    if (p.q_start) {
      int32_t lo = 0, hi = p.num_seqs - 1;
      while (lo < hi) {
        const int32_t mid = (lo + hi + 1) >> 1;
        if (__ldg(p.q_start + mid) <= t) lo = mid; else hi = mid - 1;
      }
      b = lo;
    }
    const AttendSeq s = attend_seq(p, b, h == 0 && (threadIdx.x & 31u) == 0);
    if (t < s.q0 || t >= s.q0 + s.nq) continue;
    attend_row<FMT, ND>(p, b, s.len - s.nq + (t - s.q0), t, h);
  }
}

template <int FMT>
kv_status launch_rows_any(const AttendParams& p, cudaStream_t stream) {
  const uint64_t units = static_cast<uint64_t>(p.num_q) * static_cast<uint64_t>(p.q_heads);
  return p.head_dim <= 256 ? launch(kv_attend_rows<FMT, 8>, units, p, stream, 0, 128)
                           : launch(kv_attend_rows<FMT, 32>, units, p, stream, 0, 128);
}

// Bytes of the visible cache from which on kv_attend_stream is taken.  One sequence, 32 over 8 heads of 128,
// 16-bit: 18.1 us against kv_attend_split's 17.5 at 4 MB, 15.3 against 18.3 at 16 MB, 24.7 against 31.5 at 64 MB.
constexpr int64_t kStreamMinBytes = 8ll << 20;

// Whether kv_attend_tile is the faster for `rows` query rows per sequence and KV
// head and `keys` visible keys (upper bounds: the host knows no length).  Both
// times in us, fitted to calls of 1 to 64 sequences, 512 to 65,536 keys, 1 to 1,024 rows:
//  * a CTA of the tile kernel takes 128 keys (up to 256 rows) in 1.4 (16-bit rows
//    of 128 dims), 1.5 (quantised ones) or 1.2 - 1.35 us (64 dims), bound by its
//    own latencies, in items / SMs rounds with 3 us of their own (6 where 128 dims
//    are converted; half as much again, and tiles 1.3 times as long, with all SMs
//    at it); all together read at most 5.3 TB/s;
//  * the others read the cache once per 8 or 16 rows, at 6 TB/s, or 25 (8 rows)
//    and 17 (16) quantised keys and heads of 128 dims a ns, 36 and 27 of 64; and
//    take 11 us more (two launches, the scan of the lengths, the join), 16 when
//    the warps of a CTA have eight heads to do.
// E.g. 8 sequences x 4,096 keys, 32 over 8 heads of 128, 16-bit: tile 52, the
// others 41 us at 16 rows, 52 against 65 at 32; 64 sequences x 512 keys, e2m1:
// 72 against 38 us at 16 rows, 77 against 108 at 64.
bool tiles_pay(const AttendParams& p, kv_cache_format format, int64_t rows, int64_t keys) {
  int sms = 0;
  if (current_sm_count(&sms) != KV_OK) return false;
  const bool small = p.head_dim <= 64, quant = format != KV_CACHE_SRC, fp4 = format == KV_CACHE_E2M1;
  const double heads = static_cast<double>(p.num_seqs) * p.kv_heads, n = static_cast<double>(keys);
  const double bytes = heads * n * 2.0 * p.head_dim * (fp4 ? 0.5625 : quant ? 1.0 : 2.0);
  const double row_tiles = std::ceil(rows / 256.0), items = heads * row_tiles;
  const double load = quant && items >= sms ? 1.3 : 1.0;
  const double step = (quant ? (small ? (fp4 ? 1.35 : 1.2) : 1.5) : (small ? 1.25 : 1.4)) * (rows > 128 ? 1.1 : 1.0) * load;
  const double start = quant && !small ? (load > 1.0 ? 9.0 : 6.0) : 3.0;
  const double tile = std::max(4.0 + std::ceil(items / sms) * (start + std::ceil(n / kTileKeys) * step), row_tiles * bytes / 5.3e6);
  const bool narrow = rows <= 8;
  const double blocks = narrow ? 1.0 : std::ceil(rows / 16.0);
  const double pass = std::max(bytes / 6e6, quant ? heads * n / (small ? (narrow ? 36e3 : 27e3) : (narrow ? 25e3 : 17e3)) : 0.0);
  return tile < 11.0 + 0.625 * heads_of_cta(p.kv_heads, kSplitWarps) + blocks * pass;
}

}  // namespace
}  // namespace kvimpl

using namespace kvimpl;

extern "C" kv_status kv_attend(const void* q, void* out, float* lse, const void* k_cache,
                               const void* v_cache, const int32_t* page_table, int64_t table_stride,
                               int64_t table_width, const int32_t* seq_lens, const int32_t* q_start,
                               int32_t num_seqs, int64_t num_q_tokens, int32_t num_q_heads,
                               int32_t num_heads, int32_t head_dim, kv_src_dtype dtype,
                               const kv_attend_strides* s, int64_t page_size, int64_t num_pages,
                               kv_cache_format format, const float* k_scale, const float* v_scale,
                               const kv_block_scales* scales, float sm_scale, int64_t window,
                               int64_t sinks, void* work, int64_t work_bytes, kv_error_record* d_err,
                               kv_stream_t stream_) {
  if (num_seqs < 0 || num_q_tokens < 0) return KV_ERR_INVALID_ARG;
  if (format != KV_CACHE_SRC && format != KV_CACHE_E4M3FN && format != KV_CACHE_E2M1)
    return KV_ERR_INVALID_ARG;
  if (num_seqs == 0 || num_q_tokens == 0) return KV_OK;
  if (!q || !out || !k_cache || !v_cache || !page_table || !seq_lens || !s || !d_err)
    return KV_ERR_INVALID_ARG;
  if (dtype != KV_SRC_F16 && dtype != KV_SRC_BF16) return KV_ERR_INVALID_ARG;
  if (num_q_heads < 1 || num_heads < 1 || head_dim < 1 || num_q_heads % num_heads != 0 ||
      page_size < 1 || num_pages < 1 || table_width < 1 || table_stride < table_width ||
      window < 0 || sinks < 0 || work_bytes < 0 || !std::isfinite(sm_scale))
    return KV_ERR_INVALID_ARG;
  if (!q_start && num_q_tokens != num_seqs) return KV_ERR_INVALID_ARG;
  if (((u64(page_table) | u64(seq_lens) | u64(q_start) | u64(lse) | u64(k_scale) | u64(v_scale)) & 3u) != 0 ||
      (u64(d_err) & 7u) != 0 || (work && (u64(work) & 255u) != 0))
    return KV_ERR_INVALID_ARG;
  if (format == KV_CACHE_E2M1 && (!scales || !scales->k || !scales->v)) return KV_ERR_INVALID_ARG;
  const uint64_t q_bits = u64(q) | u64(out) | u64(s->q_token) | u64(s->q_head) | u64(s->o_token) | u64(s->o_head);
  const uint64_t c_bits = u64(k_cache) | u64(v_cache) | u64(s->kc_page) | u64(s->kc_slot) | u64(s->kc_head) |
                          u64(s->vc_page) | u64(s->vc_slot) | u64(s->vc_head);
  if ((q_bits & 1u) != 0 || (format == KV_CACHE_SRC && (c_bits & 1u) != 0)) return KV_ERR_UNSUPPORTED;
  if (head_dim > 1024 || (format == KV_CACHE_E2M1 && head_dim % kFp4Block != 0)) return KV_ERR_UNSUPPORTED;
  if (num_q_tokens >= (1 << 30) || page_size >= INT_MAX || num_pages >= INT_MAX) return KV_ERR_UNSUPPORTED;
  {
    const void* in[14] = {q, out, page_table, seq_lens, k_cache, v_cache, d_err};
    int n = 7;
    if (lse) in[n++] = lse;
    if (q_start) in[n++] = q_start;
    if (work && work_bytes > 0) in[n++] = work;
    if (format == KV_CACHE_E2M1) {
      in[n++] = scales->k;
      in[n++] = scales->v;
    }
    if (format != KV_CACHE_SRC && k_scale) in[n++] = k_scale;
    if (format != KV_CACHE_SRC && v_scale) in[n++] = v_scale;
    bool on_device = true;
    const kv_status cs = classify_inputs(in, n, &on_device);
    if (cs != KV_OK) return cs;
  }

  AttendParams p = {};
  p.q = static_cast<const uint8_t*>(q);
  p.k = static_cast<const uint8_t*>(k_cache);
  p.v = static_cast<const uint8_t*>(v_cache);
  p.out = static_cast<uint8_t*>(out);
  p.lse = lse;
  p.table = page_table;
  p.seq_lens = seq_lens;
  p.q_start = q_start;
  p.table_stride = table_stride;
  p.q_token = s->q_token; p.q_head = s->q_head;
  p.o_token = s->o_token; p.o_head = s->o_head;
  p.k_page = s->kc_page; p.k_slot = s->kc_slot; p.k_head = s->kc_head;
  p.v_page = s->vc_page; p.v_slot = s->vc_slot; p.v_head = s->vc_head;
  if (format == KV_CACHE_E2M1) {
    p.k_sc = static_cast<const uint8_t*>(scales->k);
    p.v_sc = static_cast<const uint8_t*>(scales->v);
    p.ks_page = scales->k_page; p.ks_slot = scales->k_slot; p.ks_head = scales->k_head;
    p.vs_page = scales->v_page; p.vs_slot = scales->v_slot; p.vs_head = scales->v_head;
  }
  if (format != KV_CACHE_SRC) {
    p.k_scale = k_scale;
    p.v_scale = v_scale;
  }
  p.page = fast_div(static_cast<uint32_t>(page_size));
  p.group = fast_div(static_cast<uint32_t>(num_q_heads / num_heads));
  p.num_pages = static_cast<int32_t>(num_pages);
  p.num_seqs = num_seqs;
  p.num_q = static_cast<int32_t>(num_q_tokens);
  p.q_heads = num_q_heads;
  p.kv_heads = num_heads;
  p.head_dim = head_dim;
  p.max_len = static_cast<int32_t>(table_width > (int64_t{1} << 30) / page_size ? int64_t{1} << 30 : table_width * page_size);
  p.window = static_cast<int32_t>(window < (1 << 30) ? window : 1 << 30);
  p.sinks = static_cast<int32_t>(sinks < (1 << 30) ? sinks : 1 << 30);
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  p.bf16 = dtype == KV_SRC_BF16;
  p.err = d_err;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  auto fits = [](int64_t x) { return x > INT_MIN && x < INT_MAX; };
  bool near = fits(s->kc_page) && fits(s->kc_slot) && fits(s->vc_page) && fits(s->vc_slot);
  if (format == KV_CACHE_E2M1)
    near = near && fits(scales->k_page) && fits(scales->k_slot) && fits(scales->v_page) && fits(scales->v_slot);
  if (head_dim % 16 == 0 && head_dim <= 256 && ((q_bits | c_bits) & 15u) == 0 && near) {
    const int64_t per_seq = (num_q_tokens + num_seqs - 1) / num_seqs * p.group.d;
    // no list of visible keys is longer
    int64_t keys = p.max_len;
    if (window > 0 && window < keys && sinks < keys) {
      const int64_t most = window + sinks + (num_q_tokens + num_seqs - 1) / num_seqs + 16;
      keys = most < keys ? most : keys;
    }
    if (head_dim <= 128 && p.group.d <= 128 && tiles_pay(p, format, per_seq, keys)) {
      TileParams tp = {};
      tp.a = p;
      tp.k_page = static_cast<int32_t>(s->kc_page); tp.k_slot = static_cast<int32_t>(s->kc_slot);
      tp.v_page = static_cast<int32_t>(s->vc_page); tp.v_slot = static_cast<int32_t>(s->vc_slot);
      if (format == KV_CACHE_E2M1) {
        tp.ks_page = static_cast<int32_t>(scales->k_page); tp.ks_slot = static_cast<int32_t>(scales->k_slot);
        tp.vs_page = static_cast<int32_t>(scales->v_page); tp.vs_slot = static_cast<int32_t>(scales->v_slot);
        const uint64_t bits = u64(scales->k) | u64(scales->v) | u64(scales->k_page) | u64(scales->v_page) | u64(scales->k_slot) |
                              u64(scales->v_slot) | u64(scales->k_head) | u64(scales->v_head);
        tp.scale_word = (bits & 7u) == 0 && head_dim == 128 ? 8 : (bits & 3u) == 0 && head_dim % 64 == 0 ? 4 : 1;
      }
      tp.qpt = kTileRows / static_cast<int32_t>(p.group.d);
      tp.blocks = p.num_q / (2 * tp.qpt) + num_seqs;
      if (format != KV_CACHE_SRC) return tile_quant(tp, format, stream);
      // TMA: a tile is whole pages or part of one; behind a window's lower edge, and with other pages, 16 keys are
      auto divides = [&](int64_t keys) { return page_size <= keys ? keys % page_size == 0 : page_size % keys == 0; };
      const int64_t granule = window == 0 && divides(kTileKeys) ? kTileKeys : 16;
      if (page_size >= 8 && divides(granule)) {
        const int box = static_cast<int>(page_size < granule ? page_size : granule);
        if (cache_map(&tp.k_map, k_cache, 2, p.bf16, head_dim, page_size, num_heads, num_pages, s->kc_slot, s->kc_head, s->kc_page, 64,
                      box, 1, true) &&
            cache_map(&tp.v_map, v_cache, 2, p.bf16, head_dim, page_size, num_heads, num_pages, s->vc_slot, s->vc_head, s->vc_page, 64,
                      box, 1, true))
          tp.box = box;
      }
      return tile_src(tp, stream);
    }
    SplitParams sp = {};
    sp.a = p;
    sp.whole_blocks = page_size % 16 == 0;
    sp.k_page = static_cast<int32_t>(s->kc_page); sp.k_slot = static_cast<int32_t>(s->kc_slot);
    sp.v_page = static_cast<int32_t>(s->vc_page); sp.v_slot = static_cast<int32_t>(s->vc_slot);
    if (format == KV_CACHE_E2M1) {
      sp.ks_page = static_cast<int32_t>(scales->k_page); sp.ks_slot = static_cast<int32_t>(scales->k_slot);
      sp.vs_page = static_cast<int32_t>(scales->v_page); sp.vs_slot = static_cast<int32_t>(scales->v_slot);
    }
    const bool wide = per_seq > 8;  // up to 8 rows of a sequence and head take one block of mma columns, more two
    // kv_attend_stream: boxes of 16 or of a tile's keys within a page, e2m1 scales of a CTA's heads in
    // one run of whole 16 bytes, and enough cache to be worth the maps and the deep ring
    const int bits = format == KV_CACHE_SRC ? 16 : format == KV_CACHE_E4M3FN ? 8 : 4;
    const int64_t row = static_cast<int64_t>(head_dim) * bits / 8;
    if (head_dim <= 128 && page_size % 16 == 0 && num_seqs * keys * num_heads * row * 2 >= kStreamMinBytes &&
        (format != KV_CACHE_E2M1 || head_dim % 32 == 0)) {
      StreamParams tp = {};
      tp.s = sp;
      const int tile = format == KV_CACHE_SRC && head_dim > 64 ? 16 : format == KV_CACHE_E2M1 ? kStreamFp4Tile : 32;
      tp.box = tile;
      while (page_size % tp.box != 0) tp.box /= 2;
      const int hw = heads_of_cta(num_heads, kSplitWarps);
      const int padded = (head_dim <= 64 ? 64 : 128) * bits / 8, ds = head_dim / 16;
      auto map = [&](CUtensorMap* m, const void* base, int64_t slot, int64_t head, int64_t page) {
        return cache_map(m, base, 1, false, row, page_size, num_heads, num_pages, slot, head, page, padded < 128 ? padded : 128, tp.box, hw, true);
      };
      bool fit = map(&tp.k_map, k_cache, s->kc_slot, s->kc_head, s->kc_page) && map(&tp.v_map, v_cache, s->vc_slot, s->vc_head, s->vc_page);
      if (fit && format == KV_CACHE_E2M1) {
        const kv_block_scales& b = *scales;
        const int64_t run = static_cast<int64_t>(num_heads) * ds;
        fit = num_heads == 1 || (b.k_head == ds && b.v_head == ds);
        tp.flat_scales = fit && hw == num_heads && b.k_slot == run && b.v_slot == run && (tp.box * run) % 16 == 0 &&
                         ((u64(b.k) | u64(b.v) | u64(b.k_page) | u64(b.v_page) | u64(16 * run)) & 15u) == 0;
        if (fit && !tp.flat_scales)
          fit = cache_map(&tp.ks_map, b.k, 1, false, run, page_size, 1, num_pages, b.k_slot, 16, b.k_page, hw * ds, tp.box, 1, false) &&
                cache_map(&tp.vs_map, b.v, 1, false, run, page_size, 1, num_pages, b.v_slot, 16, b.v_page, hw * ds, tp.box, 1, false);
      }
      if (fit) {
        switch (format) {
          case KV_CACHE_SRC:
            return p.bf16 ? stream_bf16(tp, wide, work, work_bytes, keys, stream)
                          : stream_f16(tp, wide, work, work_bytes, keys, stream);
          case KV_CACHE_E4M3FN: return stream_e4m3(tp, wide, work, work_bytes, keys, stream);
          default: return stream_e2m1(tp, wide, work, work_bytes, keys, stream);
        }
      }
    }
    switch (format) {
      case KV_CACHE_SRC:
        return p.bf16 ? split_bf16(sp, wide, work, work_bytes, keys, stream)
                      : split_f16(sp, wide, work, work_bytes, keys, stream);
      case KV_CACHE_E4M3FN: return split_e4m3(sp, wide, work, work_bytes, keys, stream);
      default: return split_e2m1(sp, wide, work, work_bytes, keys, stream);
    }
  }
  switch (format) {
    case KV_CACHE_SRC: return launch_rows_any<KV_CACHE_SRC>(p, stream);
    case KV_CACHE_E4M3FN: return launch_rows_any<KV_CACHE_E4M3FN>(p, stream);
    default: return launch_rows_any<KV_CACHE_E2M1>(p, stream);
  }
}
