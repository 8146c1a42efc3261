// Attention over a paged cache of latent rows: parameters and the general form of one row.
#pragma once

#include "kv_attend.cuh"
#include "kv_latent.cuh"

namespace kvimpl {

// `a` holds what kv_attend's kernels know too: a.k is the cache, a.kv_heads 1, a.group all query heads,
// a.head_dim the row's dims; window and sinks are 0.
struct LatentParams {
  AttendParams a;
  const float* scales;  // of e4m3fn rows, by slot
  int64_t scale_slot;
  int32_t latent;       // the row's first dims: the values
};

// The scale of key j's row, which lies at offset `off` of page `id`.
__device__ __forceinline__ float row_scale(const LatentParams& p, int32_t id, uint32_t off) {
  return __ldg(p.scales + (static_cast<int64_t>(id) * p.a.page.d + off) * p.scale_slot);
}

// One query row by one warp, any layout: lane l owns dims l, l + 32, ... (ND of them). Reads the
// visible keys one by one and nothing else. Writes output dims d0 .. d1 - 1, and the lse with dim 0.
template <int FMT, int ND>
__device__ __noinline__ void attend_latent_row(const LatentParams& lp, int32_t b, int32_t pos, int32_t t, int32_t h, int32_t d0, int32_t d1) {
  const AttendParams& p = lp.a;
  const uint32_t lane = threadIdx.x & 31u;
  const uint32_t D = static_cast<uint32_t>(p.head_dim);
  const uint8_t* q = p.q + t * p.q_token + h * p.q_head;
  float qv[ND], o[ND];
#pragma unroll
  for (int i = 0; i < ND; ++i) {
    const uint32_t d = lane + 32u * i;
    qv[i] = d < D ? widen16(__ldg(reinterpret_cast<const uint16_t*>(q) + d), p.bf16) : 0.0f;
    o[i] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  const int32_t* row = p.table + static_cast<int64_t>(b) * p.table_stride;
  bool any = false;
  for (int32_t i = 0; i <= pos; ++i) {
    const uint32_t j = static_cast<uint32_t>(i), pg = p.page.quot(j), off = j - pg * p.page.d;
    const int32_t id = __ldg(row + pg);
    if (id < 0 || id >= p.num_pages) {
      if (lane == 0) record_oob(p.err, static_cast<uint64_t>(b));
      continue;
    }
    any = true;
    const uint8_t* kr = p.k + id * p.k_page + off * p.k_slot;
    const float f = FMT == KV_CACHE_E4M3FN ? row_scale(lp, id, off) : 1.0f;
    float s = 0.0f, v[ND];
#pragma unroll
    for (int x = 0; x < ND; ++x) {
      const uint32_t d = lane + 32u * x;
      v[x] = d < D ? cache_element<FMT>(kr, nullptr, d, p.bf16) : 0.0f;
      s = __fmaf_rn(qv[x], v[x], s);
    }
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, w);
    s *= p.scale_log2 * f;
    const float mn = fmaxf(m, s);
    const float base = mn == -INFINITY ? 0.0f : mn;  // nothing but -inf so far: exp2(-inf) = 0
    const float e = exp2_fast(s - base), a = exp2_fast(m - base);
    m = mn;
    l = __fmaf_rn(l, a, e);
#pragma unroll
    for (int x = 0; x < ND; ++x) o[x] = __fmaf_rn(o[x], a, e * (v[x] * f));
  }
  // a row with visible keys whose scores are all -inf is 0 / 0, as its definition is
  const float inv = any ? __fdiv_rn(1.0f, l) : 0.0f;
  uint16_t* out = reinterpret_cast<uint16_t*>(p.out + t * p.o_token + h * p.o_head);
#pragma unroll
  for (int x = 0; x < ND; ++x) {
    const uint32_t d = lane + 32u * x;
    if (d >= static_cast<uint32_t>(d0) && d < static_cast<uint32_t>(d1)) out[d] = round16(o[x] * inv, p.bf16);
  }
  if (p.lse && lane == 0 && d0 == 0)
    p.lse[static_cast<int64_t>(t) * p.q_heads + h] = any ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace kvimpl
