// Attention over the paged cache: parameters, the sequences' geometry, the
// visible keys of a block of query rows, and the general form of one row.
#pragma once

#include "kv_fp4.cuh"

namespace kvimpl {

// x / d for 0 <= x < 2^31 and a divisor set up on the host: the high word of a
// product with ceil(2^(32 + shift) / d) (Granlund and Montgomery, "Division by
// invariant integers using multiplication", PLDI 1994).
struct FastDiv {
  uint32_t d, mul, shift;  // mul 0: d is a power of two, shift = log2(d)
  __device__ __forceinline__ uint32_t quot(uint32_t x) const {
    return mul == 0u ? x >> shift : __umulhi(x, mul) >> shift;
  }
};

struct AttendParams {
  const uint8_t *q, *k, *v;
  uint8_t* out;
  float* lse;
  const int32_t *table, *seq_lens, *q_start;
  int64_t table_stride;
  int64_t q_token, q_head, o_token, o_head;
  int64_t k_page, k_slot, k_head, v_page, v_slot, v_head;
  const uint8_t *k_sc, *v_sc;  // e2m1 block scales
  int64_t ks_page, ks_slot, ks_head, vs_page, vs_slot, vs_head;
  const float *k_scale, *v_scale;  // tensor scales, or null: 1
  FastDiv page;                // by page_size
  FastDiv group;               // by the query heads of a KV head
  int32_t num_pages, num_seqs, num_q, q_heads, kv_heads, head_dim;
  int32_t max_len;             // table_width * page_size (at most 2^31 - 1)
  int32_t window, sinks;       // window 0: none; both at most 2^30, as lengths are
  float scale_log2;            // sm_scale * log2(e)
  int32_t bf16;
  kv_error_record* err;
};

// Sequence b: its first query row, the number of them, and its keys.
struct AttendSeq {
  int32_t q0, nq, len;
};

__device__ __forceinline__ AttendSeq attend_seq(const AttendParams& p, int32_t b, bool record) {
  AttendSeq s;
  if (p.q_start) {
    const int32_t a = min(max(__ldg(p.q_start + b), 0), p.num_q);
    s.q0 = a;
    s.nq = max(min(__ldg(p.q_start + b + 1), p.num_q) - a, 0);
  } else {
    s.q0 = b;
    s.nq = 1;
  }
  s.len = __ldg(p.seq_lens + b);
  if (s.len < 0 || s.len > p.max_len) {
    if (record) record_oob(p.err, static_cast<uint64_t>(b));
    s.len = 0;
  }
  return s;
}

// The keys that rows at positions p_lo .. p_hi see between them: the first
// `sinks` and then lo .. p_hi, as a list of n keys.  Entry i is key(i).
struct KeyList {
  int32_t sinks, lo, n;
  __device__ __forceinline__ int32_t key(int32_t i) const { return i < sinks ? i : lo + (i - sinks); }
};

__device__ __forceinline__ KeyList visible_keys(const AttendParams& p, int32_t p_lo, int32_t p_hi) {
  KeyList r;
  r.lo = p.window > 0 ? max(p_lo - p.window + 1, 0) : 0;
  r.sinks = min(p.sinks, r.lo);
  r.n = p_hi < 0 ? 0 : r.sinks + (p_hi - r.lo + 1);
  return r;
}

// Whether a query at position pos sees key j (0 <= j).
__device__ __forceinline__ bool sees(const AttendParams& p, int32_t pos, int32_t j) {
  return j <= pos && (p.window == 0 || j > pos - p.window || j < p.sinks);
}

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float tensor_scale(const float* s) { return s ? __ldg(s) : 1.0f; }

// Element d of a cached head row.
template <int FMT>
__device__ __forceinline__ float cache_element(const uint8_t* row, const uint8_t* sc, uint32_t d, bool bf16) {
  if constexpr (FMT == KV_CACHE_SRC) {
    return widen16(__ldg(reinterpret_cast<const uint16_t*>(row) + d), bf16);
  } else if constexpr (FMT == KV_CACHE_E4M3FN) {
    return f32_from_e4m3(__ldg(row + d));
  } else {
    uint32_t f[4];
    f16x2_from_e2m1x8((__ldg(row + d / 2) >> (4u * (d & 1u))) & 0xFu, f);
    return __fmul_rn(widen2<false>(f[0]).x, f32_from_e4m3(__ldg(sc + d / kFp4Block)));
  }
}

// One query row by one warp, any layout: lane l owns dims l, l + 32, ... (ND of
// them).  Reads the visible keys one by one and nothing else.
template <int FMT, int ND>
__device__ __noinline__ void attend_row(const AttendParams& p, int32_t b, int32_t pos, int32_t t,
                                        int32_t h) {
  const uint32_t lane = threadIdx.x & 31u;
  const uint32_t D = static_cast<uint32_t>(p.head_dim);
  const int32_t kvh = static_cast<int32_t>(p.group.quot(static_cast<uint32_t>(h)));
  const uint8_t* q = p.q + t * p.q_token + h * p.q_head;
  float qv[ND], o[ND];
#pragma unroll
  for (int i = 0; i < ND; ++i) {
    const uint32_t d = lane + 32u * i;
    qv[i] = d < D ? widen16(__ldg(reinterpret_cast<const uint16_t*>(q) + d), p.bf16) : 0.0f;
    o[i] = 0.0f;
  }
  const float scale = p.scale_log2 * tensor_scale(p.k_scale);
  float m = -INFINITY, l = 0.0f;
  const KeyList keys = visible_keys(p, pos, pos);
  const int32_t* row = p.table + static_cast<int64_t>(b) * p.table_stride;
  bool any = false;
  for (int32_t i = 0; i < keys.n; ++i) {
    const uint32_t j = static_cast<uint32_t>(keys.key(i));
    const uint32_t pg = p.page.quot(j), off = j - pg * p.page.d;
    const int32_t id = __ldg(row + pg);
    if (id < 0 || id >= p.num_pages) {
      if (lane == 0) record_oob(p.err, static_cast<uint64_t>(b));
      continue;
    }
    any = true;
    const uint8_t* kr = p.k + id * p.k_page + off * p.k_slot + kvh * p.k_head;
    const uint8_t* vr = p.v + id * p.v_page + off * p.v_slot + kvh * p.v_head;
    const uint8_t* ks = FMT == KV_CACHE_E2M1 ? p.k_sc + id * p.ks_page + off * p.ks_slot + kvh * p.ks_head : nullptr;
    const uint8_t* vs = FMT == KV_CACHE_E2M1 ? p.v_sc + id * p.vs_page + off * p.vs_slot + kvh * p.vs_head : nullptr;
    float s = 0.0f, vv[ND];
#pragma unroll
    for (int x = 0; x < ND; ++x) {
      const uint32_t d = lane + 32u * x;
      vv[x] = 0.0f;
      if (d < D) {
        s = __fmaf_rn(qv[x], cache_element<FMT>(kr, ks, d, p.bf16), s);
        vv[x] = cache_element<FMT>(vr, vs, d, p.bf16);
      }
    }
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, w);
    s *= scale;
    const float mn = fmaxf(m, s);
    const float base = mn == -INFINITY ? 0.0f : mn;  // nothing but -inf so far: exp2(-inf) = 0
    const float e = exp2_fast(s - base), a = exp2_fast(m - base);
    m = mn;
    l = __fmaf_rn(l, a, e);
#pragma unroll
    for (int x = 0; x < ND; ++x) o[x] = __fmaf_rn(o[x], a, e * vv[x]);
  }
  // a row with visible keys whose scores are all -inf is 0 / 0, as its definition is
  const float inv = any ? __fdiv_rn(tensor_scale(p.v_scale), l) : 0.0f;
  uint8_t* out = p.out + t * p.o_token + h * p.o_head;
#pragma unroll
  for (int x = 0; x < ND; ++x) {
    const uint32_t d = lane + 32u * x;
    if (d < D) reinterpret_cast<uint16_t*>(out)[d] = round16(o[x] * inv, p.bf16);
  }
  if (p.lse && lane == 0)
    p.lse[static_cast<int64_t>(t) * p.q_heads + h] = any ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace kvimpl
