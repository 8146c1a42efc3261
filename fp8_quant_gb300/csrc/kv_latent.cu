// Appending to a cache of latent rows (kv_store_latent) and reading it back
// (kv_gather_latent).
//
// What is computed is in kvstore.h.  Per token the latent and rotary inputs and
// the queries' rotary dims are read once and written once, with about five fp32
// operations an element, so bytes bound it.
//
//  * kv_latent_rows  latent dims that are multiples of 8 up to 1,024, rotary ones
//                    multiples of 16 up to 512 that are rotated whole, 16-byte
//                    pieces.  A token's row is one warp's: 8 dims a lane and
//                    chunk, all in registers, so that the mean and the largest
//                    magnitude are a reduction over the warp and nothing is read
//                    twice.  A lane's rotary item is eight whole pairs, as two
//                    pieces of 8 dims.  Further warps take the queries' items, up to
//                    four passes' loads in flight, their eight cosines and
//                    sines loaded once.  No row load waits for the slot or the position.
//                    At most 64 registers, so that an SM has four CTAs, although the forms
//                    with four passes, and those of more than 512 latent dims, then spill
//                    (172 bytes stored and 152 loaded in the one measured here): a prefill of
//                    32,768 fp16 rows of 512 + 64 dims with 32 heads' queries 71 us (5.0
//                    TB/s, 74 % of the copy rate), 74 with 80 registers and 40 bytes
//                    spilled, 89 with 98 and none, 90 with 48; into an e4m3fn cache 73, 75,
//                    79 and 91.  Pieces of 128 bytes in rows of 1,152, the loads' latency
//                    and the spills bound it.
//  * kv_latent_any   any layout: a warp per (token, row or query head), elements
//                    one by one, the row gone through once for each sum it needs.
//  * kv_latent_gather  an item is 32 or 16 bytes of a 16-bit row, or 16 codes; a
//                    thread has four items' slots, then rows, in flight: 65,536 rows
//                    from padded slots 24.8 us, 91 % of the copy rate.
#include <cmath>

#include "kv_fp4.cuh"
#include "kv_latent.cuh"

namespace kvimpl {
namespace {

struct LatentStoreParams {
  const uint8_t *c, *r, *weight, *q;
  uint8_t *cache, *q_out;
  float* scales;
  int64_t c_token, r_token, cache_page, cache_slot, scale_slot;
  int64_t q_token, q_head, qo_token, qo_head;
  const void *indices, *positions;
  const float* table;
  int64_t index_stride, position_stride, table_stride;
  int64_t max_position, size_limit, page_size;
  uint64_t num_units;
  uint32_t units;           // per token: the row's, then the queries'
  uint32_t q_heads, latent, rope, rotary;
  uint32_t iph, hpp;        // rotary items per head, heads per pass
  float eps;
  int idx64, pos64, bf16, interleaved, narrow;
  kv_error_record* err;
};

__device__ __forceinline__ int64_t index_at(const void* p, int64_t i, int is64) {
  return is64 ? static_cast<int64_t>(__ldg(static_cast<const long long*>(p) + i))
              : static_cast<int64_t>(__ldg(static_cast<const int*>(p) + i));
}

// A token's slot and position.
struct LatentPlace {
  int64_t slot, pos;
  bool slot_ok, pos_ok;
};

__device__ __forceinline__ LatentPlace place_of(const LatentStoreParams& p, uint64_t t, bool record) {
  LatentPlace r;
  r.slot = index_at(p.indices, static_cast<int64_t>(t) * p.index_stride, p.idx64);
  r.slot_ok = r.slot >= 0 && r.slot < p.size_limit;
  r.pos = 0;
  r.pos_ok = true;
  if (p.rope > 0) {
    r.pos = index_at(p.positions, static_cast<int64_t>(t) * p.position_stride, p.pos64);
    r.pos_ok = r.pos >= 0 && r.pos < p.max_position;
  }
  if (record && !(r.slot_ok && r.pos_ok)) record_oob(p.err, t);
  return r;
}

__device__ __forceinline__ uint8_t* row_of(const LatentStoreParams& p, int64_t slot) {
  if (p.narrow) {
    const uint32_t s = static_cast<uint32_t>(slot), n = static_cast<uint32_t>(p.page_size), pg = s / n;
    return p.cache + static_cast<int64_t>(pg) * p.cache_page + static_cast<int64_t>(s - pg * n) * p.cache_slot;
  }
  const int64_t pg = slot / p.page_size;
  return p.cache + pg * p.cache_page + (slot - pg * p.page_size) * p.cache_slot;
}

// a' and b' of a pair, every operation rounded on its own.
__device__ __forceinline__ float2 turn(float a, float b, float c, float s) {
  return make_float2(__fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s)), __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s)));
}

// The row's factor and scale for codes. 448 / amax is beyond fp32 for rows below 2^-119 (and their zeros would become NaN):
// their elements are first taken `up` by 2^64, which rounds nothing and leaves the codes what they are.
constexpr float kUp = 0x1p64f;
struct CodeFactors {
  float up, factor, scale;
};

__device__ __forceinline__ CodeFactors code_factors(float amax) {
  CodeFactors f{1.0f, 1.0f, 1.0f};
  if (amax > 0.0f) {
    if (amax < 0x1p-100f) f.up = kUp;
    f.factor = __fdiv_rn(448.0f, __fmul_rn(amax, f.up));
    f.scale = __fdiv_rn(amax, 448.0f);
  }
  return f;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  return x;
}

// 16 bytes that this kernel may overwrite later (q_out may be q): a plain load.
__device__ __forceinline__ uint4 piece_at(const uint8_t* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}

// A lane's rotary item of a row: byte offsets of its two pieces of 8 elements of `e` bytes.
template <bool kInter>
__device__ __forceinline__ uint32_t piece_a(uint32_t item, uint32_t e) { return (kInter ? 16u : 8u) * item * e; }
template <bool kInter>
__device__ __forceinline__ uint32_t piece_b(uint32_t item, uint32_t e, uint32_t half) {
  return kInter ? (16u * item + 8u) * e : (half + 8u * item) * e;
}

struct Turns {
  float c[8], s[8];
};

__device__ __forceinline__ Turns turns_of(const LatentStoreParams& p, int64_t pos, uint32_t item) {
  Turns t;
  const float4* row = reinterpret_cast<const float4*>(p.table + pos * p.table_stride + 8u * item);
  const uint32_t h4 = p.rotary / 8;  // the sines begin rotary / 2 floats on
  const float4 c0 = __ldg(row), c1 = __ldg(row + 1), s0 = __ldg(row + h4), s1 = __ldg(row + h4 + 1);
  t.c[0] = c0.x; t.c[1] = c0.y; t.c[2] = c0.z; t.c[3] = c0.w; t.c[4] = c1.x; t.c[5] = c1.y; t.c[6] = c1.z; t.c[7] = c1.w;
  t.s[0] = s0.x; t.s[1] = s0.y; t.s[2] = s0.z; t.s[3] = s0.w; t.s[4] = s1.x; t.s[5] = s1.y; t.s[6] = s1.z; t.s[7] = s1.w;
  return t;
}

template <bool kInter>
__device__ __forceinline__ void turn_item(const uint4& a, const uint4& b, const Turns& t, int bf16, float (&x)[16]) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 v = unpack2(w[i], bf16);
    x[2 * i] = v.x;
    x[2 * i + 1] = v.y;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int i0 = kInter ? 2 * i : i, i1 = kInter ? 2 * i + 1 : i + 8;
    const float2 y = turn(x[i0], x[i1], t.c[i], t.s[i]);
    x[i0] = y.x;
    x[i1] = y.y;
  }
}

__device__ __forceinline__ uint4 pack8(const float* x, int bf16) {
  return make_uint4(pack2(x[0], x[1], bf16), pack2(x[2], x[3], bf16), pack2(x[4], x[5], bf16), pack2(x[6], x[7], bf16));
}

__device__ __forceinline__ uint2 codes8(const float* x, float f) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = e4m3x2(__fmul_rn(x[4 * i], f), __fmul_rn(x[4 * i + 1], f)) |
           (e4m3x2(__fmul_rn(x[4 * i + 2], f), __fmul_rn(x[4 * i + 3], f)) << 16);
  return make_uint2(w[0], w[1]);
}

// CH: chunks of 256 latent dims; U: passes of query items a warp.
template <int FMT, bool kInter, int CH, int U>
__global__ void __launch_bounds__(kThreads, 4) kv_latent_rows(const __grid_constant__ LatentStoreParams p) {
  const uint32_t lane = threadIdx.x & 31u;
  const uint64_t nwarps = static_cast<uint64_t>(gridDim.x) * warps_per_cta();
  const uint32_t half = p.rotary / 2;
  grid_handover();
  for (uint64_t u = static_cast<uint64_t>(blockIdx.x) * warps_per_cta() + (threadIdx.x >> 5); u < p.num_units; u += nwarps) {
    const uint64_t t = u / p.units;
    const uint32_t unit = static_cast<uint32_t>(u - t * p.units);
    if (unit != 0u) {
      // -- the queries' rotary dims ----------------------------------------------------------
      const uint32_t sub = lane / p.iph, item = lane - sub * p.iph;
      const uint8_t* src = p.q + static_cast<int64_t>(t) * p.q_token;
      uint4 a[U], b[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const uint32_t h = ((unit - 1u) * U + j) * p.hpp + sub;
        a[j] = b[j] = make_uint4(0u, 0u, 0u, 0u);
        if (sub < p.hpp && h < p.q_heads) {
          const uint8_t* row = src + static_cast<int64_t>(h) * p.q_head;
          a[j] = piece_at(row + piece_a<kInter>(item, 2));
          b[j] = piece_at(row + piece_b<kInter>(item, 2, half));
        }
      }
      const LatentPlace at = place_of(p, t, false);
      if (!at.pos_ok) continue;
      const Turns turns = turns_of(p, at.pos, sub < p.hpp ? item : 0u);
      uint8_t* dst = p.q_out + static_cast<int64_t>(t) * p.qo_token;
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const uint32_t h = ((unit - 1u) * U + j) * p.hpp + sub;
        if (sub < p.hpp && h < p.q_heads) {
          float x[16];
          turn_item<kInter>(a[j], b[j], turns, p.bf16, x);
          uint8_t* row = dst + static_cast<int64_t>(h) * p.qo_head;
          *reinterpret_cast<uint4*>(row + piece_a<kInter>(item, 2)) = pack8(x, p.bf16);
          *reinterpret_cast<uint4*>(row + piece_b<kInter>(item, 2, half)) = pack8(x + 8, p.bf16);
        }
      }
      continue;
    }
    // -- the row -----------------------------------------------------------------------------
    const uint8_t* src = p.c + static_cast<int64_t>(t) * p.c_token;
    uint4 w[CH], g[CH], a = make_uint4(0u, 0u, 0u, 0u), b = a;
    const bool rot = lane < p.iph && p.rope > 0u;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const uint32_t d = 8u * (lane + 32u * i);
      w[i] = g[i] = make_uint4(0u, 0u, 0u, 0u);
      if (d < p.latent) {
        w[i] = piece_at(src + 2u * d);
        if (p.weight) g[i] = __ldg(reinterpret_cast<const uint4*>(p.weight + 2u * d));
      }
    }
    if (rot) {
      const uint8_t* row = p.r + static_cast<int64_t>(t) * p.r_token;
      a = piece_at(row + piece_a<kInter>(lane, 2));
      b = piece_at(row + piece_b<kInter>(lane, 2, half));
    }
    const LatentPlace at = place_of(p, t, lane == 0u);
    if (!at.pos_ok || !at.slot_ok) continue;
    float y[16];  // the rotary item
    if (rot) turn_item<kInter>(a, b, turns_of(p, at.pos, lane), p.bf16, y);
    uint8_t* dst = row_of(p, at.slot);
    uint8_t* rdst = dst + (FMT == KV_CACHE_SRC ? 2u : 1u) * p.latent;
    if (FMT == KV_CACHE_SRC && !p.weight) {
#pragma unroll
      for (int i = 0; i < CH; ++i)
        if (8u * (lane + 32u * i) < p.latent) *reinterpret_cast<uint4*>(dst + 16u * (lane + 32u * i)) = w[i];
    } else {
      float x[CH][8];
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = unpack2(v[j], p.bf16);
          x[i][2 * j] = f.x;
          x[i][2 * j + 1] = f.y;
          sum = __fmaf_rn(f.x, f.x, sum);
          sum = __fmaf_rn(f.y, f.y, sum);
        }
      }
      if (p.weight) {
        const float scale = rsqrtf(warp_sum(sum) / static_cast<float>(p.latent) + p.eps);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          const uint32_t v[4] = {g[i].x, g[i].y, g[i].z, g[i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = unpack2(v[j], p.bf16);
            x[i][2 * j] = __fmul_rn(__fmul_rn(x[i][2 * j], scale), f.x);
            x[i][2 * j + 1] = __fmul_rn(__fmul_rn(x[i][2 * j + 1], scale), f.y);
          }
        }
      }
      if constexpr (FMT == KV_CACHE_SRC) {
#pragma unroll
        for (int i = 0; i < CH; ++i)
          if (8u * (lane + 32u * i) < p.latent) *reinterpret_cast<uint4*>(dst + 16u * (lane + 32u * i)) = pack8(x[i], p.bf16);
      } else {
        float amax = 0.0f;  // (lanes without a chunk hold zeros)
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(x[i][j]));
        if (rot) {
#pragma unroll
          for (int j = 0; j < 16; ++j) amax = fmaxf(amax, fabsf(y[j]));
        }
        const CodeFactors f = code_factors(warp_absmax(amax));
        if (f.up != 1.0f) {  // (the whole warp)
#pragma unroll
          for (int i = 0; i < CH; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) x[i][j] = __fmul_rn(x[i][j], kUp);
          if (rot) {
#pragma unroll
            for (int j = 0; j < 16; ++j) y[j] = __fmul_rn(y[j], kUp);
          }
        }
#pragma unroll
        for (int i = 0; i < CH; ++i)
          if (8u * (lane + 32u * i) < p.latent) *reinterpret_cast<uint2*>(dst + 8u * (lane + 32u * i)) = codes8(x[i], f.factor);
        if (rot) {
          *reinterpret_cast<uint2*>(rdst + piece_a<kInter>(lane, 1)) = codes8(y, f.factor);
          *reinterpret_cast<uint2*>(rdst + piece_b<kInter>(lane, 1, half)) = codes8(y + 8, f.factor);
        }
        if (lane == 0u) p.scales[at.slot * p.scale_slot] = f.scale;
      }
    }
    if (FMT == KV_CACHE_SRC && rot) {
      *reinterpret_cast<uint4*>(rdst + piece_a<kInter>(lane, 2)) = pack8(y, p.bf16);
      *reinterpret_cast<uint4*>(rdst + piece_b<kInter>(lane, 2, half)) = pack8(y + 8, p.bf16);
    }
  }
}

template <int FMT>
__global__ void __launch_bounds__(kThreads) kv_latent_any(const __grid_constant__ LatentStoreParams p) {
  const uint32_t lane = threadIdx.x & 31u;
  const uint64_t nwarps = static_cast<uint64_t>(gridDim.x) * warps_per_cta();
  const uint32_t half = p.rotary / 2;
  grid_handover();
  for (uint64_t u = static_cast<uint64_t>(blockIdx.x) * warps_per_cta() + (threadIdx.x >> 5); u < p.num_units; u += nwarps) {
    const uint64_t t = u / p.units;
    const uint32_t unit = static_cast<uint32_t>(u - t * p.units);
    const LatentPlace at = place_of(p, t, unit == 0u && lane == 0u);
    if (!at.pos_ok) continue;
    const float* cs = p.table + at.pos * p.table_stride;
    const uint8_t* rsrc = unit == 0u ? p.r + static_cast<int64_t>(t) * p.r_token
                                     : p.q + static_cast<int64_t>(t) * p.q_token + static_cast<int64_t>(unit - 1u) * p.q_head;
    auto raw = [&](uint32_t d) { return *reinterpret_cast<const uint16_t*>(rsrc + 2u * d); };
    // both dims of pair i
    auto pair = [&](uint32_t i, uint32_t* d0, uint32_t* d1) {
      *d0 = p.interleaved ? 2u * i : i;
      *d1 = p.interleaved ? 2u * i + 1u : i + half;
      return turn(widen16(raw(*d0), p.bf16), widen16(raw(*d1), p.bf16), __ldg(cs + i), __ldg(cs + half + i));
    };
    uint32_t d0, d1;
    if (unit != 0u) {
      uint16_t* dst = reinterpret_cast<uint16_t*>(p.q_out + static_cast<int64_t>(t) * p.qo_token +
                                                  static_cast<int64_t>(unit - 1u) * p.qo_head);
      for (uint32_t i = lane; i < half; i += 32u) {
        const float2 y = pair(i, &d0, &d1);
        dst[d0] = round16(y.x, p.bf16);
        dst[d1] = round16(y.y, p.bf16);
      }
      for (uint32_t d = p.rotary + lane; d < p.rope; d += 32u) dst[d] = raw(d);
      continue;
    }
    if (!at.slot_ok) continue;
    const uint16_t* c = reinterpret_cast<const uint16_t*>(p.c + static_cast<int64_t>(t) * p.c_token);
    const uint16_t* weight = reinterpret_cast<const uint16_t*>(p.weight);
    float scale = 1.0f;
    if (p.weight) {
      float sum = 0.0f;
      for (uint32_t d = lane; d < p.latent; d += 32u) {
        const float x = widen16(c[d], p.bf16);
        sum = __fmaf_rn(x, x, sum);
      }
      scale = rsqrtf(warp_sum(sum) / static_cast<float>(p.latent) + p.eps);
    }
    auto latent = [&](uint32_t d) {
      const float x = widen16(c[d], p.bf16);
      return p.weight ? __fmul_rn(__fmul_rn(x, scale), widen16(__ldg(weight + d), p.bf16)) : x;
    };
    uint8_t* dst = row_of(p, at.slot);
    if constexpr (FMT == KV_CACHE_SRC) {
      uint16_t* o = reinterpret_cast<uint16_t*>(dst);
      for (uint32_t d = lane; d < p.latent; d += 32u) o[d] = p.weight ? round16(latent(d), p.bf16) : c[d];
      o += p.latent;
      for (uint32_t i = lane; i < half; i += 32u) {
        const float2 y = pair(i, &d0, &d1);
        o[d0] = round16(y.x, p.bf16);
        o[d1] = round16(y.y, p.bf16);
      }
      for (uint32_t d = p.rotary + lane; d < p.rope; d += 32u) o[d] = raw(d);
    } else {
      float amax = 0.0f;
      for (uint32_t d = lane; d < p.latent; d += 32u) amax = fmaxf(amax, fabsf(latent(d)));
      for (uint32_t i = lane; i < half; i += 32u) {
        const float2 y = pair(i, &d0, &d1);
        amax = fmaxf(amax, fmaxf(fabsf(y.x), fabsf(y.y)));
      }
      for (uint32_t d = p.rotary + lane; d < p.rope; d += 32u) amax = fmaxf(amax, fabsf(widen16(raw(d), p.bf16)));
      const CodeFactors f = code_factors(warp_absmax(amax));
      auto code = [&](float x) { return static_cast<uint8_t>(e4m3x2(__fmul_rn(__fmul_rn(x, f.up), f.factor), 0.0f)); };
      for (uint32_t d = lane; d < p.latent; d += 32u) dst[d] = code(latent(d));
      dst += p.latent;
      for (uint32_t i = lane; i < half; i += 32u) {
        const float2 y = pair(i, &d0, &d1);
        dst[d0] = code(y.x);
        dst[d1] = code(y.y);
      }
      for (uint32_t d = p.rotary + lane; d < p.rope; d += 32u) dst[d] = code(widen16(raw(d), p.bf16));
      if (lane == 0u) p.scales[at.slot * p.scale_slot] = f.scale;
    }
  }
}

template <int FMT, bool kInter, int CH>
kv_status launch_rows_of(LatentStoreParams& p, int64_t num_tokens, cudaStream_t stream) {
  // Few tokens: a pass of query items a warp, so that they spread over the SMs; else
  // four passes' loads in flight.
  int sms = 0;
  const kv_status st = current_sm_count(&sms);
  if (st != KV_OK) return st;
  const uint32_t passes = p.q_heads == 0u ? 0u : (p.q_heads + p.hpp - 1u) / p.hpp;
  const bool few = static_cast<uint64_t>(num_tokens) * (passes + 1u) < static_cast<uint64_t>(sms) * 16u;
  p.units = 1u + (few ? passes : (passes + 3u) / 4u);
  p.num_units = static_cast<uint64_t>(num_tokens) * p.units;
  return few ? launch(kv_latent_rows<FMT, kInter, CH, 1>, p.num_units, p, stream)
             : launch(kv_latent_rows<FMT, kInter, CH, 4>, p.num_units, p, stream);
}

template <int FMT, bool kInter>
kv_status launch_rows_ch(LatentStoreParams& p, int64_t num_tokens, cudaStream_t stream) {
  return p.latent <= 256u   ? launch_rows_of<FMT, kInter, 1>(p, num_tokens, stream)
         : p.latent <= 512u ? launch_rows_of<FMT, kInter, 2>(p, num_tokens, stream)
                            : launch_rows_of<FMT, kInter, 4>(p, num_tokens, stream);
}

// ---------------------------------------------------------------------------
// The gather
// ---------------------------------------------------------------------------

struct LatentGatherParams {
  const uint8_t* cache;
  const float* scales;
  uint8_t* out;
  const void* indices;
  int64_t out_token, cache_page, cache_slot, scale_slot;
  int64_t index_stride, size_limit, page_size;
  uint64_t num_items;
  uint32_t per_row;      // items of a row
  int idx64, bf16, narrow;
  kv_error_record* err;
};

constexpr int kGatherItems = 4;

// VEC: bytes of a 16-bit row per item, or (FMT e4m3fn) codes.
template <int FMT, int VEC>
__global__ void __launch_bounds__(kThreads) kv_latent_gather(const __grid_constant__ LatentGatherParams p) {
  constexpr int kOut = FMT == KV_CACHE_SRC ? VEC : 2 * VEC;
  grid_handover();
  const uint64_t round = static_cast<uint64_t>(blockDim.x) * kGatherItems;
  for (uint64_t first = static_cast<uint64_t>(blockIdx.x) * round; first < p.num_items; first += static_cast<uint64_t>(gridDim.x) * round) {
    const uint64_t row0 = first / p.per_row;
    const uint32_t in0 = static_cast<uint32_t>(first - row0 * p.per_row);
    int64_t slot[kGatherItems];
    uint64_t row[kGatherItems];
    uint32_t at[kGatherItems];
#pragma unroll
    for (int j = 0; j < kGatherItems; ++j) {
      const uint32_t i = in0 + threadIdx.x + static_cast<uint32_t>(j) * blockDim.x;
      const uint32_t r = i / p.per_row;
      row[j] = row0 + r;
      at[j] = i - r * p.per_row;
      slot[j] = -1;
      if (first + threadIdx.x + static_cast<uint64_t>(j) * blockDim.x < p.num_items)
        slot[j] = index_at(p.indices, static_cast<int64_t>(row[j]) * p.index_stride, p.idx64);
      else
        at[j] = 0xFFFFFFFFu;  // behind the last item
    }
    Chunk<VEC> c[kGatherItems];
    float scale[kGatherItems];
#pragma unroll
    for (int j = 0; j < kGatherItems; ++j) {
      scale[j] = 1.0f;
      if (slot[j] < 0 || slot[j] >= p.size_limit) {
        if (at[j] == 0u) record_oob(p.err, row[j]);
        slot[j] = -1;
        continue;
      }
      int64_t off;
      if (p.narrow) {
        const uint32_t s = static_cast<uint32_t>(slot[j]), n = static_cast<uint32_t>(p.page_size), pg = s / n;
        off = static_cast<int64_t>(pg) * p.cache_page + static_cast<int64_t>(s - pg * n) * p.cache_slot;
      } else {
        off = paged_offset(slot[j], p.page_size, p.cache_page, p.cache_slot);
      }
      ld_stream(c[j], p.cache + off + static_cast<uint64_t>(at[j]) * VEC);
      if constexpr (FMT == KV_CACHE_E4M3FN) scale[j] = __ldg(p.scales + slot[j] * p.scale_slot);
    }
#pragma unroll
    for (int j = 0; j < kGatherItems; ++j) {
      if (slot[j] < 0) continue;
      uint8_t* dst = p.out + static_cast<int64_t>(row[j]) * p.out_token + static_cast<uint64_t>(at[j]) * kOut;
      if constexpr (FMT == KV_CACHE_SRC) {
        st_stream(dst, c[j]);
      } else if constexpr (VEC == 1) {
        *reinterpret_cast<uint16_t*>(dst) = round16(__fmul_rn(f32_from_e4m3(c[j].h & 0xFFu), scale[j]), p.bf16);
      } else {
        Chunk<16> o[2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float2 v = mul2_rn(widen2<false>(f16x2_from_e4m3x2(c[j].w[i] >> (16 * y))), scale[j]);
            o[i >> 1].w[2 * (i & 1) + y] = pack2(v.x, v.y, p.bf16);
          }
        st_stream(dst, o[0]);
        st_stream(dst + 16, o[1]);
      }
    }
  }
}

template <int FMT, int VEC>
kv_status launch_gather(LatentGatherParams& p, int64_t num_tokens, int64_t row_bytes, cudaStream_t stream) {
  p.per_row = static_cast<uint32_t>(row_bytes / VEC);
  p.num_items = static_cast<uint64_t>(num_tokens) * p.per_row;
  return launch(kv_latent_gather<FMT, VEC>, (p.num_items + 32u * kGatherItems - 1) / (32u * kGatherItems), p, stream);
}

}  // namespace
}  // namespace kvimpl

// ---------------------------------------------------------------------------
// C ABI
// ---------------------------------------------------------------------------

using namespace kvimpl;

extern "C" kv_status kv_store_latent(const void* c, const void* r, void* cache, const void* indices,
                                     kv_index_dtype index_dtype, int64_t index_stride, int64_t num_tokens,
                                     int32_t latent_dim, int32_t rope_dim, kv_src_dtype src_dtype,
                                     const kv_latent_strides* s, int64_t page_size, int64_t size_limit,
                                     const void* weight, float eps, const kv_rope* rope, kv_cache_format format,
                                     float* scales, kv_error_record* d_err, kv_stream_t stream_) {
  if (num_tokens < 0) return KV_ERR_INVALID_ARG;
  if (format != KV_CACHE_SRC && format != KV_CACHE_E4M3FN) return KV_ERR_INVALID_ARG;
  if (num_tokens == 0) return KV_OK;
  if (!c || !cache || !indices || !s || !d_err || (u64(d_err) & 7u) != 0) return KV_ERR_INVALID_ARG;
  if (index_dtype != KV_INDEX_I32 && index_dtype != KV_INDEX_I64) return KV_ERR_INVALID_ARG;
  if (src_dtype != KV_SRC_F16 && src_dtype != KV_SRC_BF16) return KV_ERR_INVALID_ARG;
  if (index_stride < 1 || latent_dim < 1 || rope_dim < 0 || size_limit < 0 || page_size < 1 || !(eps >= 0.0f) || std::isinf(eps))
    return KV_ERR_INVALID_ARG;
  if (rope_dim > 0 && (!r || !rope)) return KV_ERR_INVALID_ARG;
  const bool fp8 = format == KV_CACHE_E4M3FN;
  if (fp8 && (!scales || (u64(scales) & 3u) != 0 || s->scale_slot < 1)) return KV_ERR_INVALID_ARG;
  kv_rope rp = {};
  if (rope_dim > 0) {
    rp = *rope;
    if ((!rp.cos_sin && rp.rotary_dim > 0) || !rp.positions || rp.position_stride < 1 || rp.max_position < 0 ||
        (rp.position_dtype != KV_INDEX_I32 && rp.position_dtype != KV_INDEX_I64) || rp.rotary_dim < 0 ||
        rp.rotary_dim > rope_dim || (rp.rotary_dim & 1) != 0 || rp.cos_sin_stride < rp.rotary_dim || (u64(rp.cos_sin) & 3u) != 0)
      return KV_ERR_INVALID_ARG;
    if (rp.q && (!rp.q_out || rp.num_q_heads < 1)) return KV_ERR_INVALID_ARG;
    if ((u64(rp.positions) & (rp.position_dtype == KV_INDEX_I64 ? 7u : 3u)) != 0) return KV_ERR_INVALID_ARG;
  }
  if ((u64(indices) & (index_dtype == KV_INDEX_I64 ? 7u : 3u)) != 0) return KV_ERR_INVALID_ARG;
  uint64_t in_bits = u64(c) | u64(s->c_token) | u64(weight);
  if (rope_dim > 0) in_bits |= u64(r) | u64(s->r_token);
  if (rp.q) in_bits |= u64(rp.q) | u64(rp.q_out) | u64(rp.q_token) | u64(rp.q_head) | u64(rp.qo_token) | u64(rp.qo_head);
  const uint64_t cache_bits = u64(cache) | u64(s->cache_page) | u64(s->cache_slot);
  if (((in_bits | (fp8 ? 0u : cache_bits)) & 1u) != 0) return KV_ERR_INVALID_ARG;
  if (latent_dim > kMaxRow || rope_dim > kMaxRow - latent_dim || num_tokens > (int64_t{1} << 40)) return KV_ERR_UNSUPPORTED;
  {
    const void* in[12] = {c, indices, cache, d_err};
    int n = 4;
    if (rope_dim > 0) {
      in[n++] = r;
      in[n++] = rp.positions;
      if (rp.rotary_dim > 0) in[n++] = rp.cos_sin;
    }
    if (rp.q) {
      in[n++] = rp.q;
      in[n++] = rp.q_out;
    }
    if (weight) in[n++] = weight;
    if (fp8) in[n++] = scales;
    const kv_status cs = classify_here(in, n);
    if (cs != KV_OK) return cs;
  }

  LatentStoreParams p = {};
  p.c = static_cast<const uint8_t*>(c);
  p.r = static_cast<const uint8_t*>(r);
  p.weight = static_cast<const uint8_t*>(weight);
  p.cache = static_cast<uint8_t*>(cache);
  p.scales = scales;
  p.c_token = s->c_token;
  p.r_token = s->r_token;
  p.cache_page = s->cache_page;
  p.cache_slot = s->cache_slot;
  p.scale_slot = s->scale_slot;
  if (rp.q) {
    p.q = static_cast<const uint8_t*>(rp.q);
    p.q_out = static_cast<uint8_t*>(rp.q_out);
    p.q_token = rp.q_token; p.q_head = rp.q_head;
    p.qo_token = rp.qo_token; p.qo_head = rp.qo_head;
    p.q_heads = static_cast<uint32_t>(rp.num_q_heads);
  }
  p.indices = indices;
  p.positions = rp.positions;
  p.table = rp.cos_sin;
  p.index_stride = index_stride;
  p.position_stride = rp.position_stride;
  p.table_stride = rp.cos_sin_stride;
  p.max_position = rp.max_position;
  p.size_limit = size_limit;
  p.page_size = page_size;
  p.latent = static_cast<uint32_t>(latent_dim);
  p.rope = static_cast<uint32_t>(rope_dim);
  p.rotary = static_cast<uint32_t>(rp.rotary_dim);
  p.eps = eps;
  p.idx64 = index_dtype == KV_INDEX_I64;
  p.pos64 = rp.position_dtype == KV_INDEX_I64;
  p.bf16 = src_dtype == KV_SRC_BF16;
  p.interleaved = rp.interleaved != 0;
  p.narrow = size_limit <= INT32_MAX && page_size <= INT32_MAX;
  p.err = d_err;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);

  if (rope_dim > 0 && rp.rotary_dim > 0) in_bits |= u64(rp.cos_sin) | u64(4 * rp.cos_sin_stride);
  const bool rows = latent_dim % 8 == 0 && rope_dim % 16 == 0 && rope_dim <= 512 && rp.rotary_dim == rope_dim &&
                    (in_bits & 15u) == 0 && (cache_bits & (fp8 ? 7u : 15u)) == 0;
  if (rows) {
    p.iph = p.rope / 16u;
    p.hpp = p.iph > 0u ? 32u / p.iph : 1u;
    if (fp8)
      return p.interleaved ? launch_rows_ch<KV_CACHE_E4M3FN, true>(p, num_tokens, stream)
                           : launch_rows_ch<KV_CACHE_E4M3FN, false>(p, num_tokens, stream);
    return p.interleaved ? launch_rows_ch<KV_CACHE_SRC, true>(p, num_tokens, stream)
                         : launch_rows_ch<KV_CACHE_SRC, false>(p, num_tokens, stream);
  }
  p.units = 1u + p.q_heads;
  p.num_units = static_cast<uint64_t>(num_tokens) * p.units;
  return fp8 ? launch(kv_latent_any<KV_CACHE_E4M3FN>, p.num_units, p, stream)
             : launch(kv_latent_any<KV_CACHE_SRC>, p.num_units, p, stream);
}

extern "C" kv_status kv_gather_latent(const void* cache, const float* scales, void* out, const void* indices,
                                      kv_index_dtype index_dtype, int64_t index_stride, int64_t num_tokens,
                                      int32_t row_dim, kv_src_dtype out_dtype, const kv_latent_strides* s,
                                      int64_t page_size, int64_t size_limit, kv_cache_format format,
                                      kv_error_record* d_err, kv_stream_t stream_) {
  if (num_tokens < 0) return KV_ERR_INVALID_ARG;
  if (format != KV_CACHE_SRC && format != KV_CACHE_E4M3FN) return KV_ERR_INVALID_ARG;
  if (num_tokens == 0) return KV_OK;
  if (!cache || !out || !indices || !s || !d_err || (u64(d_err) & 7u) != 0) return KV_ERR_INVALID_ARG;
  if (index_dtype != KV_INDEX_I32 && index_dtype != KV_INDEX_I64) return KV_ERR_INVALID_ARG;
  if (out_dtype != KV_SRC_F16 && out_dtype != KV_SRC_BF16) return KV_ERR_INVALID_ARG;
  if (index_stride < 1 || row_dim < 1 || page_size < 1 || size_limit < 0) return KV_ERR_INVALID_ARG;
  const bool fp8 = format == KV_CACHE_E4M3FN;
  if (fp8 && (!scales || (u64(scales) & 3u) != 0 || s->scale_slot < 1)) return KV_ERR_INVALID_ARG;
  if ((u64(indices) & (index_dtype == KV_INDEX_I64 ? 7u : 3u)) != 0) return KV_ERR_INVALID_ARG;
  const uint64_t out_bits = u64(out) | u64(s->c_token);
  const uint64_t cache_bits = u64(cache) | u64(s->cache_page) | u64(s->cache_slot);
  if (((out_bits | (fp8 ? 0u : cache_bits)) & 1u) != 0) return KV_ERR_INVALID_ARG;
  if (row_dim > kMaxRow || num_tokens > (int64_t{1} << 40)) return KV_ERR_UNSUPPORTED;
  {
    const void* in[5] = {cache, out, indices, d_err, scales};
    const kv_status cs = classify_here(in, fp8 ? 5 : 4);
    if (cs != KV_OK) return cs;
  }
  LatentGatherParams p = {};
  p.cache = static_cast<const uint8_t*>(cache);
  p.scales = scales;
  p.out = static_cast<uint8_t*>(out);
  p.indices = indices;
  p.out_token = s->c_token;
  p.cache_page = s->cache_page;
  p.cache_slot = s->cache_slot;
  p.scale_slot = s->scale_slot;
  p.index_stride = index_stride;
  p.size_limit = size_limit;
  p.page_size = page_size;
  p.idx64 = index_dtype == KV_INDEX_I64;
  p.bf16 = out_dtype == KV_SRC_BF16;
  p.narrow = size_limit <= INT32_MAX && page_size <= INT32_MAX;
  p.err = d_err;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (fp8)
    return row_dim % 16 == 0 && ((out_bits | cache_bits) & 15u) == 0
               ? launch_gather<KV_CACHE_E4M3FN, 16>(p, num_tokens, row_dim, stream)
               : launch_gather<KV_CACHE_E4M3FN, 1>(p, num_tokens, row_dim, stream);
  const int64_t bytes = 2 * static_cast<int64_t>(row_dim);
  switch (pow2_align(out_bits | cache_bits | u64(bytes))) {
    case 32: return launch_gather<KV_CACHE_SRC, 32>(p, num_tokens, bytes, stream);
    case 16: return launch_gather<KV_CACHE_SRC, 16>(p, num_tokens, bytes, stream);
    default: return launch_gather<KV_CACHE_SRC, 2>(p, num_tokens, bytes, stream);
  }
}
