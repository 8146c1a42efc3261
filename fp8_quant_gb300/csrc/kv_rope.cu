// Appending K and V to a paged cache with the position rotation applied on the
// way (kv_store_rope), and the dequantising gather of the 4-bit cache
// (kv_gather_fp4).
//
// What is computed is in kvstore.h.  The path is a stream: per token the rows
// of Q, K and V are read once and written once, with six fp32 operations per
// rotated pair, so bytes bound it.
//
//  * kv_rope_rows   head dims that are multiples of 16 up to 512, contiguous dims
//                   and 16-byte pieces.  A lane's item is 16 dims of a head as
//                   two pieces of 8: both halves of eight pairs, so that
//                   whatever they need is in the lane (an e2m1 block of the
//                   split-half rotation is two lanes' and takes one shuffle for
//                   its maximum, which all lanes execute).  The lanes of a warp are the items of 32 * 16
//                   / head_dim heads; a warp goes over U such groups of a
//                   token's Q, K and V heads with all their loads in flight
//                   before the first store, and since a lane keeps its item
//                   index, its eight cosines and sines are loaded once for all.
//                   Row loads do not wait for the slot or the position.
//  * kv_rope_any    any layout: one warp per (token, head), a lane per rotated
//                   pair (or unrotated dim, or 16-dim block of an e2m1 row).
//  * kv_gather_fp4_blocks  one lane per 16-dim block: 8 code bytes and a scale
//                   in, 32 bytes out.
//
// Measured on one GB300 (32 query and 8 KV heads of 128, q in and out):
// 32,768 fp16 tokens into a 16-bit cache, 822 MB, 145 us, 5.7 TB/s, 84 % of a
// copy's rate (the table's rows of scattered positions come on top of the counted bytes),
// and bf16 ones into an e4m3fn cache 149 us; 8,191 bf16 tokens into the 4-bit cache 42 us; their
// gather 11.8 us; 256 tokens into an e4m3fn cache 4.1 us and one token 2.1 us (calls
// captured one behind the other), launch and three dependent loads.
#include <cmath>

#include "kv_fp4.cuh"
#include "kv_host.h"

namespace kvimpl {
namespace {

// One of Q, K, V: where its rows come from and go to.
struct RopeSide {
  const uint8_t* src;
  uint8_t* dst;
  int64_t src_token, src_head, src_dim;            // input byte strides
  int64_t dst_page, dst_slot, dst_head, dst_dim;   // cache byte strides (Q: dst_slot per token)
  const float* inv;                                // inverse tensor scale, or null: 1
  uint8_t* scales;                                 // e2m1 block scales
  int64_t sc_page, sc_slot, sc_head;
};

struct RopeParams {
  RopeSide side[3];  // Q, K, V
  const void* indices;
  const void* positions;
  const float* table;
  int64_t index_stride, position_stride, table_stride;
  int64_t max_position, size_limit, page_size;
  uint64_t num_units;
  uint32_t q_heads, kv_heads, per_token;  // per_token: units per token
  uint32_t head_dim, rotary;
  int pos64, idx64, bf16, interleaved;
  kv_error_record* err;
};

__device__ __forceinline__ int64_t load_index(const void* p, int64_t i, int is64) {
  return is64 ? static_cast<int64_t>(__ldg(static_cast<const long long*>(p) + i))
              : static_cast<int64_t>(__ldg(static_cast<const int*>(p) + i));
}

// a' and b' of a pair: every product and sum rounded on its own (the library
// is built without contraction; the intrinsics state it).
__device__ __forceinline__ float2 rotate_pair(float a, float b, float c, float s) {
  return make_float2(__fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s)),
                     __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s)));
}

// Byte offset of cache row `slot`, in the caches and (with their strides) in
// the block scales.
__device__ __forceinline__ void slot_parts(const RopeParams& p, int64_t slot, int64_t* page,
                                           int64_t* off) {
  *page = slot / p.page_size;
  *off = slot - *page * p.page_size;
}

template <int FMT>
__global__ void __launch_bounds__(kThreads) kv_rope_any(const __grid_constant__ RopeParams p) {
  const uint32_t lane = threadIdx.x & 31u;
  const uint64_t nwarps = static_cast<uint64_t>(gridDim.x) * warps_per_cta();
  grid_handover();
  for (uint64_t u = static_cast<uint64_t>(blockIdx.x) * warps_per_cta() + (threadIdx.x >> 5);
       u < p.num_units; u += nwarps) {
    const uint64_t tu = u / p.per_token;
    const int64_t t = static_cast<int64_t>(tu);
    uint32_t h = static_cast<uint32_t>(u - tu * p.per_token);
    const bool first = h == 0;
    int which = 0;  // 0 Q, 1 K, 2 V
    if (h >= p.q_heads) {
      h -= p.q_heads;
      which = 1;
      if (h >= p.kv_heads) {
        h -= p.kv_heads;
        which = 2;
      }
    }
    const int64_t slot = load_index(p.indices, t * p.index_stride, p.idx64);
    const int64_t pos = load_index(p.positions, t * p.position_stride, p.pos64);
    const bool pos_ok = pos >= 0 && pos < p.max_position;
    const bool slot_ok = slot >= 0 && slot < p.size_limit;
    if (first && lane == 0 && !(pos_ok && slot_ok)) record_oob(p.err, tu);
    if (!pos_ok || (which != 0 && !slot_ok)) continue;

    const RopeSide& sd = p.side[which];
    const uint8_t* src = sd.src + t * sd.src_token + static_cast<int64_t>(h) * sd.src_head;
    const float* cs = p.table + pos * p.table_stride;
    const uint32_t half = which == 2 ? 0u : p.rotary / 2;
    const uint32_t rot = 2 * half;
    int64_t page = 0, off = t;
    if (which != 0) slot_parts(p, slot, &page, &off);
    uint8_t* dst = sd.dst + page * sd.dst_page + off * sd.dst_slot +
                   static_cast<int64_t>(h) * sd.dst_head;
    auto in16 = [&](uint32_t d) {
      return *reinterpret_cast<const uint16_t*>(src + static_cast<int64_t>(d) * sd.src_dim);
    };
    auto in = [&](uint32_t d) { return widen16(in16(d), p.bf16); };

    if (FMT == KV_CACHE_E2M1 && which != 0) {
      const float inv = sd.inv ? __ldg(sd.inv) : 1.0f;
      for (uint32_t b = lane; b < p.head_dim / kFp4Block; b += 32u) {
        float y[kFp4Block], amax = 0.0f;
#pragma unroll
        for (int i = 0; i < kFp4Block; ++i) {
          const uint32_t d = b * kFp4Block + i;
          float x = in(d);
          if (d < rot) {
            const uint32_t pair = p.interleaved ? d / 2 : (d < half ? d : d - half);
            const bool second = p.interleaved ? (d & 1u) != 0 : d >= half;
            const float other = in(p.interleaved ? (d ^ 1u) : (second ? d - half : d + half));
            const float c = __ldg(cs + pair), s = __ldg(cs + half + pair);
            x = second ? rotate_pair(other, x, c, s).y : rotate_pair(x, other, c, s).x;
          }
          y[i] = __fmul_rn(x, inv);
          amax = fmaxf(amax, fabsf(y[i]));
        }
        float r;
        const uint32_t sc = fp4_block_scale(amax, &r);
#pragma unroll
        for (int i = 0; i < kFp4Block; ++i) y[i] = __fmul_rn(y[i], r);
        const uint32_t c0 = e2m1x8(y), c1 = e2m1x8(y + 8);
        uint8_t* o = dst + b * (kFp4Block / 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          o[i] = static_cast<uint8_t>(c0 >> (8 * i));
          o[4 + i] = static_cast<uint8_t>(c1 >> (8 * i));
        }
        sd.scales[page * sd.sc_page + off * sd.sc_slot + static_cast<int64_t>(h) * sd.sc_head + b] =
            static_cast<uint8_t>(sc);
      }
      continue;
    }
    const bool fp8 = FMT == KV_CACHE_E4M3FN && which != 0;
    const float inv = fp8 && sd.inv ? __ldg(sd.inv) : 1.0f;
    auto out = [&](uint32_t d, float x) {
      uint8_t* o = dst + static_cast<int64_t>(d) * sd.dst_dim;
      if (fp8) {
        *o = static_cast<uint8_t>(e4m3x2(__fmul_rn(x, inv), 0.0f));
      } else {
        *reinterpret_cast<uint16_t*>(o) = round16(x, p.bf16);
      }
    };
    // one lane owns both dims of a pair, so that q_out may be q
    for (uint32_t i = lane; i < half; i += 32u) {
      const uint32_t d0 = p.interleaved ? 2 * i : i, d1 = p.interleaved ? 2 * i + 1 : i + half;
      const float2 r = rotate_pair(in(d0), in(d1), __ldg(cs + i), __ldg(cs + half + i));
      out(d0, r.x);
      out(d1, r.y);
    }
    for (uint32_t d = rot + lane; d < p.head_dim; d += 32u) {
      if (fp8) {
        out(d, in(d));
      } else {
        *reinterpret_cast<uint16_t*>(dst + static_cast<int64_t>(d) * sd.dst_dim) = in16(d);
      }
    }
  }
}

// 16 bytes that this kernel may overwrite later (q_out may be q): a plain load.
__device__ __forceinline__ uint4 ld_piece(const uint8_t* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}

struct RopeRowParams {
  RopeParams r;
  uint32_t iph, hpp;      // items per head; heads per pass
  uint32_t heads;         // of Q, K and V together
  uint32_t units;         // per token
  int narrow;             // slots and pages fit 32 bits
};

template <int FMT, bool kInter, int U>
__global__ void __launch_bounds__(kThreads) kv_rope_rows(const __grid_constant__ RopeRowParams p) {
  const RopeParams& r = p.r;
  const uint32_t lane = threadIdx.x & 31u;
  const uint64_t nwarps = static_cast<uint64_t>(gridDim.x) * warps_per_cta();
  const uint32_t sub = lane / p.iph, item = lane - sub * p.iph;
  const uint32_t half = r.rotary / 2;
  const bool turns = item < r.rotary / 16;  // a rotated item (of Q and K)
  const uint32_t qk = r.q_heads + r.kv_heads;
  grid_handover();
  for (uint64_t u = static_cast<uint64_t>(blockIdx.x) * warps_per_cta() + (threadIdx.x >> 5);
       u < r.num_units; u += nwarps) {
    const uint64_t tu = u / p.units;
    const int64_t t = static_cast<int64_t>(tu);
    const uint32_t first = static_cast<uint32_t>(u - tu * p.units) * U * p.hpp;  // the unit's first head
    uint4 a[U], b[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const uint32_t hs = first + j * p.hpp + sub;
      a[j] = b[j] = make_uint4(0u, 0u, 0u, 0u);
      if (sub < p.hpp && hs < p.heads) {
        const int side = hs < r.q_heads ? 0 : hs < qk ? 1 : 2;
        const RopeSide& sd = r.side[side];
        const uint32_t h = hs - (side == 0 ? 0u : side == 1 ? r.q_heads : qk);
        const uint8_t* src = sd.src + t * sd.src_token + static_cast<int64_t>(h) * sd.src_head;
        const bool apart = !kInter && turns && side != 2;  // the pieces are half a rotation apart
        a[j] = ld_piece(src + (apart ? 16u * item : 32u * item));
        b[j] = ld_piece(src + (apart ? 2u * half + 16u * item : 32u * item + 16u));
      }
    }
    const int64_t slot = load_index(r.indices, t * r.index_stride, r.idx64);
    const int64_t pos = load_index(r.positions, t * r.position_stride, r.pos64);
    const bool pos_ok = pos >= 0 && pos < r.max_position;
    const bool slot_ok = slot >= 0 && slot < r.size_limit;
    if (first == 0u && lane == 0u && !(pos_ok && slot_ok)) record_oob(r.err, tu);
    if (!pos_ok) continue;
    float c[8], s[8];
    if (turns && first < qk) {
      const float4* row = reinterpret_cast<const float4*>(r.table + pos * r.table_stride + 8u * item);
      const float4 c0 = __ldg(row), c1 = __ldg(row + 1), s0 = __ldg(row + half / 4), s1 = __ldg(row + half / 4 + 1);
      c[0] = c0.x; c[1] = c0.y; c[2] = c0.z; c[3] = c0.w; c[4] = c1.x; c[5] = c1.y; c[6] = c1.z; c[7] = c1.w;
      s[0] = s0.x; s[1] = s0.y; s[2] = s0.z; s[3] = s0.w; s[4] = s1.x; s[5] = s1.y; s[6] = s1.z; s[7] = s1.w;
    }
    int64_t page = 0, off = 0;
    if (slot_ok) {
      if (p.narrow) {
        const uint32_t pg = static_cast<uint32_t>(slot) / static_cast<uint32_t>(r.page_size);
        page = pg;
        off = static_cast<uint32_t>(slot) - pg * static_cast<uint32_t>(r.page_size);
      } else {
        slot_parts(r, slot, &page, &off);
      }
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const uint32_t hs = first + j * p.hpp + sub;
      const int side = hs < r.q_heads ? 0 : hs < qk ? 1 : 2;
      const bool live = sub < p.hpp && hs < p.heads && (side == 0 || slot_ok);
      const RopeSide& sd = r.side[side];
      const uint32_t h = hs - (side == 0 ? 0u : side == 1 ? r.q_heads : qk);
      const bool rot = turns && side != 2;
      uint8_t* dst = side == 0 ? sd.dst + t * sd.dst_slot : sd.dst + page * sd.dst_page + off * sd.dst_slot;
      dst += static_cast<int64_t>(h) * sd.dst_head;
      uint32_t w[8] = {a[j].x, a[j].y, a[j].z, a[j].w, b[j].x, b[j].y, b[j].z, b[j].w};
      const bool plain = FMT == KV_CACHE_SRC || side == 0;  // 16-bit rows
      // x[0 .. 7]: piece a, x[8 .. 15]: piece b, in fp32 (0 where they are copied)
      float x[16] = {};
      if (plain && !rot) {
        if (live) {
          *reinterpret_cast<uint4*>(dst + 32u * item) = a[j];
          *reinterpret_cast<uint4*>(dst + 32u * item + 16u) = b[j];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 v = unpack2(w[i], r.bf16);
          x[2 * i] = v.x;
          x[2 * i + 1] = v.y;
        }
        if (rot) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int i0 = kInter ? 2 * i : i, i1 = kInter ? 2 * i + 1 : i + 8;
            const float2 y = rotate_pair(x[i0], x[i1], c[i], s[i]);
            x[i0] = y.x;
            x[i1] = y.y;
          }
        }
        if (plain) {
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = pack2(x[2 * i], x[2 * i + 1], r.bf16);
          if (live) {
            const uint32_t at_a = kInter ? 32u * item : 16u * item;
            const uint32_t at_b = kInter ? 32u * item + 16u : 2u * half + 16u * item;
            *reinterpret_cast<uint4*>(dst + at_a) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(dst + at_b) = make_uint4(w[4], w[5], w[6], w[7]);
          }
        } else {
          const float inv = sd.inv ? __ldg(sd.inv) : 1.0f;
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = __fmul_rn(x[i], inv);
          if constexpr (FMT == KV_CACHE_E4M3FN) {
            const bool apart = !kInter && rot;
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = e4m3x2(x[4 * i], x[4 * i + 1]) | (e4m3x2(x[4 * i + 2], x[4 * i + 3]) << 16);
            if (live) {
              if (apart) {
                *reinterpret_cast<uint2*>(dst + 8u * item) = make_uint2(o[0], o[1]);
                *reinterpret_cast<uint2*>(dst + half + 8u * item) = make_uint2(o[2], o[3]);
              } else {
                *reinterpret_cast<uint4*>(dst + 16u * item) = make_uint4(o[0], o[1], o[2], o[3]);
              }
            }
          }
        }
      }
      if constexpr (FMT == KV_CACHE_E2M1) {
        // the lanes of a 16-bit row come here too, with nothing to write: the shuffles name every lane
        const bool apart = !kInter && rot;
        float ma = 0.0f, mb = 0.0f;
        if (!plain) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            ma = fmaxf(ma, fabsf(x[i]));
            mb = fmaxf(mb, fabsf(x[8 + i]));
          }
        }
        // the other half of each block: the neighbour's where the pieces are apart, else the lane's own
        float fa = fmaxf(ma, mb), fb = fa;
        if constexpr (!kInter) {
          const float na = __shfl_xor_sync(0xFFFFFFFFu, ma, 1), nb = __shfl_xor_sync(0xFFFFFFFFu, mb, 1);
          if (apart) {
            fa = fmaxf(ma, na);
            fb = fmaxf(mb, nb);
          }
        }
        if (!plain) {
          float ra, rb;
          const uint32_t sa = fp4_block_scale(fa, &ra);
          uint32_t sb = sa;
          rb = ra;
          if (apart) sb = fp4_block_scale(fb, &rb);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[i] = __fmul_rn(x[i], ra);
            x[8 + i] = __fmul_rn(x[8 + i], rb);
          }
          const uint32_t ca = e2m1x8(x), cb = e2m1x8(x + 8);
          if (live) {
            uint8_t* sc = sd.scales + page * sd.sc_page + off * sd.sc_slot + static_cast<int64_t>(h) * sd.sc_head;
            if (apart) {
              *reinterpret_cast<uint32_t*>(dst + 4u * item) = ca;
              *reinterpret_cast<uint32_t*>(dst + half / 2 + 4u * item) = cb;
              sc[(item & 1u ? half / 16 : 0u) + item / 2] = static_cast<uint8_t>(item & 1u ? sb : sa);
            } else {
              *reinterpret_cast<uint2*>(dst + 8u * item) = make_uint2(ca, cb);
              sc[item] = static_cast<uint8_t>(sa);
            }
          }
        }
      }
    }
  }
}

template <int FMT, bool kInter>
kv_status launch_rope_rows(RopeRowParams& p, int64_t num_tokens, cudaStream_t stream) {
  // Few tokens: a pass per warp, so that they spread over the SMs (one call
  // is then one round of loads); else 4 passes' loads in flight per warp.
  int sms = 0;
  const kv_status st = current_sm_count(&sms);
  if (st != KV_OK) return st;
  const uint32_t passes = (p.heads + p.hpp - 1) / p.hpp;
  const bool few = static_cast<uint64_t>(num_tokens) * passes < static_cast<uint64_t>(sms) * 16u;
  p.units = few ? passes : (passes + 3u) / 4u;
  p.r.num_units = static_cast<uint64_t>(num_tokens) * p.units;
  return few ? launch(kv_rope_rows<FMT, kInter, 1>, p.r.num_units, p, stream)
             : launch(kv_rope_rows<FMT, kInter, 4>, p.r.num_units, p, stream);
}

// ---------------------------------------------------------------------------
// The gather of a 4-bit cache.
// ---------------------------------------------------------------------------

struct Fp4Side {
  const uint8_t* codes;
  const uint8_t* scales;
  uint8_t* out;
  int64_t page, slot, head;           // codes
  int64_t sc_page, sc_slot, sc_head;  // block scales
  int64_t out_token, out_head;
  const float* scale;
};

struct Fp4GatherParams {
  Fp4Side side[2];
  const void* indices;
  int64_t index_stride, size_limit, page_size;
  uint64_t num_items;     // tokens * 2 * heads * blocks
  uint32_t heads, blocks; // blocks of 16 dims per head
  int idx64, bf16, wide;  // wide: 8-byte code loads and 16-byte output stores
  kv_error_record* err;
};

__global__ void __launch_bounds__(kThreads)
    kv_gather_fp4_blocks(const __grid_constant__ Fp4GatherParams p) {
  grid_handover();
  const uint64_t step = static_cast<uint64_t>(gridDim.x) * blockDim.x;
  const uint32_t per_side = p.heads * p.blocks, per_token = 2u * per_side;
  for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < p.num_items;
       i += step) {
    const uint64_t t = i / per_token;
    uint32_t r = static_cast<uint32_t>(i - t * per_token);
    const bool first = r == 0;
    const int64_t slot = load_index(p.indices, static_cast<int64_t>(t) * p.index_stride, p.idx64);
    if (slot < 0 || slot >= p.size_limit) {
      if (first) record_oob(p.err, t);
      continue;
    }
    const Fp4Side& sd = p.side[r >= per_side ? 1 : 0];
    if (r >= per_side) r -= per_side;
    const uint32_t h = r / p.blocks, b = r - h * p.blocks;
    const int64_t page = slot / p.page_size, off = slot - page * p.page_size;
    const uint8_t* c = sd.codes + page * sd.page + off * sd.slot + static_cast<int64_t>(h) * sd.head +
                       b * (kFp4Block / 2);
    const uint32_t sc = sd.scales[page * sd.sc_page + off * sd.sc_slot +
                                  static_cast<int64_t>(h) * sd.sc_head + b];
    uint32_t w[2];
    if (p.wide) {
      const uint2 v = *reinterpret_cast<const uint2*>(c);
      w[0] = v.x;
      w[1] = v.y;
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        w[j] = c[4 * j] | (uint32_t{c[4 * j + 1]} << 8) | (uint32_t{c[4 * j + 2]} << 16) |
               (uint32_t{c[4 * j + 3]} << 24);
    }
    const float s = f32_from_e4m3(sc);
    const float g = sd.scale ? __ldg(sd.scale) : 1.0f;
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t f[4];
      f16x2_from_e2m1x8(w[j], f);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 x = widen2<false>(f[q]);
        o[4 * j + q] = pack2(__fmul_rn(__fmul_rn(x.x, s), g), __fmul_rn(__fmul_rn(x.y, s), g), p.bf16);
      }
    }
    uint8_t* dst = sd.out + static_cast<int64_t>(t) * sd.out_token +
                   static_cast<int64_t>(h) * sd.out_head + b * (2 * kFp4Block);
    if (p.wide) {
      *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<uint4*>(dst + 16) = make_uint4(o[4], o[5], o[6], o[7]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        reinterpret_cast<uint16_t*>(dst)[2 * j] = static_cast<uint16_t>(o[j]);
        reinterpret_cast<uint16_t*>(dst)[2 * j + 1] = static_cast<uint16_t>(o[j] >> 16);
      }
    }
  }
}

}  // namespace
}  // namespace kvimpl

// ---------------------------------------------------------------------------
// C ABI
// ---------------------------------------------------------------------------

using namespace kvimpl;

extern "C" kv_status kv_store_rope(const void* k, const void* v, void* k_cache, void* v_cache,
                                   const void* indices, kv_index_dtype index_dtype,
                                   int64_t index_stride, int64_t num_tokens, int32_t num_heads,
                                   int32_t head_dim, kv_src_dtype src_dtype, const kv_strides* s,
                                   int64_t page_size, int64_t kc_page_stride,
                                   int64_t vc_page_stride, int64_t size_limit, const kv_rope* rope,
                                   kv_cache_format format, const float* inv_k_scale,
                                   const float* inv_v_scale, const kv_block_scales* scales,
                                   kv_error_record* d_err, kv_stream_t stream_) {
  if (num_tokens < 0) return KV_ERR_INVALID_ARG;
  if (format != KV_CACHE_SRC && format != KV_CACHE_E4M3FN && format != KV_CACHE_E2M1)
    return KV_ERR_INVALID_ARG;
  if (num_tokens == 0) return KV_OK;
  if (!common_args_ok(k, v, k_cache, v_cache, indices, index_dtype, index_stride, num_heads,
                      head_dim, s, size_limit, d_err) || !rope)
    return KV_ERR_INVALID_ARG;
  if (src_dtype != KV_SRC_F16 && src_dtype != KV_SRC_BF16) return KV_ERR_INVALID_ARG;
  if (page_size < 1) return KV_ERR_INVALID_ARG;
  const kv_rope& rp = *rope;
  if ((!rp.cos_sin && rp.rotary_dim > 0) || !rp.positions || rp.position_stride < 1 || rp.max_position < 0 ||
      (rp.position_dtype != KV_INDEX_I32 && rp.position_dtype != KV_INDEX_I64) ||
      rp.rotary_dim < 0 || rp.rotary_dim > head_dim || (rp.rotary_dim & 1) != 0 ||
      rp.cos_sin_stride < rp.rotary_dim || (u64(rp.cos_sin) & 3u) != 0)
    return KV_ERR_INVALID_ARG;
  if (rp.q && (!rp.q_out || rp.num_q_heads < 1)) return KV_ERR_INVALID_ARG;
  if ((u64(indices) & (index_dtype == KV_INDEX_I64 ? 7u : 3u)) != 0 ||
      (u64(rp.positions) & (rp.position_dtype == KV_INDEX_I64 ? 7u : 3u)) != 0)
    return KV_ERR_INVALID_ARG;
  uint64_t even = u64(k) | u64(v) | u64(s->k_token) | u64(s->k_head) | u64(s->k_dim) |
                  u64(s->v_token) | u64(s->v_head) | u64(s->v_dim);
  if (rp.q)
    even |= u64(rp.q) | u64(rp.q_out) | u64(rp.q_token) | u64(rp.q_head) | u64(rp.qo_token) |
            u64(rp.qo_head);
  if (format == KV_CACHE_SRC)
    even |= u64(k_cache) | u64(v_cache) | u64(s->kc_slot) | u64(s->kc_head) | u64(s->kc_dim) |
            u64(s->vc_slot) | u64(s->vc_head) | u64(s->vc_dim) | u64(kc_page_stride) |
            u64(vc_page_stride);
  if ((even & 1u) != 0) return KV_ERR_INVALID_ARG;
  if (((u64(inv_k_scale) | u64(inv_v_scale)) & 3u) != 0) return KV_ERR_INVALID_ARG;
  if (format == KV_CACHE_E2M1) {
    if (!scales || !scales->k || !scales->v) return KV_ERR_INVALID_ARG;
    if (head_dim % kFp4Block != 0 || s->kc_dim != 1 || s->vc_dim != 1) return KV_ERR_UNSUPPORTED;
  }
  if (num_tokens > (int64_t{1} << 40)) return KV_ERR_UNSUPPORTED;
  {
    const void* in[14] = {k, v, indices, rp.positions, k_cache, v_cache, d_err};
    int n = 7;
    if (rp.q) {
      in[n++] = rp.q;
      in[n++] = rp.q_out;
    }
    if (rp.rotary_dim > 0) in[n++] = rp.cos_sin;
    if (format == KV_CACHE_E2M1) {
      in[n++] = scales->k;
      in[n++] = scales->v;
    }
    if (format != KV_CACHE_SRC && inv_k_scale) in[n++] = inv_k_scale;
    if (format != KV_CACHE_SRC && inv_v_scale) in[n++] = inv_v_scale;
    bool on_device = true;
    const kv_status cs = classify_inputs(in, n, &on_device);
    if (cs != KV_OK) return cs;
  }

  RopeParams p = {};
  if (rp.q) {
    p.side[0] = RopeSide{static_cast<const uint8_t*>(rp.q), static_cast<uint8_t*>(rp.q_out),
                         rp.q_token, rp.q_head, 2, 0, rp.qo_token, rp.qo_head, 2,
                         nullptr, nullptr, 0, 0, 0};
    p.q_heads = static_cast<uint32_t>(rp.num_q_heads);
  }
  const bool scaled = format != KV_CACHE_SRC;
  p.side[1] = RopeSide{static_cast<const uint8_t*>(k), static_cast<uint8_t*>(k_cache), s->k_token,
                       s->k_head, s->k_dim, kc_page_stride, s->kc_slot, s->kc_head, s->kc_dim,
                       scaled ? inv_k_scale : nullptr, nullptr, 0, 0, 0};
  p.side[2] = RopeSide{static_cast<const uint8_t*>(v), static_cast<uint8_t*>(v_cache), s->v_token,
                       s->v_head, s->v_dim, vc_page_stride, s->vc_slot, s->vc_head, s->vc_dim,
                       scaled ? inv_v_scale : nullptr, nullptr, 0, 0, 0};
  if (format == KV_CACHE_E2M1) {
    p.side[1].scales = static_cast<uint8_t*>(scales->k);
    p.side[1].sc_page = scales->k_page;
    p.side[1].sc_slot = scales->k_slot;
    p.side[1].sc_head = scales->k_head;
    p.side[2].scales = static_cast<uint8_t*>(scales->v);
    p.side[2].sc_page = scales->v_page;
    p.side[2].sc_slot = scales->v_slot;
    p.side[2].sc_head = scales->v_head;
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
  p.kv_heads = static_cast<uint32_t>(num_heads);
  p.per_token = p.q_heads + 2u * p.kv_heads;
  p.num_units = static_cast<uint64_t>(num_tokens) * p.per_token;
  p.head_dim = static_cast<uint32_t>(head_dim);
  p.rotary = static_cast<uint32_t>(rp.rotary_dim);
  p.pos64 = rp.position_dtype == KV_INDEX_I64;
  p.idx64 = index_dtype == KV_INDEX_I64;
  p.bf16 = src_dtype == KV_SRC_BF16;
  p.interleaved = rp.interleaved != 0;
  p.err = d_err;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);

  // kv_rope_rows: whole items of 16 dims, 16-byte pieces on the 16-bit sides, what an item writes to
  // a cache aligned to its size, and e2m1 blocks that do not straddle the halves of the rotation
  const int32_t R = rp.rotary_dim;
  uint64_t in_bits = u64(k) | u64(v) | u64(s->k_token) | u64(s->k_head) | u64(s->v_token) | u64(s->v_head);
  if (rp.q) in_bits |= u64(rp.q) | u64(rp.q_out) | u64(rp.q_token) | u64(rp.q_head) | u64(rp.qo_token) | u64(rp.qo_head);
  if (R > 0) in_bits |= u64(rp.cos_sin) | u64(4 * rp.cos_sin_stride);
  const uint64_t cache_bits = u64(k_cache) | u64(v_cache) | u64(s->kc_slot) | u64(s->kc_head) | u64(s->vc_slot) |
                              u64(s->vc_head) | u64(kc_page_stride) | u64(vc_page_stride);
  const int32_t elem = format == KV_CACHE_SRC ? 2 : 1;
  const bool rows = head_dim % 16 == 0 && head_dim <= 512 && R % 16 == 0 && (in_bits & 15u) == 0 &&
                    (cache_bits & (format == KV_CACHE_E2M1 ? 7u : 15u)) == 0 && s->k_dim == 2 && s->v_dim == 2 &&
                    s->kc_dim == elem && s->vc_dim == elem &&
                    (format != KV_CACHE_E2M1 || p.interleaved || (R % 32 == 0 && head_dim % 32 == 0));
  if (rows) {
    RopeRowParams q = {};
    q.r = p;
    q.iph = static_cast<uint32_t>(head_dim / 16);
    q.hpp = 32u / q.iph;
    q.heads = p.per_token;
    q.narrow = size_limit <= INT32_MAX && page_size <= INT32_MAX;
    switch (format) {
      case KV_CACHE_SRC:
        return p.interleaved ? launch_rope_rows<KV_CACHE_SRC, true>(q, num_tokens, stream)
                             : launch_rope_rows<KV_CACHE_SRC, false>(q, num_tokens, stream);
      case KV_CACHE_E4M3FN:
        return p.interleaved ? launch_rope_rows<KV_CACHE_E4M3FN, true>(q, num_tokens, stream)
                             : launch_rope_rows<KV_CACHE_E4M3FN, false>(q, num_tokens, stream);
      default:
        return p.interleaved ? launch_rope_rows<KV_CACHE_E2M1, true>(q, num_tokens, stream)
                             : launch_rope_rows<KV_CACHE_E2M1, false>(q, num_tokens, stream);
    }
  }
  switch (format) {
    case KV_CACHE_SRC: return launch(kv_rope_any<KV_CACHE_SRC>, p.num_units, p, stream);
    case KV_CACHE_E4M3FN: return launch(kv_rope_any<KV_CACHE_E4M3FN>, p.num_units, p, stream);
    default: return launch(kv_rope_any<KV_CACHE_E2M1>, p.num_units, p, stream);
  }
}

extern "C" kv_status kv_gather_fp4(const void* k_cache, const void* v_cache,
                                   const kv_block_scales* scales, void* k_out, void* v_out,
                                   const void* indices, kv_index_dtype index_dtype,
                                   int64_t index_stride, int64_t num_tokens, int32_t num_heads,
                                   int32_t head_dim, kv_src_dtype out_dtype, const kv_strides* s,
                                   int64_t page_size, int64_t kc_page_stride,
                                   int64_t vc_page_stride, int64_t size_limit,
                                   const float* k_scale, const float* v_scale,
                                   kv_error_record* d_err, kv_stream_t stream_) {
  if (num_tokens < 0) return KV_ERR_INVALID_ARG;
  if (num_tokens == 0) return KV_OK;
  if (!common_args_ok(k_out, v_out, k_cache, v_cache, indices, index_dtype, index_stride, num_heads,
                      head_dim, s, size_limit, d_err) || !scales || !scales->k || !scales->v)
    return KV_ERR_INVALID_ARG;
  if (out_dtype != KV_SRC_F16 && out_dtype != KV_SRC_BF16) return KV_ERR_INVALID_ARG;
  if (page_size < 1 || ((u64(k_scale) | u64(v_scale)) & 3u) != 0) return KV_ERR_INVALID_ARG;
  if ((u64(indices) & (index_dtype == KV_INDEX_I64 ? 7u : 3u)) != 0) return KV_ERR_INVALID_ARG;
  const uint64_t out_bits = u64(k_out) | u64(v_out) | u64(s->k_token) | u64(s->v_token) |
                            u64(s->k_head) | u64(s->v_head);
  if ((out_bits & 1u) != 0) return KV_ERR_INVALID_ARG;
  if (head_dim % kFp4Block != 0 || s->k_dim != 2 || s->v_dim != 2) return KV_ERR_UNSUPPORTED;
  const uint64_t per_token = 2ull * static_cast<uint64_t>(num_heads) * static_cast<uint64_t>(head_dim / kFp4Block);
  if (num_tokens > (int64_t{1} << 40) || per_token >= (1ull << 31)) return KV_ERR_UNSUPPORTED;
  {
    const void* in[10] = {k_out, v_out, indices, k_cache, v_cache, scales->k, scales->v, d_err};
    int n = 8;
    if (k_scale) in[n++] = k_scale;
    if (v_scale) in[n++] = v_scale;
    bool on_device = true;
    const kv_status cs = classify_inputs(in, n, &on_device);
    if (cs != KV_OK) return cs;
  }
  Fp4GatherParams p = {};
  p.side[0] = Fp4Side{static_cast<const uint8_t*>(k_cache), static_cast<const uint8_t*>(scales->k),
                      static_cast<uint8_t*>(k_out), kc_page_stride, s->kc_slot, s->kc_head,
                      scales->k_page, scales->k_slot, scales->k_head, s->k_token, s->k_head, k_scale};
  p.side[1] = Fp4Side{static_cast<const uint8_t*>(v_cache), static_cast<const uint8_t*>(scales->v),
                      static_cast<uint8_t*>(v_out), vc_page_stride, s->vc_slot, s->vc_head,
                      scales->v_page, scales->v_slot, scales->v_head, s->v_token, s->v_head, v_scale};
  p.indices = indices;
  p.index_stride = index_stride;
  p.size_limit = size_limit;
  p.page_size = page_size;
  p.heads = static_cast<uint32_t>(num_heads);
  p.blocks = static_cast<uint32_t>(head_dim / kFp4Block);
  p.num_items = static_cast<uint64_t>(num_tokens) * per_token;
  p.idx64 = index_dtype == KV_INDEX_I64;
  p.bf16 = out_dtype == KV_SRC_BF16;
  const uint64_t code_bits = u64(k_cache) | u64(v_cache) | u64(kc_page_stride) | u64(vc_page_stride) |
                             u64(s->kc_slot) | u64(s->kc_head) | u64(s->vc_slot) | u64(s->vc_head);
  p.wide = (code_bits & 7u) == 0 && (out_bits & 15u) == 0;
  p.err = d_err;
  return launch(kv_gather_fp4_blocks, (p.num_items + 31u) / 32u, p,
                reinterpret_cast<cudaStream_t>(stream_));
}
