// Attention for few query rows per sequence (decode, speculative steps): the
// key axis is split over the GPU and the parts are joined.
//
// Bytes bound it: every visible K and V row is read once per KV head and meets
// the few query rows of that head's group.  So
//  * a warp takes one KV head and tiles of TW keys.  cp.async brings a tile's K
//    and V rows from their pages into a ring of NU units of the warp's own
//    shared memory, two or three units in flight at any time; keys behind the
//    list's end and head dims behind D are zero-filled, not read.  The warps
//    of a CTA take the heads of the same keys (their rows lie together) and,
//    with fewer than eight heads, neighbouring tiles.
//  * a lane copies exactly the 16-byte pieces that it will multiply, so it
//    reads its own shared memory back, in order and without conflicts:
//    S^T = K Q^T has the tile's keys as the 16 rows of mma.m16n8k16, and lane
//    (g, t) needs row g's dims in any order that Q's registers share;
//    O^T = V^T P^T has dims as rows, and lane (g, t) needs tokens 2t, 2t+1,
//    2t+8, 2t+9 of any dims that it writes out in the end.  P^T leaves S^T's
//    accumulators by movmatrix, and the running maximum, sum and O share one
//    mapping of query rows to lanes, so no statistic crosses a lane but the
//    maximum (three shuffles per tile and two rows) and, once, the sum.
//  * quantised elements become fp16 in registers, exactly: e4m3 and e2m1 codes
//    by the hardware's conversions, e2m1 blocks times their e4m3 scale (at
//    most 6 significant bits).  The pair of tokens that V^T wants in one
//    register is interleaved byte- or nibble-wise before the conversion.
//    Queries in bf16 are brought to fp16 by a power of two per row that puts
//    the row's largest element at 2^13 .. 2^14 (elements 2^-38 of it and
//    smaller lose bits).  The tensor scale and the power go into the softmax's
//    scale.
//  * weights multiply 16-bit caches as two 16-bit terms (p = hi + lo), so their
//    rounding does not add to the output's; the mma pipe has room for the
//    second product there.  For quantised caches they are fp16 (2^-12 of each).
//    fp16 weights begin at 2^15 instead of 1, so that they keep their bits down to 2^-29
//    of the largest and end at 2^-40, not at 2^-14 and 2^-25: many small ones add up.
//  * all (sequence, block of rows, head group, tile) steps, counted by a scan
//    over the lengths on the device, are cut into contiguous shares: one of
//    80 % of an equal part for each CTA, the rest in shares of half the size and
//    half again that CTAs take as they become free.  Ragged batches are
//    balanced without the host knowing a length, and so are the SMs, whose
//    share of the memory's bandwidth differs by a third (with equal shares the
//    first SMs ended a 400 us call at 290 us).  A share that begins or ends
//    inside an item leaves its sums in the workspace, and a second kernel joins
//    them in the order of the keys, whoever computed them.
//    Two launches and their scans are what a short call costs: one query over
//    1,000 16-bit keys, 32 over 8 heads of 128, 16 us; 16 sequences of 40 - 130
//    tokens, unsplit, 11 us; 48 windows of 4,096 in pages of 20 keys, 781 MB, 160 us, 4.9 TB/s.
//  * a row whose sum is 0 or whose output is not finite is done again by
//    attend_row, which touches its visible keys alone: a NaN value that the
//    mask hides from a row must not reach it through a weight of 0.
#pragma once

#include <atomic>

#include "kv_async.cuh"
#include "kv_attend.cuh"
#include "kv_host.h"

namespace kvimpl {

constexpr int kFirstShares = 80;  // percent of the steps in the CTAs' first shares
// Steps of a share at least; kLastSteps where a CTA has eight times as many to do: each share of
// an item is a part to be written and joined (windows of 4,096 in 128 sequences: 317 us at 12
// steps, 332 at 4; one sequence of 1,000 keys, one share a CTA: 26 us at 16, 17.5 at 4).
constexpr int kMinSteps = 4, kLastSteps = 12;

// The shares: level k holds shares of `size` steps from step `start` on, numbered from `first`.
struct ShareLevel {
  int64_t start;
  int32_t size, first;
};
constexpr int kLevels = 6;

// The workspace's head: zero between calls that complete.
struct SplitWork {
  unsigned int next;     // the shares that CTAs have taken beyond their first
  unsigned int gave_up;  // a CTA left before its shares were done (not reset here)
  unsigned int pad[62];
  ShareLevel level[kLevels];
  int32_t levels, shares;  // in use
};
constexpr int64_t kSplitHead = 512;
static_assert(sizeof(SplitWork) <= kSplitHead, "the workspace's head");

struct SplitParams {
  AttendParams a;
  int32_t hw, subs;       // KV heads per CTA; warps per head
  int32_t hgroups;        // kv_heads / hw
  int32_t rows;           // query rows per item
  int32_t whole_blocks;   // page_size is a multiple of 16: 16 aligned keys share a page
  int32_t k_page, k_slot, v_page, v_slot;      // byte strides, in 32 bits
  int32_t ks_page, ks_slot, vs_page, vs_slot;  // of the block scales
  int32_t split;          // 0: an item is one CTA's
  int32_t min_steps;      // a share is at least this long
  int32_t max_shares;     // that the workspace has room for
  int32_t part_rows;      // rows of an item that can be there
  SplitWork* head;
  int64_t* meta;          // [num_seqs]: first step of each sequence
  float *part_o, *part_ml;  // [2 * max_shares][hw][part_rows] x DP and x 2
};

// Cuts `total` steps into shares for `ctas` CTAs.
__device__ __forceinline__ void cut_shares(int64_t total, int32_t ctas, int32_t max_shares, int32_t min_steps,
                                           SplitWork* w) {
  int64_t each = (total + ctas - 1) / ctas;
  if (each < min_steps) each = min_steps;
  min_steps = static_cast<int32_t>(max(static_cast<int64_t>(min_steps), min(each / 8, static_cast<int64_t>(kLastSteps))));
  int32_t n = 0, made = 0;
  int64_t at = 0, size = each;
  if (each >= 4 * min_steps && max_shares >= 3 * ctas) {
    size = each * kFirstShares / 100;
    while (n < kLevels - 1) {
      w->level[n++] = ShareLevel{at, static_cast<int32_t>(size), made};
      at += size * ctas;
      made += ctas;
      size = (total - at) / (2 * ctas);
      if (size < 2 * min_steps || max_shares - made < 3 * ctas) break;
    }
    const int64_t room = max_shares - made;
    size = (total - at + room - 1) / room;
    if (size < min_steps) size = min_steps;
  }
  w->level[n++] = ShareLevel{at, static_cast<int32_t>(size), made};
  w->levels = n;
  w->shares = made + static_cast<int32_t>((total - at + size - 1) / size);
}

__device__ __forceinline__ int32_t share_of(const SplitWork* w, int64_t step) {
  int32_t k = w->levels - 1;
  while (k > 0 && w->level[k].start > step) --k;
  return w->level[k].first + static_cast<int32_t>((step - w->level[k].start) / w->level[k].size);
}

// An item is (sequence, block of query rows, head group); its steps are the
// tiles of TW keys, aligned to TW, that hold a key some row of it sees, `subs`
// at a time.  The step count is the same for all items of a sequence: an upper
// bound over its blocks, and at least one, so that rows without keys are
// written too.
struct SplitGeom {
  int32_t blocks, steps;
};

template <int TW>
__device__ __forceinline__ SplitGeom split_geom(const SplitParams& p, const AttendSeq& s) {
  SplitGeom r;
  const uint32_t rows = static_cast<uint32_t>(s.nq) * p.a.group.d;
  r.blocks = static_cast<int32_t>((rows + p.rows - 1) / static_cast<uint32_t>(p.rows));
  int32_t tiles = (s.len + TW - 1) / TW;
  if (p.a.window > 0 && p.a.window < s.len) {
    // a block of rows spans at most `span` positions, and its windows window + span - 1 keys
    const int32_t span = min(s.nq, (p.rows - 1) / static_cast<int32_t>(p.a.group.d) + 2);
    const int32_t sinks = (min(p.a.sinks, s.len) + TW - 1) / TW;
    tiles = min(tiles, sinks + (p.a.window + span + TW - 3) / TW + 1);
  }
  r.steps = max((tiles + p.subs - 1) / p.subs, 1);
  return r;
}

// The tiles of a block of rows at positions p_lo .. p_hi: the first `sinks`
// tiles, then lo, lo + 1, ...; n in all.
struct TileList {
  int32_t sinks, lo, n;
  int32_t lo_key;  // first key of the windows
  __device__ __forceinline__ int32_t tile(int32_t i) const { return i < sinks ? i : lo + (i - sinks); }
};

template <int TW>
__device__ __forceinline__ TileList visible_tiles(const AttendParams& p, int32_t p_lo, int32_t p_hi) {
  const KeyList k = visible_keys(p, p_lo, p_hi);
  TileList r;
  r.lo_key = k.lo;
  r.lo = k.lo / TW;
  r.sinks = min((k.sinks + TW - 1) / TW, r.lo);
  r.n = p_hi < 0 ? 0 : r.sinks + p_hi / TW - r.lo + 1;
  return r;
}

template <int TW>
__device__ __forceinline__ int64_t seq_units(const SplitParams& p, int32_t b, bool record) {
  const SplitGeom g = split_geom<TW>(p, attend_seq(p.a, b, record));
  return static_cast<int64_t>(g.blocks) * p.hgroups * (p.split ? g.steps : 1);
}

// ---------------------------------------------------------------------------
// Formats: what a lane copies and how it becomes operands.
// ---------------------------------------------------------------------------

template <int FMT, int DP>
struct Layout {
  static constexpr int kBits = FMT == KV_CACHE_SRC ? 16 : FMT == KV_CACHE_E4M3FN ? 8 : 4;
  static constexpr int kRow = DP * kBits / 8;                     // bytes of a padded row
  static constexpr int KC = kRow / 4 < 16 ? kRow / 4 : 16;        // K: bytes a lane copies at once (4 lanes a row)
  static constexpr int KN = kRow / 4 / KC;                        //    and how often
  static constexpr int VC = kRow / 8 < 16 ? kRow / 8 : 16;        // V: 8 lanes a row
  static constexpr int VN = kRow / 8 / VC;
  static constexpr int KD = KC * 8 / kBits;                       // dims of a K piece
  static constexpr int VD = VC * 8 / kBits;
  static constexpr int TW = (FMT == KV_CACHE_SRC && DP >= 128) ? 16 : 32;  // keys of a warp's tile
  static constexpr int MB = TW / 16;
  // e2m1: room for a row's scales: the words around them and a word for where in them they begin;
  // 16 or 24 bytes spread eight rows over the banks
  static constexpr int kScaleRow = FMT == KV_CACHE_E2M1 ? (DP <= 128 ? 16 : 24) : 0;
  static constexpr int kUnit = TW * (kRow + kScaleRow);
};

// A byte offset in 64 bits from 32-bit factors.
__device__ __forceinline__ int64_t wide(int32_t n, int32_t stride) { return static_cast<int64_t>(n) * stride; }
__device__ __forceinline__ int64_t wide(uint32_t n, int32_t stride) { return wide(static_cast<int32_t>(n), stride); }

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const uint8_t* src, uint32_t bytes) {
  if constexpr (BYTES == 16) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
  } else {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(bytes), "n"(BYTES) : "memory");
  }
}

__device__ __forceinline__ void commit_async() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void wait_async() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <int BYTES>
__device__ __forceinline__ void ld_own(uint32_t (&w)[BYTES / 4], uint32_t addr) {
  if constexpr (BYTES == 16) {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr) : "memory");
  } else if constexpr (BYTES == 8) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr) : "memory");
  } else {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(addr) : "memory");
  }
}

__device__ __forceinline__ uint32_t ld_shared_u8(uint32_t addr) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(addr) : "memory");
  return r;
}

__device__ __forceinline__ uint32_t ld_shared_u16(uint32_t addr) {
  uint16_t r;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(addr) : "memory");
  return r;
}

__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(addr) : "memory");
  return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}

template <bool kBF16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if constexpr (kBF16) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  } else {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
}

// Pieces are converted a word at a time, so that few operands are live.  A word holds kWord dims.
template <int FMT>
constexpr int kWord = FMT == KV_CACHE_SRC ? 2 : FMT == KV_CACHE_E4M3FN ? 4 : 8;

// A K word as kWord / 2 packed pairs.  s2: its block's scale in both halves (e2m1).
template <int FMT>
__device__ __forceinline__ void k_word(uint32_t (&f)[kWord<FMT> / 2], uint32_t w, uint32_t s2) {
  if constexpr (FMT == KV_CACHE_SRC) {
    f[0] = w;
  } else if constexpr (FMT == KV_CACHE_E4M3FN) {
    f[0] = f16x2_from_e4m3x2(w);
    f[1] = f16x2_from_e4m3x2(w >> 16);
  } else {
    f16x2_from_e2m1x8(w, f);
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = mul_f16x2(f[j], s2);
  }
}

// A V word of tokens a and b as kWord words (a, b).  s2: the tokens' block scales (e2m1).
template <int FMT>
__device__ __forceinline__ void v_word(uint32_t (&f)[kWord<FMT>], uint32_t a, uint32_t b, uint32_t s2) {
  if constexpr (FMT == KV_CACHE_SRC) {
    f[0] = __byte_perm(a, b, 0x5410);
    f[1] = __byte_perm(a, b, 0x7632);
  } else if constexpr (FMT == KV_CACHE_E4M3FN) {
    const uint32_t lo = __byte_perm(a, b, 0x5140), hi = __byte_perm(a, b, 0x7362);
    f[0] = f16x2_from_e4m3x2(lo);
    f[1] = f16x2_from_e4m3x2(lo >> 16);
    f[2] = f16x2_from_e4m3x2(hi);
    f[3] = f16x2_from_e4m3x2(hi >> 16);
  } else {
    const uint32_t even = (a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u);
    const uint32_t odd = ((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u);
    uint32_t e[4], o[4];
    f16x2_from_e2m1x8(even, e);
    f16x2_from_e2m1x8(odd, o);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = mul_f16x2(e[j], s2);
      f[2 * j + 1] = mul_f16x2(o[j], s2);
    }
  }
}

// S^T += K Q^T for one piece of rows g (w[..][0]) and g + 8 (w[..][1]) of each 16 keys: KD / 4 products
// a block of queries, whose pairs for it begin at qf[..][first].  sc: the rows' block scale codes
// (e2m1).  The 16s take turns: a product waits for the one before it in the same sums.
template <int FMT, int DP, int NB, bool kBF16, int MB>
__device__ __forceinline__ void k_products(float (&s)[MB][NB][4], const uint32_t (&w)[MB][2][Layout<FMT, DP>::KC / 4],
                                           const uint32_t (&sc)[MB][2], const uint32_t (&qf)[NB][DP / 8], int first) {
  constexpr int kWords = Layout<FMT, DP>::KC / 4;
  if constexpr (FMT == KV_CACHE_SRC) {
#pragma unroll
    for (int i = 0; i < kWords; i += 2)
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
          mma16816<kBF16>(s[mb][nb], w[mb][0][i], w[mb][1][i], w[mb][0][i + 1], w[mb][1][i + 1], qf[nb][first + i], qf[nb][first + i + 1]);
  } else {
    uint32_t two[MB][2];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int rh = 0; rh < 2; ++rh) two[mb][rh] = FMT == KV_CACHE_E2M1 ? f16x2_from_e4m3x2(sc[mb][rh]) : 0u;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      uint32_t f[MB][2][kWord<FMT> / 2];
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int rh = 0; rh < 2; ++rh)
          k_word<FMT>(f[mb][rh], w[mb][rh][i], __byte_perm(two[mb][rh], 0u, i * 8 / kFp4Block == 0 ? 0x1010 : 0x3232));
#pragma unroll
      for (int j = 0; j < kWord<FMT> / 2; j += 2)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
            mma16816<kBF16>(s[mb][nb], f[mb][0][j], f[mb][1][j], f[mb][0][j + 1], f[mb][1][j + 1],
                            qf[nb][first + i * (kWord<FMT> / 2) + j], qf[nb][first + i * (kWord<FMT> / 2) + j + 1]);
    }
  }
}

// O^T += V^T P^T for one piece of tokens 2t, 2t + 1 (w[0], w[1]), 2t + 8, 2t + 9 (w[2], w[3]): VD / 2
// products a block of queries, from o[..][first] on.  sc: the scale codes of the first and of the
// second two tokens, a byte each, per block of the piece (e2m1).
template <int FMT, int DP, int NB, bool kBF16, int OM>
__device__ __forceinline__ void v_products(float (&o)[NB][OM][4], const uint32_t (&w)[4][Layout<FMT, DP>::VC / 4],
                                           const uint32_t (&sc)[2][2], const uint32_t (&pt)[NB][2], const uint32_t (&pl)[NB][2], int first) {
  constexpr int kWords = Layout<FMT, DP>::VC / 4;
#pragma unroll
  for (int i = 0; i < kWords; ++i) {
    uint32_t f[2][kWord<FMT>];
#pragma unroll
    for (int pr = 0; pr < 2; ++pr)
      v_word<FMT>(f[pr], w[2 * pr][i], w[2 * pr + 1][i], FMT == KV_CACHE_E2M1 ? f16x2_from_e4m3x2(sc[pr][i * 8 / kFp4Block]) : 0u);
#pragma unroll
    for (int j = 0; j < kWord<FMT> / 2; ++j)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float (&acc)[4] = o[nb][first + i * (kWord<FMT> / 2) + j];
        mma16816<kBF16>(acc, f[0][2 * j], f[0][2 * j + 1], f[1][2 * j], f[1][2 * j + 1], pt[nb][0], pt[nb][1]);
        if constexpr (FMT == KV_CACHE_SRC)
          mma16816<kBF16>(acc, f[0][2 * j], f[0][2 * j + 1], f[1][2 * j], f[1][2 * j + 1], pl[nb][0], pl[nb][1]);
      }
  }
}

// ---------------------------------------------------------------------------
// A warp's share of the work on one block of query rows: lane (g, t) is lane 4 g + t.
// ---------------------------------------------------------------------------

// The queries as the products' second operand: lane (g, t) holds row g of each eight; pair i of it
// are dims dim_of(i), dim_of(i) + 1 (four pairs at a time are eight dims in a row).  rs: the
// softmax scale (log2) of rows 2t, 2t + 1.
template <int FMT, int DP, int NB, typename DimOf>
__device__ __forceinline__ void load_queries(const AttendParams& a, const AttendSeq& seq, int32_t kvh, int32_t row0, int32_t nrows,
                                             float kscale, DimOf dim_of, uint32_t (&qf)[NB][DP / 8], float (&rs)[NB][2]) {
  constexpr int QP = DP / 8;
  const uint32_t lane = threadIdx.x & 31u, g = lane >> 2, t = lane & 3u;
  const int32_t G = static_cast<int32_t>(a.group.d);
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int32_t r = nb * 8 + static_cast<int32_t>(g);
    const bool ok = r < nrows;
    const uint32_t qi = a.group.quot(static_cast<uint32_t>(row0 + (ok ? r : 0)));
    const int32_t h = kvh * G + (row0 + (ok ? r : 0) - static_cast<int32_t>(qi) * G);
    const uint8_t* src = a.q + (static_cast<int64_t>(seq.q0) + qi) * a.q_token + h * a.q_head;
#pragma unroll
    for (int i = 0; i < QP; i += 4) {
      const int d = dim_of(i);
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (ok && d < a.head_dim) w = __ldg(reinterpret_cast<const uint4*>(src + 2 * d));
      qf[nb][i] = w.x; qf[nb][i + 1] = w.y; qf[nb][i + 2] = w.z; qf[nb][i + 3] = w.w;
    }
    float inv = 1.0f;
    if constexpr (FMT != KV_CACHE_SRC) {
      if (a.bf16) {
        uint32_t amax = 0u;
#pragma unroll
        for (int i = 0; i < QP; ++i) amax = absmax_pair<true>(amax, qf[nb][i]);
        uint32_t m = __float_as_uint(absmax_pair_value<true>(amax));
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        const uint32_t e = m >> 23;  // 2^(140 - e): the largest element to 2^13 .. 2^14
        const float f = __uint_as_float(min(254u, 267u - e) << 23);
        inv = __fdiv_rn(1.0f, f);
#pragma unroll
        for (int i = 0; i < QP; ++i) {
          const float2 x = widen2<true>(qf[nb][i]);
          qf[nb][i] = pack2(x.x * f, x.y * f, false);
        }
      }
    }
    if (kscale < 0.0f) {  // the running maximum is taken before the scale
#pragma unroll
      for (int i = 0; i < QP; ++i) qf[nb][i] ^= 0x80008000u;
    }
    float full = fabsf(kscale) * inv;
    if (full == 0.0f) full = __uint_as_float(1u);  // a scale of 0: hidden scores (-inf) must stay -inf
    rs[nb][0] = __shfl_sync(0xFFFFFFFFu, full, 8u * t);
    rs[nb][1] = __shfl_sync(0xFFFFFFFFu, full, 8u * t + 4u);
  }
}

// Scores s[..][0], [1] are those of key `key` of each 16 and rows 2t, 2t + 1, [2], [3] of key + 8.
// Those of keys (from j0 on, up to key_hi) that their row does not see become -inf; pages: some
// page id was out of range, so look each key's up.
template <int NB, int MB>
__device__ __forceinline__ void hide_scores(const AttendParams& a, const int32_t* table, int32_t j0, int32_t key_hi, bool pages,
                                            int32_t p_first, int32_t row0, uint32_t key, float (&s)[MB][NB][4]) {
  const uint32_t t = threadIdx.x & 3u;
  int32_t pos_of[NB][2];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int c = 0; c < 2; ++c)
      pos_of[nb][c] = p_first + static_cast<int32_t>(a.group.quot(static_cast<uint32_t>(row0 + nb * 8 + 2 * t + c)));
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int rh = 0; rh < 2; ++rh) {
      const int32_t j = j0 + mb * 16 + rh * 8 + static_cast<int32_t>(key);
      bool have = j <= key_hi;
      if (have && pages) {
        const int32_t id = __ldg(table + a.page.quot(static_cast<uint32_t>(j)));
        have = id >= 0 && id < a.num_pages;
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          if (!have || !sees(a, pos_of[nb][c], j)) s[mb][nb][rh * 2 + c] = -INFINITY;
    }
}

// The running maximum is kept less this power, so the largest weight is 2 to it.
template <bool kBF16>
constexpr float kRoom = kBF16 ? 0.0f : 15.0f;

// Running maximum (less kRoom) and sum of rows 2t, 2t + 1; the weights, transposed to the second operand of
// O^T = V^T P^T (pt; pl: what their rounding left, 16-bit caches).
template <int FMT, int NB, int MB, int OM, bool kBF16>
__device__ __forceinline__ void softmax_step(float (&s)[MB][NB][4], const float (&rs)[NB][2], float (&m)[NB][2], float (&l)[NB][2],
                                             float (&o)[NB][OM][4], uint32_t (&pt)[MB][NB][2], uint32_t (&pl)[MB][NB][2]) {
  bool grew = false;
  float alpha[NB][2];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float x = s[0][nb][c];
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) x = fmaxf(x, fmaxf(s[mb][nb][c], s[mb][nb][2 + c]));
      x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
      x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
      x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
      x = fmaxf(m[nb][c], __fmaf_rn(x, rs[nb][c], -kRoom<kBF16>));
      const float ref = x == -INFINITY ? 0.0f : x;
      grew |= x > m[nb][c];
      alpha[nb][c] = exp2_fast(m[nb][c] - ref);
      m[nb][c] = x;
      float sum = 0.0f;
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int rh = 0; rh < 2; ++rh) {
          float& e = s[mb][nb][2 * rh + c];
          e = exp2_fast(__fmaf_rn(e, rs[nb][c], -ref));
          sum += e;
        }
      l[nb][c] = __fmaf_rn(l[nb][c], alpha[nb][c], sum);
    }
  // (e2m1: without the branch the compiler mixes this with the next products' loads and conversions)
  if (FMT == KV_CACHE_E2M1 || __any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < OM; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[nb][i][c] *= alpha[nb][c & 1];
  }
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int rh = 0; rh < 2; ++rh) {
        const float x = s[mb][nb][2 * rh], y = s[mb][nb][2 * rh + 1];
        const uint32_t w = pack2(x, y, kBF16);
        pt[mb][nb][rh] = transpose8x8(w);
        if constexpr (FMT == KV_CACHE_SRC) {
          const float2 r = widen2<kBF16>(w);
          pl[mb][nb][rh] = transpose8x8(pack2(x - r.x, y - r.y, kBF16));
        }
      }
}

// Dim of the lane's i-th O^T product (rows g are even dims of its pieces, rows g + 8 the odd ones).
template <int FMT, int DP>
__device__ __forceinline__ int out_dim(int i) {
  using L = Layout<FMT, DP>;
  return (static_cast<int>((threadIdx.x & 31u) >> 2) + 8 * (2 * i / L::VD)) * L::VD + 2 * i % L::VD;
}

// The rows of an item that one warp has whole.
template <int FMT, int DP, int NB, int OM>
__device__ __forceinline__ void write_rows(const AttendParams& a, int32_t b, const AttendSeq& seq, int32_t kvh, int32_t row0, int32_t nrows,
                                           float vscale, const float (&o)[NB][OM][4], const float (&m)[NB][2], const float (&l)[NB][2],
                                           WaitState* waits = nullptr) {
  const uint32_t lane = threadIdx.x & 31u, g = lane >> 2, t = lane & 3u;
  const int32_t G = static_cast<int32_t>(a.group.d);
  uint32_t again = 0u;  // rows to be done once more, a bit each
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int32_t r = nb * 8 + 2 * static_cast<int32_t>(t) + c;
      if (r < nrows) {
        const float inv = __fdiv_rn(vscale, l[nb][c]);
        bool fine = l[nb][c] > 0.0f;
        const uint32_t qi = a.group.quot(static_cast<uint32_t>(row0 + r));
        const int32_t tok = seq.q0 + static_cast<int32_t>(qi), h = kvh * G + (row0 + r - static_cast<int32_t>(qi) * G);
        uint8_t* out = a.out + tok * a.o_token + h * a.o_head;
#pragma unroll
        for (int i = 0; i < OM; i += 4) {
          const int d = out_dim<FMT, DP>(i);
          uint32_t w[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float lo = o[nb][i + x][c] * inv, hi = o[nb][i + x][2 + c] * inv;
            fine = fine && fabsf(lo) < INFINITY && fabsf(hi) < INFINITY;
            w[x] = pack2(lo, hi, a.bf16);
          }
          if (d < a.head_dim) *reinterpret_cast<uint4*>(out + 2 * d) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (a.lse && g == 0u)
          a.lse[static_cast<int64_t>(tok) * a.q_heads + h] = (m[nb][c] + log2f(l[nb][c])) * 0.6931471805599453f;
        if (!fine) again |= 1u << r;
      }
    }
  again = __reduce_or_sync(0xFFFFFFFFu, again);
  if (again == 0u) return;
  const bool hold = waits != nullptr && lane == 0u;
  if (hold) waits->hold(1);
  __syncwarp();  // other lanes write these rows now (a reduction orders no memory)
  while (again != 0u) {
    const int32_t r = __ffs(static_cast<int>(again)) - 1;
    again &= again - 1u;
    const uint32_t qi = a.group.quot(static_cast<uint32_t>(row0 + r));
    attend_row<FMT, 8>(a, b, seq.len - seq.nq + static_cast<int32_t>(qi), seq.q0 + static_cast<int32_t>(qi),
                       kvh * G + (row0 + r - static_cast<int32_t>(qi) * G));
  }
  if (hold) waits->hold(-1);
}

// The sums of a part of an item, from row `at` of the workspace on.
template <int FMT, int DP, int NB, int OM>
__device__ __forceinline__ void write_part(const SplitParams& p, int64_t at, int32_t nrows, const float (&o)[NB][OM][4],
                                           const float (&m)[NB][2], const float (&l)[NB][2]) {
  const uint32_t lane = threadIdx.x & 31u, g = lane >> 2, t = lane & 3u;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int32_t r = nb * 8 + 2 * static_cast<int32_t>(t) + c;
      if (r >= nrows) continue;
      float* row = p.part_o + (at + r) * DP;
#pragma unroll
      for (int i = 0; i < OM; i += 2)
        *reinterpret_cast<float4*>(row + out_dim<FMT, DP>(i)) =
            make_float4(o[nb][i][c], o[nb][i][2 + c], o[nb][i + 1][c], o[nb][i + 1][2 + c]);
      if (g == 0u) *reinterpret_cast<float2*>(p.part_ml + (at + r) * 2) = make_float2(m[nb][c], l[nb][c]);
    }
}

// ---------------------------------------------------------------------------
// The kernel
// ---------------------------------------------------------------------------

constexpr int kSplitWarps = 8;

// Two CTAs an SM where the accumulators leave room for it.
template <int DP, int NB>
constexpr int kSplitCtas = DP * NB <= 128 ? 2 : 1;

// Ring units of a warp: as many (up to 6) as those CTAs can hold in 220 KB.
template <int FMT, int DP, int NB>
constexpr int kSplitFit = (220 * 1024 / kSplitCtas<DP, NB> - 2048) / (kSplitWarps * Layout<FMT, DP>::kUnit);
template <int FMT, int DP, int NB>
constexpr int kSplitUnits = kSplitFit<FMT, DP, NB> > 6 ? 6 : kSplitFit<FMT, DP, NB>;

// kBF16: the products' type (e4m3 and e2m1 caches: fp16).  kExact: head_dim is
// DP and a row's block scales begin at a multiple of their size, so that every
// piece is whole; otherwise pieces behind head_dim are cut or zero, and scales
// come by the words around them.
template <int FMT, int DP, int NB, bool kBF16, bool kExact>
__global__ void __launch_bounds__(32 * kSplitWarps, (kSplitCtas<DP, NB>))
    kv_attend_split(const __grid_constant__ SplitParams p) {
  using L = Layout<FMT, DP>;
  constexpr int NU = kSplitUnits<FMT, DP, NB>;
  static_assert(NU >= 3, "ring");
  static_assert(NU * L::kUnit >= NB * 8 * (DP + 2) * 4, "the join of a head's warps reuses the ring");
  constexpr int TW = L::TW, MB = L::MB;
  constexpr int QP = DP / 8;               // query pairs of a lane per row block
  constexpr int OM = L::VN * L::VD / 2;    // O^T products per key block
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t sh_scan[kSplitWarps];
  __shared__ int64_t sh_excl[32 * kSplitWarps + 1];  // first step of each thread's sequences; the total
  __shared__ int64_t sh_first[2];  // the share's first step's sequence, and that sequence's first step
  __shared__ SplitWork sh_work;
  __shared__ int32_t sh_next;

  const AttendParams& a = p.a;
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
  const uint32_t g = lane >> 2, t = lane & 3u;
  const int32_t G = static_cast<int32_t>(a.group.d);
  grid_handover();

  // -- the share of this CTA ------------------------------------------------
  // one row a sequence and no splits: item n is head group n % hgroups of sequence n / hgroups
  const bool direct = !p.split && a.q_start == nullptr && static_cast<int32_t>(a.group.d) <= p.rows;
  const int32_t per_thread = (a.num_seqs + static_cast<int32_t>(blockDim.x) - 1) / static_cast<int32_t>(blockDim.x);
  if (!direct) {
    const int32_t b0 = min(static_cast<int32_t>(threadIdx.x) * per_thread, a.num_seqs);
    const int32_t b1 = min(b0 + per_thread, a.num_seqs);
    int64_t mine = 0;
    for (int32_t b = b0; b < b1; ++b) mine += seq_units<L::TW>(p, b, blockIdx.x == 0);
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= static_cast<uint32_t>(o)) incl += v;
    }
    if (lane == 31u) sh_scan[warp] = incl;
    __syncthreads();
    {
      int64_t excl = incl - mine, total = 0;
      const uint32_t nwarps = blockDim.x >> 5;
      for (uint32_t w = 0; w < nwarps; ++w) {
        if (w < warp) excl += sh_scan[w];
        total += sh_scan[w];
      }
      sh_excl[threadIdx.x] = excl;
      if (threadIdx.x == 0) sh_excl[blockDim.x] = total;
      if (p.split && blockIdx.x == 0) {  // for the join
        for (int32_t i = b0; i < b1; ++i) {
          p.meta[i] = excl;
          excl += seq_units<L::TW>(p, i, false);
        }
      }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      if (p.split) {
        cut_shares(sh_excl[blockDim.x], static_cast<int32_t>(gridDim.x), p.max_shares, p.min_steps, &sh_work);
        if (blockIdx.x == 0) {
          for (int i = 0; i < sh_work.levels; ++i) p.head->level[i] = sh_work.level[i];
          p.head->levels = sh_work.levels;
        }
      } else {
        sh_work.level[0] = ShareLevel{0, 1, 0};
        sh_work.levels = 1;
        sh_work.shares = static_cast<int32_t>(sh_excl[blockDim.x]);
      }
    }
    __syncthreads();
  }

  const int32_t hl = static_cast<int32_t>(warp) % p.hw, sub = static_cast<int32_t>(warp) / p.hw;
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + warp * (NU * L::kUnit);
  const float kscale = a.scale_log2 * tensor_scale(a.k_scale);
  const float vscale = tensor_scale(a.v_scale);
  const uint32_t row_bytes = static_cast<uint32_t>(a.head_dim) * L::kBits / 8;
  // bytes of the lane's i-th K or V piece: less than a whole one behind head_dim
  auto kbytes = [&](int i) -> uint32_t {
    if (kExact) return L::KC;
    return static_cast<uint32_t>(min(max(static_cast<int32_t>(row_bytes) - static_cast<int32_t>(t + 4 * i) * L::KC, 0), L::KC));
  };
  auto vbytes = [&](int i) -> uint32_t {
    if (kExact) return L::VC;
    return static_cast<uint32_t>(min(max(static_cast<int32_t>(row_bytes) - static_cast<int32_t>(g + 8 * i) * L::VC, 0), L::VC));
  };

  // The scale code of a row's block. Blocks behind head_dim have none (their codes are 0; the bytes there,
  // in the copied words, are another head's or key's, and may be NaN).
  auto scale_of = [&](uint32_t block, uint32_t at) -> uint32_t {
    const uint32_t x = ld_shared_u8(at);
    return kExact || block < row_bytes / (kFp4Block / 2) ? x : 0u;
  };

  for (int32_t share = static_cast<int32_t>(blockIdx.x); direct || share < sh_work.shares;) {
    int64_t pos = share, end = share + 1, base = 0;
    int32_t b = 0;
    if (direct) {
      b = share / p.hgroups;
      base = static_cast<int64_t>(b) * p.hgroups;
    } else {
      int32_t level = sh_work.levels - 1;
      while (level > 0 && sh_work.level[level].first > share) --level;
      pos = sh_work.level[level].start + static_cast<int64_t>(share - sh_work.level[level].first) * sh_work.level[level].size;
      end = min(sh_excl[blockDim.x], pos + sh_work.level[level].size);
      if (pos >= sh_excl[threadIdx.x] && pos < sh_excl[threadIdx.x + 1]) {
        int64_t at = sh_excl[threadIdx.x];
        int32_t i = static_cast<int32_t>(threadIdx.x) * per_thread;
        for (; i < a.num_seqs; ++i) {
          const int64_t n = seq_units<L::TW>(p, i, false);
          if (pos < at + n) break;
          at += n;
        }
        sh_first[0] = i;
        sh_first[1] = at;
      }
      __syncthreads();
      b = static_cast<int32_t>(sh_first[0]);
      base = sh_first[1];
    }
  while (pos < end && b < a.num_seqs) {
    const AttendSeq seq = attend_seq(a, b, direct && threadIdx.x == 0 && share == b * p.hgroups);
    const SplitGeom geom = split_geom<TW>(p, seq);
    const int32_t unit = p.split ? geom.steps : 1;
    const int64_t local = pos - base;
    if (local >= static_cast<int64_t>(geom.blocks) * p.hgroups * unit) {
      base += static_cast<int64_t>(geom.blocks) * p.hgroups * unit;
      ++b;
      continue;
    }
    const int32_t item = static_cast<int32_t>(local / unit);
    const int32_t s_in = static_cast<int32_t>(local - static_cast<int64_t>(item) * unit);
    const int32_t s_out = static_cast<int32_t>(min(static_cast<int64_t>(unit), s_in + (end - pos)));
    const bool whole = s_out - s_in == unit;
    const int32_t step0 = p.split ? s_in : 0, step1 = p.split ? s_out : geom.steps;
    pos += s_out - s_in;
    const int32_t rb = item / p.hgroups, hg = item - rb * p.hgroups;
    const int32_t kvh = hg * p.hw + hl;
    const int32_t row0 = rb * p.rows;
    const int32_t nrows = min(p.rows, seq.nq * G - row0);
    const int32_t p_first = seq.len - seq.nq;  // position of the sequence's first query
    const int32_t q_lo = static_cast<int32_t>(a.group.quot(static_cast<uint32_t>(row0)));
    const int32_t q_hi = static_cast<int32_t>(a.group.quot(static_cast<uint32_t>(row0 + nrows - 1)));
    const int32_t p_lo = p_first + q_lo, p_hi = p_first + q_hi;
    const TileList list = visible_tiles<TW>(a, p_lo, p_hi);

    float o[NB][OM][4], m[NB][2], l[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int i = 0; i < OM; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[nb][i][c] = 0.0f;
      m[nb][0] = m[nb][1] = -INFINITY;
      l[nb][0] = l[nb][1] = 0.0f;
    }

    // -- the tiles ----------------------------------------------------------------------
    const int32_t* table = a.table + static_cast<int64_t>(b) * a.table_stride;
    const uint8_t* kbase = a.k + kvh * a.k_head;
    const uint8_t* vbase = a.v + kvh * a.v_head;
    // where the lane's first K row (g) and V row (2t) of 16 keys begin, less the block's own offset
    const uint8_t* klane = kbase + wide(g, p.k_slot) + t * L::KC;
    const uint8_t* vlane = vbase + wide(2 * t, p.v_slot) + g * L::VC;
    bool bad = false;  // a page id out of range was met
    // a lane's key of step i's tile: page id (-1: no row needs the key) and offset in the page
    auto lookup = [&](int32_t step, int32_t* id, uint32_t* off) {
      const int32_t i = step * p.subs + sub;
      const int32_t j = list.tile(i) * TW + static_cast<int32_t>(lane);
      *id = -1;
      *off = 0;
      if (lane < TW && step < step1 && i < list.n && j <= p_hi && (j >= list.lo_key || j < a.sinks)) {
        const uint32_t pg = a.page.quot(static_cast<uint32_t>(j));
        *off = static_cast<uint32_t>(j) - pg * a.page.d;
        const int32_t x = __ldg(table + pg);
        *id = x < 0 ? -2 : x;
      }
    };
    int32_t cur_id = -1, next_id;
    uint32_t cur_off = 0, next_off;
    bool cur_all = false;     // every key of the tile is wanted, and each 16 of them share a page
    lookup(step0, &next_id, &next_off);
    int32_t step_in = step0;  // step whose units are copied next
    uint32_t slot_in = 0;     // and the ring slot
    // the K rows of step `step_in` (kv 0) or its V rows (kv 1)
    auto copy_unit = [&](int kv) {
      if (kv == 0) {
        cur_id = next_id;
        cur_off = next_off;
        if (cur_id >= a.num_pages || cur_id == -2) {
          bad = true;
          record_oob(a.err, static_cast<uint64_t>(b));
          cur_id = -1;
        }
        cur_all = p.whole_blocks && __all_sync(0xFFFFFFFFu, lane >= TW || cur_id >= 0);
        lookup(step_in + 1, &next_id, &next_off);
      }
      if (step_in < step1) {
        const uint32_t unit_at = ring + slot_in * L::kUnit;
        const uint32_t kat = unit_at + lane * L::KC, vat = unit_at + lane * L::VC;
        if (cur_all) {
#pragma unroll
          for (int mb = 0; mb < MB; ++mb) {
            const int32_t id = __shfl_sync(0xFFFFFFFFu, cur_id, 16 * mb);
            const uint32_t off = __shfl_sync(0xFFFFFFFFu, cur_off, 16 * mb);
            if (kv == 0) {
              const uint8_t* src = klane + wide(id, p.k_page) + wide(off, p.k_slot);
#pragma unroll
              for (int rh = 0; rh < 2; ++rh) {
#pragma unroll
                for (int i = 0; i < L::KN; ++i)
                  copy_async<L::KC>(kat + ((2 * mb + rh) * L::KN + i) * 32 * L::KC, src + 4 * i * L::KC, kbytes(i));
                src += wide(8, p.k_slot);
              }
            } else {
              const uint8_t* src = vlane + wide(id, p.v_page) + wide(off, p.v_slot);
#pragma unroll
              for (int r = 0; r < 4; ++r) {
#pragma unroll
                for (int i = 0; i < L::VN; ++i)
                  copy_async<L::VC>(vat + ((4 * mb + r) * L::VN + i) * 32 * L::VC, src + 8 * i * L::VC, vbytes(i));
                src += wide((r & 1) ? 7 : 1, p.v_slot);
              }
            }
          }
        } else if (kv == 0) {
#pragma unroll
          for (int r = 0; r < 2 * MB; ++r) {
            const int32_t id = __shfl_sync(0xFFFFFFFFu, cur_id, 8 * r + g);
            const uint32_t off = __shfl_sync(0xFFFFFFFFu, cur_off, 8 * r + g);
            const uint8_t* src = kbase + t * L::KC + (id < 0 ? 0 : wide(id, p.k_page) + wide(off, p.k_slot));
#pragma unroll
            for (int i = 0; i < L::KN; ++i) {
              const uint32_t n = id < 0 ? 0u : kbytes(i);
              copy_async<L::KC>(kat + (r * L::KN + i) * 32 * L::KC, n ? src + 4 * i * L::KC : kbase, n);
            }
          }
        } else {
#pragma unroll
          for (int r = 0; r < 4 * MB; ++r) {
            const uint32_t tok = 16u * (r / 4) + 2u * t + (r & 1) + 8u * ((r >> 1) & 1);
            const int32_t id = __shfl_sync(0xFFFFFFFFu, cur_id, tok);
            const uint32_t off = __shfl_sync(0xFFFFFFFFu, cur_off, tok);
            const uint8_t* src = vbase + g * L::VC + (id < 0 ? 0 : wide(id, p.v_page) + wide(off, p.v_slot));
#pragma unroll
            for (int i = 0; i < L::VN; ++i) {
              const uint32_t n = id < 0 ? 0u : vbytes(i);
              copy_async<L::VC>(vat + (r * L::VN + i) * 32 * L::VC, n ? src + 8 * i * L::VC : vbase, n);
            }
          }
        }
        if constexpr (FMT == KV_CACHE_E2M1) {
          // lane = key: the aligned words around its row's scales, and where in them the row begins
          const uint8_t* sbase = kv == 0 ? a.k_sc + kvh * a.ks_head : a.v_sc + kvh * a.vs_head;
          const uint8_t* src = sbase + (cur_id < 0 ? 0
                                        : kv == 0 ? wide(cur_id, p.ks_page) + wide(cur_off, p.ks_slot)
                                                  : wide(cur_id, p.vs_page) + wide(cur_off, p.vs_slot));
          const uint32_t at = unit_at + TW * L::kRow + lane * L::kScaleRow;
          uint32_t need = cur_id < 0 ? 0u : row_bytes / 8;  // a scale per 8 code bytes
          if constexpr (kExact) {
            copy_async<DP / 16>(at, src, cur_id < 0 ? 0u : DP / 16);
          } else {
            const uint32_t mis = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(src) & 3u);
            need += cur_id < 0 ? 0u : mis;
#pragma unroll
            for (int i = 0; i < L::kScaleRow / 4 - 1; ++i)
              copy_async<4>(at + 4 * i, 4u * i < need ? src - mis + 4 * i : src - mis, 4u * i < need ? 4u : 0u);
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + L::kScaleRow - 4), "r"(mis) : "memory");
          }
        }
      }
      commit_async();
      if (kv == 1) ++step_in;
      slot_in = slot_in + 1 == NU ? 0u : slot_in + 1;
    };
#pragma unroll
    for (int i = 0; i < NU - 1; ++i) copy_unit(i & 1);

    // -- queries: lane (g, t) holds the pairs of row g that K's pieces t, t + 4, .. meet -----
    uint32_t qf[NB][QP];
    float rs[NB][2];  // softmax scale of rows 2t, 2t + 1
    load_queries<FMT, DP, NB>(a, seq, kvh, row0, nrows, kscale,
                              [&](int i) { return (static_cast<int>(t) + 4 * ((2 * i) / L::KD)) * L::KD + (2 * i) % L::KD; }, qf, rs);

    uint32_t slot = 0;
    auto next_slot = [&] { slot = slot + 1 == NU ? 0u : slot + 1; };
    for (int32_t step = step0; step < step1; ++step) {
      // S^T = K Q^T
      wait_async<NU - 2>();
      __syncwarp();
      copy_unit((NU - 1) & 1);
      float s[MB][NB][4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[mb][nb][c] = 0.0f;
      const uint32_t kat = ring + slot * L::kUnit;
#pragma unroll
      for (int i = 0; i < L::KN; ++i) {
        uint32_t w[MB][2][L::KC / 4], sc[MB][2];
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int rh = 0; rh < 2; ++rh) {
            ld_own<L::KC>(w[mb][rh], kat + (((mb * 2 + rh) * L::KN + i) * 32 + lane) * L::KC);
            sc[mb][rh] = 0u;
            if constexpr (FMT == KV_CACHE_E2M1) {
              const uint32_t srow = kat + TW * L::kRow + (mb * 16 + rh * 8 + g) * L::kScaleRow;
              const uint32_t block = (t + 4 * i) * (L::KD / kFp4Block);
              uint32_t sat = srow + block;
              if (!kExact) sat += ld_shared_u32(srow + L::kScaleRow - 4);
              if (L::KD > kFp4Block && kExact) {
                sc[mb][rh] = ld_shared_u16(sat);
              } else {
                sc[mb][rh] = scale_of(block, sat);
                if constexpr (L::KD > kFp4Block) sc[mb][rh] |= scale_of(block + 1, sat + 1) << 8;
              }
            }
          }
        k_products<FMT, DP, NB, kBF16>(s, w, sc, qf, i * (L::KD / 2));
      }
      next_slot();

      // mask: s[..][0], [1]: key g, rows 2t, 2t + 1; [2], [3]: key g + 8
      const int32_t li = step * p.subs + sub, j0 = list.tile(li) * TW;
      const bool all_seen = li < list.n && j0 + TW - 1 <= p_lo &&
                            (a.window == 0 || j0 > p_hi - a.window || j0 + TW - 1 < a.sinks);
      const bool any_bad = __any_sync(0xFFFFFFFFu, bad);
      if (!all_seen || any_bad) {
        hide_scores<NB, MB>(a, table, j0, li < list.n ? p_hi : -1, any_bad, p_first, row0, g, s);
      }

      // running maximum and sum
      uint32_t pt[MB][NB][2], pl[MB][NB][2];
      softmax_step<FMT, NB, MB, OM, kBF16>(s, rs, m, l, o, pt, pl);

      // O^T += V^T P^T
      wait_async<NU - 2>();
      __syncwarp();
      copy_unit(NU & 1);
      const uint32_t vat = ring + slot * L::kUnit;
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        uint32_t srow[4];
        if constexpr (FMT == KV_CACHE_E2M1) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const uint32_t tok = 16u * mb + 2u * t + (r & 1) + 8u * (r >> 1);
            const uint32_t at = vat + TW * L::kRow + tok * L::kScaleRow;
            srow[r] = at;
            if (!kExact) srow[r] += ld_shared_u32(at + L::kScaleRow - 4);
          }
        }
#pragma unroll
        for (int i = 0; i < L::VN; ++i) {
          uint32_t w[4][L::VC / 4], sc[2][2] = {{0u, 0u}, {0u, 0u}};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            ld_own<L::VC>(w[x], vat + (((mb * 4 + x) * L::VN + i) * 32 + lane) * L::VC);
            if constexpr (FMT == KV_CACHE_E2M1) {
#pragma unroll
              for (int y = 0; y < (L::VD + kFp4Block - 1) / kFp4Block; ++y) {
                const uint32_t block = (g + 8 * i) * L::VD / kFp4Block + y;
                sc[x >> 1][y] |= scale_of(block, srow[x] + block) << (8 * (x & 1));
              }
            }
          }
          v_products<FMT, DP, NB, kBF16>(o, w, sc, pt[mb], pl[mb], i * (L::VD / 2));
        }
      }
      next_slot();
    }
    wait_async<0>();

    // -- the item's end -----------------------------------------------------------------
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x = l[nb][c];
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 4);
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 8);
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 16);
        l[nb][c] = x;
      }
    if (p.subs > 1) {
      // the warps of a head join theirs in shared memory: [row][DP + 2] floats each
      float* own = reinterpret_cast<float*>(smem + warp * (NU * L::kUnit));
      __syncwarp();
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float* row = own + (nb * 8 + 2 * t + c) * (DP + 2);
#pragma unroll
          for (int i = 0; i < OM; ++i) {
            const int d = (static_cast<int>(g) + 8 * (2 * i / L::VD)) * L::VD + 2 * i % L::VD;
            row[d] = o[nb][i][c];
            row[d + 1] = o[nb][i][2 + c];
          }
          if (g == 0u) {
            row[DP] = m[nb][c];
            row[DP + 1] = l[nb][c];
          }
        }
      __syncthreads();
      for (int32_t r = sub; r < nrows; r += p.subs) {
        float mm = -INFINITY;
        for (int32_t x = 0; x < p.subs; ++x)
          mm = fmaxf(mm, reinterpret_cast<const float*>(smem + (x * p.hw + hl) * (NU * L::kUnit))[r * (DP + 2) + DP]);
        const float ref = mm == -INFINITY ? 0.0f : mm;
        float ll = 0.0f, acc[DP / 32];
#pragma unroll
        for (int i = 0; i < DP / 32; ++i) acc[i] = 0.0f;
        for (int32_t x = 0; x < p.subs; ++x) {
          const float* row = reinterpret_cast<const float*>(smem + (x * p.hw + hl) * (NU * L::kUnit)) + r * (DP + 2);
          const float e = exp2_fast(row[DP] - ref);
          ll = __fmaf_rn(row[DP + 1], e, ll);
#pragma unroll
          for (int i = 0; i < DP / 32; ++i) acc[i] = __fmaf_rn(row[lane + 32 * i], e, acc[i]);
        }
        if (whole) {
          const uint32_t qi = a.group.quot(static_cast<uint32_t>(row0 + r));
          const int32_t tok = seq.q0 + static_cast<int32_t>(qi), h = kvh * G + (row0 + r - static_cast<int32_t>(qi) * G);
          const float inv = __fdiv_rn(vscale, ll);
          bool fine = ll > 0.0f;
#pragma unroll
          for (int i = 0; i < DP / 32; ++i) fine = fine && fabsf(acc[i] * inv) < INFINITY;
          if (!__all_sync(0xFFFFFFFFu, fine)) {
            attend_row<FMT, 8>(a, b, p_first + static_cast<int32_t>(qi), tok, h);
            continue;
          }
          uint16_t* out = reinterpret_cast<uint16_t*>(a.out + tok * a.o_token + h * a.o_head);
#pragma unroll
          for (int i = 0; i < DP / 32; ++i)
            if (static_cast<int32_t>(lane) + 32 * i < a.head_dim) out[lane + 32 * i] = round16(acc[i] * inv, a.bf16);
          if (a.lse && lane == 0u)
            a.lse[static_cast<int64_t>(tok) * a.q_heads + h] = (mm + log2f(ll)) * 0.6931471805599453f;
        } else {
          const int64_t at = (static_cast<int64_t>(2 * share + (step0 == 0 ? 1 : 0)) * p.hw + hl) * p.part_rows + r;
#pragma unroll
          for (int i = 0; i < DP / 32; ++i) p.part_o[at * DP + lane + 32 * i] = acc[i];
          if (lane == 0u) *reinterpret_cast<float2*>(p.part_ml + at * 2) = make_float2(mm, ll);
        }
      }
      __syncthreads();
      continue;
    }
    if (whole) {
      write_rows<FMT, DP, NB>(a, b, seq, kvh, row0, nrows, vscale, o, m, l);
    } else {
      write_part<FMT, DP, NB>(p, (static_cast<int64_t>(2 * share + (step0 == 0 ? 1 : 0)) * p.hw + hl) * p.part_rows, nrows, o, m, l);
    }
  }
    if (!p.split) break;  // as many CTAs as items
    __syncthreads();      // all warps have read sh_first
    if (threadIdx.x == 0) sh_next = static_cast<int32_t>(gridDim.x + atomicAdd(&p.head->next, 1u));
    __syncthreads();
    share = sh_next;
  }
}

constexpr int kJoinWarps = 16;

// Joins the parts of the items that were split, in the order of their keys:
// `wpr` warps of the CTA take one output row.
template <int FMT, int DP, int TW>
__global__ void __launch_bounds__(32 * kJoinWarps) kv_attend_join(const __grid_constant__ SplitParams p, const int32_t wpr) {
  __shared__ float sh[kJoinWarps][DP + 2];
  const AttendParams& a = p.a;
  const uint32_t lane = threadIdx.x & 31u;
  const int32_t warp = static_cast<int32_t>(threadIdx.x >> 5), part = warp % wpr;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kJoinWarps / wpr) + warp / wpr;
  const int32_t tok = static_cast<int32_t>(unit / a.q_heads), h = static_cast<int32_t>(unit - static_cast<int64_t>(tok) * a.q_heads);
  grid_handover();
  if (blockIdx.x == 0 && threadIdx.x == 0) p.head->next = 0u;
  int32_t b = tok, c0 = 0, c1 = 0, hl = 0, r = 0, pos = 0;
  bool joined = false, lost = false;
  if (tok < a.num_q) {
    if (a.q_start) {
      int32_t lo = 0, hi = a.num_seqs - 1;
      while (lo < hi) {
        const int32_t mid = (lo + hi + 1) >> 1;
        if (__ldg(a.q_start + mid) <= tok) lo = mid; else hi = mid - 1;
      }
      b = lo;
    }
    const AttendSeq s = attend_seq(a, b, false);
    if (tok >= s.q0 && tok < s.q0 + s.nq) {
      const SplitGeom geom = split_geom<TW>(p, s);
      const int32_t G = static_cast<int32_t>(a.group.d), kvh = static_cast<int32_t>(a.group.quot(static_cast<uint32_t>(h)));
      const int32_t row = (tok - s.q0) * G + (h - kvh * G);
      const int32_t rb = row / p.rows, hg = kvh / p.hw;
      hl = kvh - hg * p.hw;
      r = row - rb * p.rows;
      pos = s.len - s.nq + (tok - s.q0);
      const int64_t s0 = p.meta[b] + (static_cast<int64_t>(rb) * p.hgroups + hg) * geom.steps;
      c0 = share_of(p.head, s0);
      c1 = share_of(p.head, s0 + geom.steps - 1);
      joined = c0 != c1;
      lost = p.head->gave_up != 0u;
    }
  }
  // all warps of a row agree on `joined`; with one warp a row there is no barrier below
  float mm = -INFINITY, ll = 0.0f, acc[DP / 32];
#pragma unroll
  for (int i = 0; i < DP / 32; ++i) acc[i] = 0.0f;
  if (joined) {
    for (int32_t c = c0 + part; c <= c1; c += 4 * wpr) {
      float2 ml[4];
      float v[4][DP / 32];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int32_t cc = c + x * wpr;
        ml[x] = make_float2(-INFINITY, 0.0f);
#pragma unroll
        for (int i = 0; i < DP / 32; ++i) v[x][i] = 0.0f;
        if (cc <= c1) {
          const int64_t at = (static_cast<int64_t>(2 * cc + (cc == c0 ? 1 : 0)) * p.hw + hl) * p.part_rows + r;
          ml[x] = __ldcg(reinterpret_cast<const float2*>(p.part_ml + at * 2));
#pragma unroll
          for (int i = 0; i < DP / 32; ++i) v[x][i] = __ldcg(p.part_o + at * DP + lane + 32 * i);
        }
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float mn = fmaxf(mm, ml[x].x), ref = mn == -INFINITY ? 0.0f : mn;
        const float ea = exp2_fast(mm - ref), eb = exp2_fast(ml[x].x - ref);
        mm = mn;
        ll = __fmaf_rn(ll, ea, ml[x].y * eb);
#pragma unroll
        for (int i = 0; i < DP / 32; ++i) acc[i] = __fmaf_rn(acc[i], ea, v[x][i] * eb);
      }
    }
  }
  if (wpr > 1) {
#pragma unroll
    for (int i = 0; i < DP / 32; ++i) sh[warp][lane + 32 * i] = acc[i];
    if (lane == 0u) {
      sh[warp][DP] = mm;
      sh[warp][DP + 1] = ll;
    }
    __syncthreads();
    if (part != 0) return;
    for (int32_t w = warp + 1; w < warp + wpr; ++w) {
      const float mw = sh[w][DP], mn = fmaxf(mm, mw), ref = mn == -INFINITY ? 0.0f : mn;
      const float ea = exp2_fast(mm - ref), eb = exp2_fast(mw - ref);
      mm = mn;
      ll = __fmaf_rn(ll, ea, sh[w][DP + 1] * eb);
#pragma unroll
      for (int i = 0; i < DP / 32; ++i) acc[i] = __fmaf_rn(acc[i], ea, sh[w][lane + 32 * i] * eb);
    }
  }
  uint16_t* out = reinterpret_cast<uint16_t*>(a.out + tok * a.o_token + h * a.o_head);
  if (lost) {  // parts are missing, or whole rows: NaN, whatever was computed
    for (int32_t d = static_cast<int32_t>(lane); d < a.head_dim; d += 32) out[d] = 0x7FFFu;
    if (a.lse && lane == 0u) a.lse[static_cast<int64_t>(tok) * a.q_heads + h] = __uint_as_float(0x7FFFFFFFu);
    return;
  }
  if (!joined) return;
  const float inv = __fdiv_rn(tensor_scale(a.v_scale), ll);
  bool fine = ll > 0.0f;
#pragma unroll
  for (int i = 0; i < DP / 32; ++i) fine = fine && fabsf(acc[i] * inv) < INFINITY;
  if (!__all_sync(0xFFFFFFFFu, fine)) {
    attend_row<FMT, 8>(a, b, pos, tok, h);
    return;
  }
#pragma unroll
  for (int i = 0; i < DP / 32; ++i)
    if (static_cast<int32_t>(lane) + 32 * i < a.head_dim) out[lane + 32 * i] = round16(acc[i] * inv, a.bf16);
  if (a.lse && lane == 0u)
    a.lse[static_cast<int64_t>(tok) * a.q_heads + h] = (mm + log2f(ll)) * 0.6931471805599453f;
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------

// Raises a kernel's dynamic shared memory limit once per device.
struct SmemOptIn {
  std::atomic<uint64_t> done{0};
  kv_status operator()(const void* kernel, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    const uint64_t bit = dev >= 0 && dev < kMaxDevices ? uint64_t{1} << dev : 0u;
    if ((done.load(std::memory_order_acquire) & bit) != 0u) return KV_OK;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return cuda_fail(e);
    done.fetch_or(bit, std::memory_order_release);
    return KV_OK;
  }
};

// A launch that may overlap its predecessor's end (programmatic dependent launch).
template <typename... P, typename... A>
kv_status launch_chained(void (*kernel)(P...), int64_t grid, int threads, int smem, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  return e == cudaSuccess ? KV_OK : cuda_fail(e);
}

// The KV heads that a CTA with room for `most` takes: the most that divide them.
inline int heads_of_cta(int kv_heads, int most) {
  int n = 1;
  for (int h = 2; h <= most; ++h)
    if (kv_heads % h == 0) n = h;
  return n;
}

// Heads and warps of a CTA, and the workspace; returns the CTAs to launch, at most `full` where items
// are split.
template <int DP>
int64_t set_up_split(SplitParams& p, int heads, int rows, int tile, int64_t full, void* work, int64_t work_bytes, int64_t max_keys) {
  const AttendParams& a = p.a;
  p.rows = rows;
  p.hw = heads_of_cta(a.kv_heads, heads);
  p.subs = heads / p.hw;
  p.hgroups = a.kv_heads / p.hw;
  p.min_steps = kMinSteps;
  // An item that cannot be longer than the shortest share is not split, nor is
  // any where the workspace holds the parts of less than half the GPU.
  const int64_t meta = (static_cast<int64_t>(a.num_seqs) + 31) / 32 * 256;
  p.part_rows = a.q_start || static_cast<int32_t>(a.group.d) > p.rows ? p.rows : static_cast<int32_t>(a.group.d);
  const int64_t slot = static_cast<int64_t>(p.hw) * p.part_rows * (DP + 2) * 4;
  int64_t fit = work && work_bytes > kSplitHead + meta ? (work_bytes - kSplitHead - meta) / (2 * slot) : 0;
  if (fit > kLevels * full) fit = kLevels * full;
  p.split = max_keys > static_cast<int64_t>(p.min_steps) * p.subs * tile && 2 * fit >= full;
  if (p.split) {
    p.max_shares = static_cast<int32_t>(fit);
    p.head = static_cast<SplitWork*>(work);
    p.meta = reinterpret_cast<int64_t*>(static_cast<uint8_t*>(work) + kSplitHead);
    p.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(work) + kSplitHead + meta);
    p.part_ml = p.part_o + 2 * fit * p.hw * p.part_rows * DP;
    return fit < full ? fit : full;
  }
  if (!a.q_start && static_cast<int32_t>(a.group.d) <= p.rows)  // one row a sequence: the kernel's direct items
    return static_cast<int64_t>(a.num_seqs) * p.hgroups;
  // a CTA an item: at most this many
  const int64_t items = (static_cast<int64_t>(a.num_q) * a.group.d / p.rows + a.num_seqs) * p.hgroups;
  return items < 0x7FFFFFFF ? items : 0x7FFFFFFF;
}

// The fewer the rows, the more parts has each and the more warps take it.
template <int FMT, int DP, int TW>
kv_status launch_join(const SplitParams& p, int sms, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(p.a.num_q) * p.a.q_heads;
  int32_t wpr = 1;
  while (wpr < kJoinWarps && rows * wpr < 16ll * sms) wpr *= 2;
  const int64_t per = kJoinWarps / wpr;
  return launch_chained(kv_attend_join<FMT, DP, TW>, (rows + per - 1) / per, 32 * kJoinWarps, 0, stream, p, wpr);
}

// Launches the split kernel (and the join) of one format and padded head dim.
template <int FMT, int DP, int NB, bool kBF16, bool kExact>
kv_status launch_split(SplitParams p, void* work, int64_t work_bytes, int64_t max_keys, cudaStream_t stream) {
  using L = Layout<FMT, DP>;
  constexpr int kSmem = kSplitWarps * kSplitUnits<FMT, DP, NB> * L::kUnit;
  auto* kernel = kv_attend_split<FMT, DP, NB, kBF16, kExact>;
  int sms = 0;
  kv_status st = current_sm_count(&sms);
  if (st != KV_OK) return st;
  static SmemOptIn opt_in;
  st = opt_in(reinterpret_cast<const void*>(kernel), kSmem);
  if (st != KV_OK) return st;
  const int64_t grid = set_up_split<DP>(p, kSplitWarps, 8 * NB, L::TW, static_cast<int64_t>(sms) * kSplitCtas<DP, NB>, work, work_bytes, max_keys);
  st = launch_chained(kernel, grid, 32 * p.hw * p.subs, kSmem, stream, p);
  if (st != KV_OK || !p.split) return st;
  return launch_join<FMT, DP, L::TW>(p, sms, stream);
}

template <int FMT, bool kBF16>
kv_status launch_split_fmt(const SplitParams& p, bool wide, void* work, int64_t work_bytes, int64_t max_keys,
                           cudaStream_t stream) {
  const int d = p.a.head_dim;
  bool exact = d == 64 || d == 128;
  if (FMT == KV_CACHE_E2M1)
    exact = exact && ((u64(p.a.k_sc) | u64(p.a.v_sc) | u64(p.a.ks_head) | u64(p.a.vs_head) | u64(int64_t{p.ks_page}) |
                       u64(int64_t{p.ks_slot}) | u64(int64_t{p.vs_page}) | u64(int64_t{p.vs_slot})) &
                      static_cast<uint64_t>(d / 16 - 1)) == 0;
#define KV_SPLIT(DP, NB, EX) launch_split<FMT, DP, NB, kBF16, EX>(p, work, work_bytes, max_keys, stream)
  if (d <= 64)
    return exact ? (wide ? KV_SPLIT(64, 2, true) : KV_SPLIT(64, 1, true))
                 : (wide ? KV_SPLIT(64, 2, false) : KV_SPLIT(64, 1, false));
  if (d <= 128)
    return exact ? (wide ? KV_SPLIT(128, 2, true) : KV_SPLIT(128, 1, true))
                 : (wide ? KV_SPLIT(128, 2, false) : KV_SPLIT(128, 1, false));
  return KV_SPLIT(256, 1, false);
#undef KV_SPLIT
}

// The formats' instantiations, a translation unit each.
kv_status split_bf16(const SplitParams& p, bool wide, void* work, int64_t work_bytes, int64_t max_keys, cudaStream_t stream);
kv_status split_f16(const SplitParams& p, bool wide, void* work, int64_t work_bytes, int64_t max_keys, cudaStream_t stream);
kv_status split_e4m3(const SplitParams& p, bool wide, void* work, int64_t work_bytes, int64_t max_keys, cudaStream_t stream);
kv_status split_e2m1(const SplitParams& p, bool wide, void* work, int64_t work_bytes, int64_t max_keys, cudaStream_t stream);

}  // namespace kvimpl
