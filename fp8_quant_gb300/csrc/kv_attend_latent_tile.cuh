// Attention over a paged cache of latent rows on the tensor cores (tcgen05).
//
// All query heads share one row of D dims per key, L of them values, so a key's
// bytes meet HQ rows a query: 4 * HQ * (D + L) / (4 * D) operations a byte, 60
// for 32 heads of 576 / 512. One query a sequence is bound by the cache's
// bytes, from about four queries on by the products.
//
// A CTA takes up to NR = 64 or 32 query rows, a row being a (query, head)
// pair, and goes over tiles of 32 keys:
//   S [rows][keys] = Q K^T       M = 64 (Q: 320 dims in TMEM, with 32 rows all, the others in shared memory), N = 32 keys;
//   O^T [dims][rows] += V^T P^T  M = 128 dims, N = NR rows: the tile's first L
//                                dims as they lie (dims contiguous), P in
//                                shared memory.
// O^T of 512 dims then is 4 x NR columns of TMEM (256 of 512 for 64 rows; with
// rows as M it would be all of it), a key tile is brought in once for both
// products, and the rows that do not fill M = 128 cost nothing.
//
//   warps 0-3  the softmax: S by 16x256b loads (a thread has 8 keys of two rows),
//              running maximum and sums in registers, P to shared memory. A tile's scores are only compared with the
//              running maxima; these, and O^T, are brought up to date when some row's grew by 2^8 or more (the reduction
//              over a row's threads in every tile: 32 heads over e4m3fn 172 us, 154 without). With 32 rows the 64 of a
//              product hold them twice, and warps 2 and 3 take half of the keys. They also bring the queries in and
//              write the outputs.
//   warps 4, 8 issue the products S, of every other tile each, up to three tiles ahead of
//   warp  5    P V. (A product takes 31 clocks to issue and 25 to 48 to run: with one warp for S decode below takes
//              152 us, where two take 137; over e4m3fn 209 and 154; chunks 1,229 and 927.)
//   warp  6    cuts the work: finds the CTA's next items and hands them to the others.
//   warp  7    brings the keys, a tile a unit of the ring: by TMA, a box for all of it where its 32 keys exist and share a
//              page, else by cp.async. e4m3fn rows come as they are, into a ring of their own, and become fp16 (exact) by
//   warps 9-15 on their way into the ring of units.
//   A unit lies as [8 keys][64 dims][key][128 bytes in the 128-byte swizzle], as a box of the cache's eights of keys does.
//   It is given back when P V has gone over it. Tiles are small because that time is what the
//   ring has to cover beside the memory's latency: tiles of 64 keys hold it twice as long (decode 13 % slower when both
//   forms were there), and so do products S over two tiles at once, which run 36 % faster a key (chunks 19 % slower).
//
// Measured (one GB300): 64 sequences of 4,000 - 16,384 bf16 keys, 32 heads, one token each (decode) 136 us, 83 % of the
// copy rate for its bytes; chunks of 700 - 1,023 tokens over 5,000 - 8,190 keys 915 - 927 us, 846 - 834 TFLOP/s: the products' own
// time, 36 x 25 + 8 x 48 clocks a tile, is 83 % of it; 32 sequences of 16,000 - 32,768 e4m3fn keys 154 us: products and
// conversions share the 128 bytes a clock of shared memory (S 288, P V 320, conversions 576 of 1,730 clocks a tile).
//
// Rows beyond NR (more queries, more heads) are further items, which read the same keys: mostly from L2.
//
// Weights are rounded once to 16 bits, as the product's operand (a second term, as kv_attend's split kernels keep for 16-bit
// caches, would be P V a second time; up to 2^-9 or 2^-12 of sum p |k| / sum p, as the header says); their sums are
// of the unrounded ones in fp32. An e4m3fn row's scale f multiplies its scores,
// and its weights p before they are rounded: the running reference is the
// maximum of score + log2 f, so that p f, not p, begins at 2^7.
//
// Few long sequences are split over the CTAs by keys, in steps of a tile, counted
// on the device, a share for each CTA; parts are joined in the order of the keys by a second kernel.
//
// Every wait has a limit (kSpin); a CTA whose wait ran out records that in the
// error record and in the workspace's head, lets its copies and products end and leaves.
#pragma once

#include <type_traits>

#include "kv_attend_latent.cuh"
#include "kv_attend_tile.cuh"

namespace kvimpl {

constexpr int kLatKeys = 32;        // keys of a tile, which is a unit of the ring
constexpr int kLatMaxChunks = 9;    // 64-dim chunks of a row: up to 576 dims
constexpr int kLatMaxUnits = 8, kLatMaxRaws = 8;
constexpr int kLatScores = 3;       // tiles whose scores may be in TMEM
constexpr int kLatMinSteps = 2;     // steps of a share at least
// Steps that an item counts beside its tiles where items are split: what its queries, first scores and outputs take. (24 heads,
// 200 - 777 tokens over e4m3fn keys 469 us with none, 453 with 4, 435 with 8, 433 with 12; 32 heads, one token 158, 156.5, 154,
// 152; over 16-bit keys 140, 137.5, 136.5, 135.5.)
constexpr int kLatItemSteps = 8;

struct LatentTileParams {
  LatentParams l;
  CUtensorMap map;
  int32_t box;       // groups of eight keys in a TMA box: 1, 2 or 4; 0: cp.async alone
  int32_t box_chunks;  // chunks of one: 1 or all
  int32_t page_stride, slot_stride;  // of the cache, bytes in 32 bits
  int32_t chunks;    // 64-dim chunks of a row, the last perhaps cut
  int32_t ksteps;    // 16-dim steps of a row
  int32_t blocks;    // 128-dim blocks of the values
  int32_t units, raws;  // of the ring, and of that of e4m3fn rows
  int32_t split;     // 0: an item is one CTA's
  int32_t part_rows;
  SplitWork* head;
  int64_t* meta;     // [num_seqs]: first step of each sequence
  float *part_o, *part_ml;  // [2 * shares][part_rows] x 128 * blocks and x 2
};

constexpr int kLatConverters = 7;  // warps
template <int FMT>
constexpr int kLatThreads = 288 + (FMT == KV_CACHE_SRC ? 0 : 32 * kLatConverters);

// A CTA's next piece of work.
struct LatentSeg {
  int32_t b, q0, nq, p_first;  // sequence, its first query row and their number, position of the first
  int32_t row0, nrows, last;   // its rows: (query, head) pairs of the sequence; the last, from row0
  int32_t p_hi;                // position of the item's last row
  int32_t t0, t1;              // tiles
  int32_t part;                // -1: the item is whole; else the part's place
  int32_t stop;
};

template <int FMT, int NR>
struct LatentSmem {  // units, raw units, queries, weights, and
  static constexpr int kP = NR * 128;
  static constexpr int kBars = 2 * kLatMaxUnits + 2 * kLatMaxRaws + 2 * kLatScores + 15;
  static __host__ __device__ constexpr int unit(int chunks) { return kLatKeys * 128 * chunks; }
  static __host__ __device__ constexpr int raw(int chunks) { return kLatKeys * 64 * chunks; }
  // chunks of the queries that are in TMEM, beside O^T and the scores; the others are in shared memory
  static constexpr int kInTmem = NR == 64 ? 5 : 9;
  static __host__ __device__ constexpr int q_bytes(int chunks) { return chunks > kInTmem ? (chunks - kInTmem) * NR * 128 : 0; }
  static constexpr int kOffBars = 0, kOffSegs = (kBars * 8 + 15) / 16 * 16, kOffAlpha = kOffSegs + 2 * 64, kOffInv = kOffAlpha + NR * 4,
                       kOffQf = kOffInv + NR * 4, kOffTop = kOffQf + NR * 4, kOffMisc = kOffTop + 64 * 4, kOffValid = kOffMisc + 64,
                       kOffRawValid = kOffValid + kLatMaxUnits * 4, kOffScale = kOffRawValid + kLatMaxRaws * 4;
  static __host__ __device__ constexpr int total(int chunks, int units, int raws) {
    return units * (unit(chunks) + (FMT == KV_CACHE_SRC ? 0 : 2 * kLatKeys * 4)) + raws * (raw(chunks) + kLatKeys * 4) + q_bytes(chunks) + kP + kOffScale;
  }
};
static_assert(sizeof(LatentSeg) <= 64, "segments");
static_assert(kLatThreads<KV_CACHE_E4M3FN> == 512, "176 + 3 x 112 registers of four warpgroups are the launch's 512 x 128");
static_assert(LatentSmem<KV_CACHE_SRC, 64>::total(kLatMaxChunks, 5, 0) <= 227 * 1024 &&
                  LatentSmem<KV_CACHE_E4M3FN, 64>::total(kLatMaxChunks, 3, 4) <= 227 * 1024, "the widest rows fit");
static_assert(4 * 64 + kLatScores * kLatKeys + 32 * LatentSmem<KV_CACHE_SRC, 64>::kInTmem <= 512 &&
                  4 * 32 + kLatScores * kLatKeys + 32 * LatentSmem<KV_CACHE_SRC, 32>::kInTmem <= 512, "TMEM");

// Rows of the sequence's queries in blocks of NR, and steps of each: kLatItemSteps, and its tiles (an upper bound, at
// least one).
struct LatentGeom {
  int32_t blocks, steps;
};

template <int NR>
__device__ __forceinline__ LatentGeom latent_geom(const LatentTileParams& p, const AttendSeq& s) {
  LatentGeom g;
  g.blocks = static_cast<int32_t>((static_cast<uint32_t>(s.nq) * p.l.a.group.d + NR - 1) / NR);
  g.steps = max((s.len + kLatKeys - 1) / kLatKeys, 1) + kLatItemSteps;
  return g;
}

template <int NR>
__device__ __forceinline__ int64_t latent_units(const LatentTileParams& p, int32_t b, bool record) {
  const LatentGeom g = latent_geom<NR>(p, attend_seq(p.l.a, b, record));
  return static_cast<int64_t>(g.blocks) * (p.split ? g.steps : 1);
}

// Of non-negative numbers, most of them short.
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t d) {
  return ((x | d) >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(x) / static_cast<uint32_t>(d)) : x / d;
}

// A share for each CTA, all of a size. (Smaller shares behind them, for those that are done first, cost more in
// queries brought in and parts written than they balance.)
__device__ __forceinline__ ShareLevel latent_cut(int64_t total, int32_t ctas, int32_t* shares) {
  int64_t each = quotient(total + ctas - 1, ctas);
  if (each < kLatMinSteps) each = kLatMinSteps;
  *shares = static_cast<int32_t>(quotient(total + each - 1, each));
  return ShareLevel{0, static_cast<int32_t>(each), 0};
}

// The bits of a warp's own keys, kCols of a unit's 32.
template <int kCols>
__host__ __device__ constexpr uint32_t own_keys(uint32_t valid, uint32_t half) {
  return valid >> (kCols * half) & (~0u >> (32 - kCols));
}
static_assert(own_keys<32>(~0u, 0) == ~0u && own_keys<16>(~0u, 0) == 0xFFFFu && own_keys<16>(~0u, 1) == 0xFFFFu &&
                  own_keys<16>(0xABCD1234u, 0) == 0x1234u && own_keys<16>(0xABCD1234u, 1) == 0xABCDu, "the warp's own, and no others");

// 16 lanes x 32 (or 16) columns over the warp: thread (g, t) = (lane / 4, lane % 4) gets columns 8 i + 2 t, + 1 of
// rows g (r[4 i], r[4 i + 1]) and g + 8 (r[4 i + 2], r[4 i + 3]).
__device__ __forceinline__ void tc_ld_rows(float (&s)[16], uint32_t addr) {
  uint32_t r[16];
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 "
               "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
               "tcgen05.wait::ld.sync.aligned;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                 "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]) : "r"(addr) : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) s[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tc_ld_rows(float (&s)[8], uint32_t addr) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]) : "r"(addr) : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = __uint_as_float(r[i]);
}

// The same, stored.
__device__ __forceinline__ void tc_st_rows(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.16x256b.x4.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};"
               ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
               "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr) : "memory");
}

// smem_desc with groups of eight rows (or keys) `group` bytes apart.
__device__ __forceinline__ uint64_t smem_desc_groups(uint32_t addr, uint32_t lead, uint32_t group) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(lead >> 4) << 16) |
         (static_cast<uint64_t>(group >> 4) << 32) | (uint64_t{1} << 46) | (uint64_t{2} << 61);
}

// Products D (TMEM) = or += A B (shared memory), by a whole, converged warp as tc_mma_ss: four whose operands' descriptors
// step by 2 (32 bytes), or two whose steps are given (in 16 bytes). The descriptors' low words alone change. One election for
// all, and no carries: a product then takes 31 clocks to issue, 40 each on its own.
#define KV_FIRST "{\n\t.reg .pred e, p;\n\t.reg .b64 x, y;\n\t.reg .b32 u, v;\n\telect.sync _|e, 0xFFFFFFFF;\n\tsetp.ne.b32 p, %6, 0;\n\t" \
  "mov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %4};\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, p;\n\t"
#define KV_NEXT(i, j) "add.u32 u, %1, " i ";\n\tadd.u32 v, %3, " j ";\n\tmov.b64 x, {u, %2};\n\tmov.b64 y, {v, %4};\n\t" \
  "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, 1;\n\t"
#define KV_OPERANDS "r"(d), "r"(static_cast<uint32_t>(a)), "r"(static_cast<uint32_t>(a >> 32)), "r"(static_cast<uint32_t>(b)), \
  "r"(static_cast<uint32_t>(b >> 32)), "r"(idesc), "r"(acc ? 1u : 0u)
__device__ __forceinline__ void tc_mma_chunk(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(KV_FIRST KV_NEXT("2", "2") KV_NEXT("4", "4") KV_NEXT("6", "6") "}" ::KV_OPERANDS : "memory");
}
__device__ __forceinline__ void tc_mma_two(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc, uint32_t a_step, uint32_t b_step) {
  asm volatile(KV_FIRST KV_NEXT("%7", "%8") "}" ::KV_OPERANDS, "r"(a_step), "r"(b_step) : "memory");
}
#undef KV_FIRST
#undef KV_NEXT
#undef KV_OPERANDS
// A in TMEM: its 64 dims are 32 columns.
__device__ __forceinline__ void tc_mma_chunk_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
#define KV_NEXT(i, j) "add.u32 u, %1, " i ";\n\tadd.u32 v, %2, " j ";\n\tmov.b64 y, {v, %3};\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [u], y, %4, 1;\n\t"
  asm volatile("{\n\t.reg .pred e, p;\n\t.reg .b64 y;\n\t.reg .b32 u, v;\n\telect.sync _|e, 0xFFFFFFFF;\n\tsetp.ne.b32 p, %5, 0;\n\t"
               "mov.b64 y, {%2, %3};\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t"
               KV_NEXT("8", "2") KV_NEXT("16", "4") KV_NEXT("24", "6") "}"
               ::"r"(d), "r"(a), "r"(static_cast<uint32_t>(b)), "r"(static_cast<uint32_t>(b >> 32)), "r"(idesc), "r"(acc ? 1u : 0u) : "memory");
#undef KV_NEXT
}

// A box of a cache of latent rows (latent_map), by one lane of a converged warp.
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t dim, int32_t group, int32_t page) {
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xFFFFFFFF;\n\t"
               "@e cp.async.bulk.tensor.5d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %6, %6, %4, %5}], [%2];\n\t}"
               ::"r"(dst), "l"(map), "r"(bar), "r"(dim), "r"(group), "r"(page), "r"(0) : "memory");
}

__device__ __forceinline__ float lg2_fast(float x) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Whether any of the 128 threads says so; a barrier of theirs.
__device__ __forceinline__ bool any_of_softmax(bool x) {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
               "barrier.cta.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(r) : "r"(x ? 1u : 0u) : "memory");
  return r != 0u;
}
__device__ __forceinline__ void sync_softmax() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }
// A row that overflowed, in full precision; a call, as it is seldom and the loops want the instruction cache.
template <int FMT>
__device__ __noinline__ void latent_row_again(const LatentParams& lp, int32_t b, int32_t pos, int32_t t, int32_t h, int32_t L) {
  attend_latent_row<FMT, 18>(lp, b, pos, t, h, 0, L);
}

template <int FMT, int NR, bool kBF16>
__global__ void __launch_bounds__(kLatThreads<FMT>, 1) kv_attend_latent_tile(const __grid_constant__ LatentTileParams p) {
  using S = LatentSmem<FMT, NR>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const LatentParams& lp = p.l;
  const AttendParams& a = lp.a;
  const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u;
  // (no static shared memory: the dynamic part begins at a multiple of 1,024, which the swizzle wants)
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem_raw));
  const int32_t HQ = static_cast<int32_t>(a.group.d);
  const uint32_t units = static_cast<uint32_t>(p.units), raws = static_cast<uint32_t>(p.raws);
  const uint32_t group_bytes = static_cast<uint32_t>(p.chunks) * 1024u, unit_bytes = 4u * group_bytes, raw_bytes = 2u * group_bytes;
  const uint32_t raw_ring = ring + units * unit_bytes;
  const uint32_t q_at = raw_ring + raws * raw_bytes;
  const uint32_t p_at = q_at + static_cast<uint32_t>(S::q_bytes(p.chunks));
  const uint32_t small = p_at + S::kP;
  uint8_t* const small_ptr = smem_raw + (small - ring);
  const uint32_t full = small + S::kOffBars, empty = full + 8 * kLatMaxUnits, raw_full = empty + 8 * kLatMaxUnits,
                 raw_empty = raw_full + 8 * kLatMaxRaws, q_full = raw_empty + 8 * kLatMaxRaws, s_full = q_full + 32,
                 s_free = s_full + 8 * kLatScores, p_full = s_free + 8 * kLatScores, pv_done = p_full + 16, seg_full = pv_done + 16,
                 seg_empty = seg_full + 16, done = seg_empty + 16;
  LatentSeg* const segs = reinterpret_cast<LatentSeg*>(small_ptr + S::kOffSegs);
  float* const sh_alpha = reinterpret_cast<float*>(small_ptr + S::kOffAlpha);   // [NR]
  float* const sh_inv = reinterpret_cast<float*>(small_ptr + S::kOffInv);
  float* const sh_qf = reinterpret_cast<float*>(small_ptr + S::kOffQf);
  float* const sh_top = reinterpret_cast<float*>(small_ptr + S::kOffTop);       // [64 / NR][NR]
  uint32_t* const sh_valid = reinterpret_cast<uint32_t*>(small_ptr + S::kOffValid);  // of a unit's keys, a bit each
  uint32_t* const sh_raw_valid = reinterpret_cast<uint32_t*>(small_ptr + S::kOffRawValid);
  float* const sh_scale = reinterpret_cast<float*>(small_ptr + S::kOffScale);        // [units][32], then [raws][32]
  float* const sh_log = sh_scale + (units + raws) * kLatKeys;                        // [units][32]: of the scales
  WaitState* const state = reinterpret_cast<WaitState*>(small_ptr + S::kOffMisc);
  uint32_t* const sh_tmem = reinterpret_cast<uint32_t*>(small_ptr + S::kOffMisc + 16);
  unsigned long long* const sh_bad = reinterpret_cast<unsigned long long*>(small_ptr + S::kOffMisc + 24);
  constexpr int kFillers = FMT == KV_CACHE_SRC ? 1 : kLatConverters;  // that arrive for a full unit

  if (warp == 4) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
        static_cast<uint32_t>(__cvta_generic_to_shared(sh_tmem))) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    for (uint32_t i = 0; i < units; ++i) {
      bar_init(full + 8 * i, kFillers);
      bar_init(empty + 8 * i, 1);
    }
    for (uint32_t i = 0; i < raws; ++i) {
      bar_init(raw_full + 8 * i, 33);
      bar_init(raw_empty + 8 * i, kLatConverters);
    }
    for (int i = 0; i < 4; ++i) bar_init(q_full + 8 * i, 4);
    for (int i = 0; i < kLatScores; ++i) {
      bar_init(s_full + 8 * i, 1);
      bar_init(s_free + 8 * i, 4);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(p_full + 8 * i, 4);
      bar_init(pv_done + 8 * i, 1);
      bar_init(seg_full + 8 * i, 1);
      bar_init(seg_empty + 8 * i, 8 + (FMT == KV_CACHE_SRC ? 0 : kLatConverters));
    }
    for (int i = 0; i < 3; ++i) bar_init(done + 8 * i, 1);
    *state = WaitState{(ring & 1023u) != 0u ? 1 : 0, 0};
    *sh_bad = 0ull;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *sh_tmem;
  bool ok = !state->ran_out();
  grid_handover();

  // A consumer's next segment; false after a wait that ran out. (By a whole warp.)
  auto take = [&](uint32_t k, LatentSeg* s) {
    ok = ok && __all_sync(0xFFFFFFFFu, bar_wait(seg_full + 8 * (k & 1u), (k >> 1) & 1u, state));
    if (!ok) return false;
    *s = segs[k & 1u];
    __syncwarp();
    if (lane == 0u) bar_arrive(seg_empty + 8 * (k & 1u));
    return s->stop == 0;
  };
  const uint32_t tm_s = tmem + 4 * NR;  // S, kLatScores buffers of kLatKeys columns, behind O^T; then Q
  const uint32_t tm_q = tm_s + kLatScores * kLatKeys;
  // a warp's place in the ring of units
  struct Place {
    uint32_t unit, phase;
  };
  auto next_unit = [&](Place* w) {
    if (++w->unit == units) {
      w->unit = 0u;
      w->phase ^= 1u;
    }
  };

  if constexpr (FMT != KV_CACHE_SRC) {  // 512 threads of 128 registers: the softmax takes more, the others leave them
    if (warp < 4) asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 112;");
  }
  if (warp < 4) {
    // ======================================================================================
    // the softmax
    // ======================================================================================
    const uint32_t g = lane >> 2, t = lane & 3u;
    // With 32 rows the other half of the 64 that a product has anyway are the same ones again: warps 2 and 3 take the last 16
    // keys of each tile.
    constexpr int kHalves = 64 / NR, kCols = kLatKeys / kHalves;  // keys of a warp
    const uint32_t half = NR == 64 ? 0u : warp >> 1;
    const int32_t r0 = static_cast<int32_t>(16u * (warp & (NR / 16 - 1u)) + g);  // and r0 + 8
    const bool first = t == 0u && half == 0u;  // that writes what a row has once
    const uint32_t lanes = warp << 21;
    const uint32_t flip = a.scale_log2 < 0.0f ? 0x80008000u : 0u;  // the maximum is taken before the scale
    constexpr float kSmall = kBF16 ? 0.0f : 7.0f;
    // The queries. (All products that read the last ones have ended, as their scores were waited for.) A power of two brings
    // bf16 ones over e4m3fn rows into fp16's range: the row's largest element to 2^13 .. 2^14.
    auto row_of = [&](const LatentSeg& s, int32_t r) {
      const int32_t x = s.row0 + min(r, s.last), qi = static_cast<int32_t>(a.group.quot(static_cast<uint32_t>(x)));
      return a.q + static_cast<int64_t>(s.q0 + qi) * a.q_token + static_cast<int64_t>(x - qi * HQ) * a.q_head;
    };
    uint32_t items = 0u;  // that have tiles
    auto load_q = [&](const LatentSeg& s) {
      // chunks in TMEM; chunks in flight (decode 145 us with one, 136.5 with three, 142.5 with nine; over e4m3fn 154 with one
      // or three)
      constexpr int kIn = S::kInTmem, kAt = FMT == KV_CACHE_SRC && NR == 32 ? 3 : 1;
      const bool shift = FMT != KV_CACHE_SRC && a.bf16;
      auto shifted = [](uint32_t z, float f) {
        const float2 v = widen2<true>(z);
        return pack2(v.x * f, v.y * f, false);
      };
      // thread (g, t): dims 16 i + 4 t .. + 3 of each chunk of rows g and g + 8
      const uint8_t* src[2] = {row_of(s, r0) + 8 * t, row_of(s, r0 + 8) + 8 * t};
      const bool live[2] = {r0 < s.nrows, r0 + 8 < s.nrows};
      auto piece = [&](int c, int chunk, int i) {
        uint2 w = make_uint2(0u, 0u);
        if (live[c] && 4 * chunk + i < p.ksteps) w = __ldg(reinterpret_cast<const uint2*>(src[c] + 128 * chunk + 32 * i));
        return w;
      };
      float f[2] = {1.0f, 1.0f};
      if (shift) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t m = 0u;
#pragma unroll 3
          for (int32_t chunk = 0; chunk < p.chunks; ++chunk)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint2 w = piece(c, chunk, i);
              m = absmax_pair<true>(absmax_pair<true>(m, w.x), w.y);
            }
          uint32_t e = __float_as_uint(absmax_pair_value<true>(m));
          e = max(e, __shfl_xor_sync(0xFFFFFFFFu, e, 1));
          e = max(e, __shfl_xor_sync(0xFFFFFFFFu, e, 2)) >> 23;
          f[c] = __uint_as_float(min(254u, 267u - e) << 23);
        }
      }
      if constexpr (FMT != KV_CACHE_SRC) {
        if (t == 0u) {
          sh_qf[r0] = f[0];
          sh_qf[r0 + 8] = f[1];
        }
      }
#pragma unroll 1
      for (int32_t c0 = 0; c0 < min(kIn, p.chunks); c0 += kAt) {
        uint2 w[kAt][2][4];
#pragma unroll
        for (int y = 0; y < kAt; ++y)
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) w[y][c][i] = piece(c, c0 + y, i);
#pragma unroll
        for (int y = 0; y < kAt; ++y) {
          if (c0 + y >= kIn) break;
          uint32_t r[16];
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const uint2 z = w[y][c][i];
              r[4 * i + 2 * c] = (shift ? shifted(z.x, f[c]) : z.x) ^ flip;
              r[4 * i + 2 * c + 1] = (shift ? shifted(z.y, f[c]) : z.y) ^ flip;
            }
          tc_st_rows(tm_q + 32 * (c0 + y) + lanes, r);
        }
      }
      tc_wait_st();
      if (kIn < kLatMaxChunks && p.chunks > kIn) {  // the last chunks to shared memory: a warp has NR / 4 rows, 16 bytes a lane
        constexpr int kRows = NR / 4;
        if (shift) sync_softmax();  // sh_qf
        const uint32_t rest = static_cast<uint32_t>(a.head_dim) / 8u - 8u * kIn;  // pieces, at most 32
        uint4 w[kRows];
#pragma unroll
        for (int y = 0; y < kRows; ++y) {
          const int32_t r = static_cast<int32_t>(warp) * kRows + y;
          w[y] = make_uint4(0u, 0u, 0u, 0u);
          if (r < s.nrows && lane < rest) w[y] = __ldg(reinterpret_cast<const uint4*>(row_of(s, r) + 128 * kIn + 16u * lane));
        }
#pragma unroll
        for (int y = 0; y < kRows; ++y) {
          const uint32_t r = warp * kRows + y;
          if (shift) {
            const float f = sh_qf[r];
            w[y] = make_uint4(shifted(w[y].x, f), shifted(w[y].y, f), shifted(w[y].z, f), shifted(w[y].w, f));
          }
          if (lane < rest)
            st_shared16(q_at + (lane >> 3) * (NR * 128u) + r * 128u + (((lane & 7u) ^ (r & 7u)) << 4), w[y].x ^ flip, w[y].y ^ flip, w[y].z ^ flip,
                        w[y].w ^ flip);
        }
        fence_async_shared();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0u) bar_arrive(q_full + 8 * (items++ & 3u));
    };
    uint32_t k = 0u, T = 0u;  // segments and tiles that went by
    Place at{0u, 0u}, buf{0u, 0u};  // of units, and of scores
    LatentSeg seg, next;
    bool have = take(k++, &seg);
    const bool lost = any_of_softmax(!ok);
    if (!lost && have && seg.t1 > seg.t0) load_q(seg);
    while (!lost && have) {
      const int32_t pos[2] = {seg.p_first + static_cast<int32_t>(a.group.quot(static_cast<uint32_t>(seg.row0 + min(r0, seg.last)))),
                              seg.p_first + static_cast<int32_t>(a.group.quot(static_cast<uint32_t>(seg.row0 + min(r0 + 8, seg.last))))};
      const int32_t p_lo = seg.p_first + static_cast<int32_t>(a.group.quot(static_cast<uint32_t>(seg.row0)));
      float rs[2], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        rs[c] = fabsf(a.scale_log2);
        if constexpr (FMT != KV_CACHE_SRC) rs[c] *= __fdiv_rn(1.0f, sh_qf[r0 + 8 * c]);
        if (rs[c] == 0.0f) rs[c] = __uint_as_float(1u);  // hidden scores (-inf) must stay -inf
      }
      // N tiles from j on; false: a wait ran out, and all leave together
      auto tiles = [&](auto count, int32_t j) {
        constexpr int N = decltype(count)::value;
        // The units are long there; their keys' bits and scales are read while S is waited for. (Threads that gave up a wait
        // go on to the barrier below.)
        uint32_t valid[N];
        [[maybe_unused]] float kf[N][kCols / 4], lv[N][kCols / 4];  // the keys' scales, and their binary logarithms
        float s[N][kCols / 2], alpha[2] = {1.0f, 1.0f};             // scores, factors of the rows' sums
#pragma unroll
        for (int x = 0; x < N; ++x) {
          ok = bar_wait(full + 8 * at.unit, at.phase, state) && ok;
          valid[x] = own_keys<kCols>(sh_valid[at.unit], half);
          if constexpr (FMT != KV_CACHE_SRC) {
#pragma unroll
            for (int i = 0; i < kCols / 8; ++i) {
              const uint32_t key = at.unit * kLatKeys + kCols * half + 8 * i + 2 * t;
              const float2 f = *reinterpret_cast<const float2*>(sh_scale + key), v = *reinterpret_cast<const float2*>(sh_log + key);
              kf[x][2 * i] = f.x;
              kf[x][2 * i + 1] = f.y;
              lv[x][2 * i] = v.x;
              lv[x][2 * i + 1] = v.y;
            }
          }
          next_unit(&at);
        }
#pragma unroll
        for (int x = 0; x < N; ++x) {
          ok = bar_wait(s_full + 8 * buf.unit, buf.phase, state) && ok;
          __syncwarp();
          tc_fence_after();
          tc_ld_rows(s[x], tm_s + kLatKeys * buf.unit + kCols * half + lanes);
          tc_fence_before();
          __syncwarp();
          if (lane == 0u) bar_arrive(s_free + 8 * buf.unit);
          if (++buf.unit == kLatScores) {
            buf.unit = 0u;
            buf.phase ^= 1u;
          }
        }
        float top[2] = {-INFINITY, -INFINITY};  // of the thread's own
#pragma unroll
        for (int x = 0; x < N; ++x) {
          if constexpr (FMT != KV_CACHE_SRC) {
#pragma unroll
            for (int i = 0; i < kCols / 2; ++i) s[x][i] *= kf[x][2 * (i / 4) + (i & 1)];
          }
          if ((j + x) * kLatKeys + kLatKeys - 1 > p_lo || valid[x] != ~0u >> (32 - kCols)) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int32_t n = pos[c] - ((j + x) * kLatKeys + kCols * static_cast<int32_t>(half)) + 1;  // the first n keys
              const uint32_t see = ((n >= kCols ? ~0u : n <= 0 ? 0u : (1u << n) - 1u) & valid[x]) >> (2 * t);
#pragma unroll
              for (int i = 0; i < kCols / 8; ++i)
#pragma unroll
                for (int y = 0; y < 2; ++y)
                  if ((see >> (8 * i + y) & 1u) == 0u) s[x][4 * i + 2 * c + y] = -INFINITY;
            }
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float z[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < kCols / 8; ++i)
#pragma unroll
              for (int y = 0; y < 2; ++y)
                z[y] = fmaxf(z[y], FMT == KV_CACHE_SRC ? s[x][4 * i + 2 * c + y] : __fmaf_rn(s[x][4 * i + 2 * c + y], rs[c], lv[x][2 * i + y]));
            top[c] = fmaxf(top[c], fmaxf(z[0], z[1]));
          }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) top[c] = FMT == KV_CACHE_SRC ? __fmaf_rn(top[c], rs[c], -kSmall) : top[c] - kSmall;
        // A maximum that grew little is kept (the weights stay below 2^(kSmall + 8)), so that a tile seldom asks for the
        // others' scores: the rows' new maxima, and O^T, which is all warps', are brought up to date when some row grew.
        auto grows = [&](int c) { return top[c] > m[c] + 8.0f || (m[c] == -INFINITY && top[c] > m[c]); };
        const bool renew = any_of_softmax(grows(0) || grows(1) || !ok), rescale = renew && j > seg.t0;
        if (renew) {
#pragma unroll
          for (int o = 1; o < 4; o <<= 1)
#pragma unroll
            for (int c = 0; c < 2; ++c) top[c] = fmaxf(top[c], __shfl_xor_sync(0xFFFFFFFFu, top[c], o));
          if constexpr (kHalves > 1) {
            if (t == 0u) {
              sh_top[NR * half + r0] = top[0];
              sh_top[NR * half + r0 + 8] = top[1];
            }
            sync_softmax();
#pragma unroll
            for (int c = 0; c < 2; ++c) top[c] = fmaxf(top[c], sh_top[NR * (half ^ 1u) + r0 + 8 * c]);
          }
#pragma unroll
          for (int c = 0; c < 2; ++c)
            if (grows(c)) {
              alpha[c] = exp2_fast(m[c] - top[c]);
              m[c] = top[c];
            }
          if (first) {
            sh_alpha[r0] = alpha[0];
            sh_alpha[r0 + 8] = alpha[1];
          }
          if (any_of_softmax(!ok)) return false;
        }
        uint32_t pw[N][kCols / 4];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float ref = m[c] == -INFINITY ? 0.0f : m[c];
          float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
          for (int x = 0; x < N; ++x)
#pragma unroll
            for (int i = 0; i < kCols / 8; ++i) {
              float2 z = make_float2(s[x][4 * i + 2 * c], s[x][4 * i + 2 * c + 1]);
              z = fma2(z, rs[c], -ref);
              float2 e = make_float2(exp2_fast(z.x), exp2_fast(z.y));
              sum[i & 1] = add2(sum[i & 1], e);
              if constexpr (FMT != KV_CACHE_SRC) {
                e.x *= kf[x][2 * i];
                e.y *= kf[x][2 * i + 1];
              }
              pw[x][2 * i + c] = pack2(e.x, e.y, kBF16);
            }
          sum[0] = add2(sum[0], sum[1]);
          l[c] = __fmaf_rn(l[c], alpha[c], sum[0].x + sum[0].y);
        }
        // tiles take turns in the halves of P's rows: P V of the last but one has read its
#pragma unroll
        for (int x = 0; x < N; ++x)
          if (T + x > 1u) ok = bar_wait(pv_done + 8 * ((T + x) & 1u), (((T + x) >> 1) - 1u) & 1u, state) && ok;
        if (rescale) {  // and that of the last one has written O^T
          ok = bar_wait(pv_done + 8 * ((T - 1u) & 1u), ((T - 1u) >> 1) & 1u, state) && ok;
          __syncwarp();
          tc_fence_after();
          for (int32_t b = 0; b < p.blocks; ++b)
#pragma unroll 1
            for (int c = 0; c < NR / 16; ++c) {
              uint32_t w[16];
              tc_ld16(w, tmem + lanes + b * NR + 16 * c);
#pragma unroll
              for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * sh_alpha[16 * c + i]);
              tc_st16(tmem + lanes + b * NR + 16 * c, w);
            }
          tc_wait_st();
        }
#pragma unroll
        for (int x = 0; x < N; ++x)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t r = static_cast<uint32_t>(r0 + 8 * c);
#pragma unroll
            for (int i = 0; i < kCols / 8; ++i)
              asm volatile("st.shared.u32 [%0], %1;" ::"r"(p_at + r * 128u + (((i + kCols / 8 * half + 4u * ((T + x) & 1u)) ^ (r & 7u)) << 4) + 4u * t),
                           "r"(pw[x][2 * i + c]) : "memory");
          }
        fence_async_shared();
        tc_fence_before();
        __syncwarp();
        if (lane < static_cast<uint32_t>(N)) bar_arrive(p_full + 8 * ((T + lane) & 1u));
        T += N;
        return true;
      };
      // Where the products are the longer two tiles go together, as what a step costs whatever its keys is a third of it: 64
      // rows over e4m3fn keys (24 heads, 200 - 777 tokens 435 us, 500 with one; but 48 heads, 2 - 5 tokens 236 and 187), or of
      // sequences with so many rows that their keys come from L2 (chunks 927 and 964 us). Else a tile does not wait for the
      // next: 48 heads, 2 - 5 tokens over 16-bit keys 164 us with two and 153 with one, 128 heads, one token 98 and 92.
      bool left = false;
      for (int32_t j = seg.t0; j < seg.t1 && !left;) {
        if (NR == 64 && (FMT != KV_CACHE_SRC || seg.nq * HQ > 4 * NR) && j + 1 < seg.t1) {
          left = !tiles(std::integral_constant<int, NR / 32>(), j);
          j += 2;
        } else {
          left = !tiles(std::integral_constant<int, 1>(), j);
          ++j;
        }
      }
      if (left) break;
      if (any_of_softmax(!ok)) break;
      have = take(k++, &next);
      if (any_of_softmax(!ok)) break;
      const bool live = seg.t1 > seg.t0;
      if (have && next.t1 > next.t0) load_q(next);
      // -- outputs ----------------------------------------------------------------------------
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        l[c] += __shfl_xor_sync(0xFFFFFFFFu, l[c], 1);
        l[c] += __shfl_xor_sync(0xFFFFFFFFu, l[c], 2);
      }
      if constexpr (kHalves > 1) {
        if (t == 0u && half != 0u) {
          sh_top[r0] = l[0];
          sh_top[r0 + 8] = l[1];
        }
        sync_softmax();
      }
      if (first) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if constexpr (kHalves > 1) l[c] += sh_top[r0 + 8 * c];
          sh_inv[r0 + 8 * c] = l[c] < INFINITY ? __fdiv_rn(1.0f, l[c]) : NAN;
        }
      }
      if (live) {
        ok = bar_wait(pv_done + 8 * ((T - 1u) & 1u), ((T - 1u) >> 1) & 1u, state) && ok;
        __syncwarp();
        tc_fence_after();
      }
      if (any_of_softmax(!ok)) break;
      const int32_t L = lp.latent;
      if (seg.part < 0) {
        // 32 dims of some rows at a time through shared memory (P's, which all products have read), so that four lanes write 64
        // bytes of a row
        constexpr int kOut = NR / 2;  // rows
        const uint32_t stage = p_at + warp * (kOut * 64u);
        unsigned long long bad = 0ull;
        for (int32_t b = 0; b < p.blocks; ++b) {
          const int32_t d0 = 128 * b + 32 * static_cast<int32_t>(warp);
          const bool mine = d0 + static_cast<int32_t>(lane) < L;
          for (int32_t r1 = 0; r1 < seg.nrows; r1 += kOut) {
#pragma unroll
            for (int c = 0; c < kOut / 16; ++c) {
              uint32_t w[16];
              if (live) {
                tc_ld16(w, tmem + lanes + b * NR + r1 + 16 * c);
              } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = 0u;
              }
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float v = live ? __uint_as_float(w[i]) * sh_inv[r1 + 16 * c + i] : 0.0f;
                if (mine && !(fabsf(v) < INFINITY)) bad |= 1ull << (r1 + 16 * c + i);
                asm volatile("st.shared.u16 [%0], %1;" ::"r"(stage + (16 * c + i) * 64u + 2u * lane), "h"(round16(v, a.bf16)) : "memory");
              }
            }
            __syncwarp();
            if (d0 + 8 * static_cast<int32_t>(lane & 3u) < L) {
#pragma unroll
              for (int y = 0; y < kOut / 8; ++y) {
                const int32_t r = r1 + 8 * y + static_cast<int32_t>(lane >> 2);
                if (r < seg.nrows) {
                  const int32_t qi = static_cast<int32_t>(a.group.quot(static_cast<uint32_t>(seg.row0 + r))), h = seg.row0 + r - qi * HQ;
                  *reinterpret_cast<uint4*>(a.out + static_cast<int64_t>(seg.q0 + qi) * a.o_token + static_cast<int64_t>(h) * a.o_head + 2 * d0 +
                                            16 * (lane & 3u)) = ld_shared16(stage + (8 * y + (lane >> 2)) * 64u + 16u * (lane & 3u));
                }
              }
            }
            __syncwarp();
          }
        }
        // (rows behind the last have no sums)
        if (seg.nrows < 64) bad &= (1ull << seg.nrows) - 1ull;
        const uint32_t lo = __reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(bad)), hi = __reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(bad >> 32));
        if (lane == 0u && (lo | hi) != 0u) atomicOr(sh_bad, static_cast<unsigned long long>(hi) << 32 | lo);
        sync_softmax();
        unsigned long long again = *const_cast<volatile unsigned long long*>(sh_bad);
        if (a.lse && first) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int32_t r = r0 + 8 * c;
            if (r < seg.nrows && (again >> r & 1ull) == 0ull) {
              const int32_t qi = static_cast<int32_t>(a.group.quot(static_cast<uint32_t>(seg.row0 + r))), h = seg.row0 + r - qi * HQ;
              a.lse[static_cast<int64_t>(seg.q0 + qi) * HQ + h] = live ? (m[c] + log2f(l[c])) * 0.6931471805599453f : -INFINITY;
            }
          }
        }
        if (again != 0ull) {
          if (lane == 0u) state->hold(1);
          __syncwarp();
          for (int32_t r = static_cast<int32_t>(warp); r < seg.nrows; r += 4) {
            if ((again >> r & 1ull) == 0ull) continue;
            const int32_t qi = static_cast<int32_t>(a.group.quot(static_cast<uint32_t>(seg.row0 + r))), h = seg.row0 + r - qi * HQ;
            latent_row_again<FMT>(lp, seg.b, seg.p_first + qi, seg.q0 + qi, h, L);
          }
          if (lane == 0u) state->hold(-1);
          sync_softmax();
          if (tid == 0u) *sh_bad = 0ull;
        }
      } else {
        const int64_t at = static_cast<int64_t>(seg.part) * p.part_rows;
        const int32_t width = 128 * p.blocks;
        for (int32_t c = 0; 32 * c < seg.nrows; ++c) {
          float* const to = p.part_o + (at + 32 * c) * width + tid;
          for (int32_t b = 0; b < p.blocks; ++b) {
            uint32_t w[32];
            if (live) {
              tc_ld32(w, tmem + lanes + b * NR + 32 * c);
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) w[i] = 0u;
            }
            float* row = to + 128 * b;
            const int32_t rows = seg.nrows - 32 * c;
#pragma unroll
            for (int i = 0; i < 32; ++i, row += width)
              if (i < rows) *row = __uint_as_float(w[i]);
          }
        }
        if (first) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
            if (r0 + 8 * c < seg.nrows) *reinterpret_cast<float2*>(p.part_ml + (at + r0 + 8 * c) * 2) = make_float2(m[c], l[c]);
        }
      }
      tc_fence_before();
      seg = next;
    }
  } else if (warp == 4 || warp == 5 || warp == 8) {
    // ======================================================================================
    // the products: warps 4 and 8 S = Q K^T, of every other tile each, warp 5 O^T += V^T P^T
    // ======================================================================================
    auto wait = [&](uint32_t bar, uint32_t parity) {
      if (ok) ok = __all_sync(0xFFFFFFFFu, bar_wait(bar, parity, state));
      tc_fence_after();
    };
    // Descriptors and addresses are to be in uniform registers: a reduction's result is in one, loops end by the
    // parameters alone, and products stand in straight lines. (With descriptors in any register a product took 70 to 140
    // clocks to issue.)
    auto same = [](uint32_t x) { return __reduce_or_sync(0xFFFFFFFFu, x); };
    const uint32_t ring0 = same(ring);
    constexpr uint32_t kType = (1u << 4) | (kBF16 ? 1u << 7 | 1u << 10 : 0u);
    uint32_t k = 0u, T = 0u;
    Place at{0u, 0u};
    LatentSeg seg;
    if (warp != 5) {
      constexpr uint32_t kDesc = kType | ((static_cast<uint32_t>(kLatKeys) >> 3) << 17) | ((64u >> 4) << 24);
      const uint32_t turn = warp >> 3;  // tiles with this parity are the warp's
      const uint32_t s_at = same(tm_s), q_col = same(tm_q);
      const uint64_t q_desc = smem_desc(same(q_at), 16);  // of the chunks that are not in TMEM
      uint32_t items = 0u;
      while (take(k++, &seg)) {
        if (seg.t1 <= seg.t0) continue;
        // (four barriers in turn: a warp without a tile of an item can be late, but not by more items than the queue of
        // segments holds, so that no phase passes it by)
        wait(q_full + 8 * (items & 3u), (items >> 2) & 1u);
        ++items;
        for (int32_t j = seg.t0; j < seg.t1; ++j, ++T) {
          if ((T & 1u) == turn) {
            const uint32_t u = same(at.unit | (T % kLatScores) << 8), un = u & 255u, buf = u >> 8, d = s_at + kLatKeys * buf;
            const uint64_t kd = smem_desc_groups(ring0 + un * unit_bytes, 16, group_bytes);
            if (T >= kLatScores) wait(s_free + 8 * (T % kLatScores), (T / kLatScores - 1u) & 1u);
            wait(full + 8 * at.unit, at.phase);
            if (!ok) break;
            auto chunk = [&](int32_t c) {
              if (c < S::kInTmem) tc_mma_chunk_ts(d, q_col + 32 * c, kd + c * (1024 >> 4), kDesc, c > 0);
              else tc_mma_chunk(d, q_desc + (c - S::kInTmem) * (NR * 128 >> 4), kd + c * (1024 >> 4), kDesc, c > 0);
            };
            auto rest = [&] {
#pragma unroll 1
              for (int32_t i = p.ksteps & ~3; i < p.ksteps; ++i) {
                const uint64_t b = kd + ((i / 4) * (1024 >> 4) + (i % 4) * 2);
                if (i < 4 * S::kInTmem) tc_mma_ts(d, q_col + 8 * i, b, kDesc, i > 0);
                else tc_mma_ss(d, q_desc + ((i / 4 - S::kInTmem) * (NR * 128 >> 4) + (i % 4) * 2), b, kDesc, true);
              }
            };
            if constexpr (FMT == KV_CACHE_SRC) {
#pragma unroll
              for (int c = 0; c < kLatMaxChunks; c += 3) {
                if (p.ksteps >= 4 * c + 12) {
                  chunk(c); chunk(c + 1); chunk(c + 2);
                } else {
#pragma unroll 1
                  for (int32_t y = c; 4 * y + 4 <= p.ksteps; ++y) chunk(y);
                  rest();
                  break;
                }
              }
            } else {  // loops: beside the converters' code straight lines do not stay in the instruction cache (chunks 516 us, 435 with loops)
              const int32_t whole = p.ksteps >> 2, ts = min(whole, S::kInTmem);
#pragma unroll 1
              for (int32_t c = 0; c < ts; ++c) tc_mma_chunk_ts(d, q_col + 32 * c, kd + c * (1024 >> 4), kDesc, c > 0);
              if constexpr (S::kInTmem < kLatMaxChunks) {
#pragma unroll 1
                for (int32_t c = S::kInTmem; c < whole; ++c) chunk(c);
              }
              rest();
            }
            tc_commit(s_full + 8 * buf);
          }
          next_unit(&at);
        }
        if (!ok) break;
      }
    } else {
      constexpr uint32_t kDesc = kType | (1u << 15) | ((static_cast<uint32_t>(NR) >> 3) << 17) | ((128u >> 4) << 24);
      const uint32_t o_at = same(tmem), free0 = same(empty), step = same(group_bytes >> 3);  // 16 keys, in 16 bytes
      const uint64_t p_desc = smem_desc(same(p_at), 16);
      while (take(k++, &seg)) {
        for (int32_t j = seg.t0; j < seg.t1; ++j, ++T) {
          const uint32_t u = same(at.unit | (T & 1u) << 8 | (j > seg.t0 ? 1u << 16 : 0u)), un = u & 255u, odd = (u >> 8) & 1u;
          wait(full + 8 * at.unit, at.phase);
          wait(p_full + 8 * (T & 1u), (T >> 1) & 1u);
          if (!ok) break;
          const uint64_t v = smem_desc_groups(ring0 + un * unit_bytes, 1024, group_bytes), pd = p_desc + 4 * odd;
          auto block = [&](int32_t b) { tc_mma_two(o_at + b * NR, v + b * (2048 >> 4), pd, kDesc, (u >> 16) != 0u, step, 2u); };
          if (FMT == KV_CACHE_SRC && p.blocks == 4) {
            block(0); block(1); block(2); block(3);
          } else {
#pragma unroll 1
            for (int32_t b = 0; b < p.blocks; ++b) block(b);
          }
          tc_commit(free0 + 8 * un);
          tc_commit(pv_done + 8 * odd);
          next_unit(&at);
        }
        if (!ok) break;
      }
    }
    if (!ok) {  // products still in flight read shared memory and write TMEM: let them end
      const uint32_t bar = done + 8 * (warp == 8 ? 2u : warp - 4u);
      tc_commit(bar);
      for (uint32_t i = 0; i < kSpin && !bar_try(bar, 0); ++i) {}
    }
    __syncwarp();
  } else if (warp == 6) {
    // ======================================================================================
    // the work, item by item
    // ======================================================================================
    // total units, and (for the join) each sequence's first
    int64_t total = 0;
    for (int32_t b0 = 0; b0 < a.num_seqs; b0 += 32) {
      const int32_t b = b0 + static_cast<int32_t>(lane);
      const int64_t u = b < a.num_seqs ? latent_units<NR>(p, b, blockIdx.x == 0) : 0;
      int64_t incl = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= static_cast<uint32_t>(o)) incl += v;
      }
      if (p.split && blockIdx.x == 0 && b < a.num_seqs) p.meta[b] = total + incl - u;
      total += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
    ShareLevel level = {};
    int32_t shares = 0;
    const int32_t ctas = static_cast<int32_t>(gridDim.x), cta = static_cast<int32_t>(blockIdx.x);
    if (p.split) {
      level = latent_cut(total, ctas, &shares);
      if (blockIdx.x == 0 && lane == 0u) {
        p.head->level[0] = level;
        p.head->levels = 1;
      }
    }
    // the cursor: sequences cur_b .. cur_b + 31, whose first unit is cur_at; a lane has its sequence's units
    int32_t cur_b = -32;
    int64_t cur_at = 0, cur_n = 0, mine_at = 0, mine_n = 0;
    uint32_t k = 0u;
    auto publish = [&](const LatentSeg& s) {
      if (k >= 2u) ok = ok && __all_sync(0xFFFFFFFFu, bar_wait(seg_empty + 8 * (k & 1u), ((k >> 1) - 1u) & 1u, state));
      if (!ok) return;
      if (lane == 0u) {
        segs[k & 1u] = s;
        bar_arrive(seg_full + 8 * (k & 1u));
      }
      __syncwarp();
      ++k;
    };
    int32_t round = 0;
    int32_t share = cta;
    while (ok) {
      int64_t pos, end;
      if (p.split) {
        if (share >= shares) break;
        pos = static_cast<int64_t>(share) * level.size;
        end = min(total, pos + level.size);
      } else {  // items in turn, every second round the other way
        pos = static_cast<int64_t>(round) * ctas + ((round & 1) ? ctas - 1 - cta : cta);
        end = pos + 1;
        ++round;
        if (pos >= total) {
          if (static_cast<int64_t>(round) * ctas >= total) break;
          continue;
        }
      }
      while (ok && pos < end) {
        while (pos >= cur_at + cur_n) {  // (pos < total: some sequence has it)
          cur_at += cur_n;
          cur_b += 32;
          const int32_t b = cur_b + static_cast<int32_t>(lane);
          mine_n = b < a.num_seqs ? latent_units<NR>(p, b, false) : 0;
          int64_t incl = mine_n;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= static_cast<uint32_t>(o)) incl += v;
          }
          mine_at = cur_at + incl - mine_n;
          cur_n = __shfl_sync(0xFFFFFFFFu, incl, 31);
        }
        const int src = __ffs(static_cast<int>(__ballot_sync(0xFFFFFFFFu, pos >= mine_at && pos < mine_at + mine_n))) - 1;
        const int64_t local = pos - __shfl_sync(0xFFFFFFFFu, mine_at, src);
        LatentSeg s = {};
        s.b = cur_b + src;
        const AttendSeq seq = attend_seq(a, s.b, false);
        const LatentGeom geom = latent_geom<NR>(p, seq);
        const int32_t unit = p.split ? geom.steps : 1;
        int32_t item = static_cast<int32_t>(quotient(local, unit));
        const int32_t s_in = static_cast<int32_t>(local - static_cast<int64_t>(item) * unit);
        const int32_t s_out = static_cast<int32_t>(min(static_cast<int64_t>(unit), s_in + (end - pos)));
        pos += s_out - s_in;
        if (!p.split) item = geom.blocks - 1 - item;  // the last queries, which see the most keys, first
        s.q0 = seq.q0;
        s.nq = seq.nq;
        s.p_first = seq.len - seq.nq;
        const int32_t rows = seq.nq * HQ, first = item * NR;
        s.row0 = first;
        s.nrows = min(NR, rows - first);
        s.last = s.nrows - 1;
        s.p_hi = s.p_first + static_cast<int32_t>(a.group.quot(static_cast<uint32_t>(first + s.last)));
        const int32_t tiles = s.p_hi < 0 ? 0 : s.p_hi / kLatKeys + 1;
        s.t0 = p.split ? min(max(s_in - kLatItemSteps, 0), tiles) : 0;
        s.t1 = p.split ? min(max(s_out - kLatItemSteps, 0), tiles) : tiles;
        s.part = s_out - s_in == unit ? -1 : 2 * share + (s_in == 0 ? 1 : 0);
        publish(s);
        // its queries into L2: they are wanted when the item before ends (32 heads, one token 138.8 us without, 136.5 with; over
        // e4m3fn 157.5 and 154.3; chunks 925 and 927, but 966 where the compiler leaves it out of the 64-row form)
        if (s.t1 > s.t0) {
          const int32_t lines = (a.head_dim * 2 + 127) / 128;
          for (int32_t i = static_cast<int32_t>(lane); i < s.nrows * lines; i += 32) {
            const int32_t r = i / lines, qi = static_cast<int32_t>(a.group.quot(static_cast<uint32_t>(s.row0 + r)));
            prefetch_l2_line(a.q + static_cast<int64_t>(s.q0 + qi) * a.q_token + static_cast<int64_t>(s.row0 + r - qi * HQ) * a.q_head +
                             min(128 * (i - r * lines), a.head_dim * 2 - 1));
          }
        }
      }
      share += ctas;
    }
    LatentSeg s = {};
    s.stop = 1;
    publish(s);
  } else if (warp == 7) {
    // ======================================================================================
    // the keys, a unit of 32 at a time
    // ======================================================================================
    uint32_t k = 0u, n = 0u;  // units that went by
    Place at{0u, 0u};         // in the ring of units, or of raw ones
    const uint32_t places = FMT == KV_CACHE_SRC ? units : raws;
    const uint32_t full_at = FMT == KV_CACHE_SRC ? full : raw_full, empty_at = FMT == KV_CACHE_SRC ? empty : raw_empty;
    const uint32_t pieces = static_cast<uint32_t>(a.head_dim) / (FMT == KV_CACHE_SRC ? 8u : 16u);  // 16-byte pieces of a row
    LatentSeg seg;
    // 16-bit units that were copied by cp.async, and not yet handed over: the copies land while the next ones are issued
    uint32_t pending[2] = {0u, 0u}, waiting = 0u;
    auto hand_over = [&](bool all) {
      if constexpr (FMT == KV_CACHE_SRC) {
        while (waiting > (all ? 0u : 1u)) {
          if (waiting == 2u) wait_async<1>(); else wait_async<0>();
          fence_async_shared();
          __syncwarp();
          if (lane == 0u) bar_arrive(full + 8 * pending[0]);
          pending[0] = pending[1];
          --waiting;
        }
      }
    };
    while (take(k++, &seg)) {
      const int32_t* table = a.table + static_cast<int64_t>(seg.b) * a.table_stride;
      const int32_t n0 = seg.t0, n1 = seg.t1;
      // 32 entries of the table, a lane each, from entry e0 on, and where the next 32 are needed them
      const int32_t e_last = static_cast<int32_t>(a.page.quot(static_cast<uint32_t>(max(seg.p_hi, 0))));
      auto entries = [&](int32_t e) { return __ldg(table + min(e + static_cast<int32_t>(lane), e_last)); };
      int32_t e0 = static_cast<int32_t>(a.page.quot(static_cast<uint32_t>(n0 * kLatKeys))), ids = 0, ahead = 0;
      if (n0 < n1) {
        ids = entries(e0);
        ahead = entries(e0 + 32);
      }
      for (int32_t unit = n0; unit < n1 && ok; ++unit, ++n) {
        const int32_t key = unit * kLatKeys + static_cast<int32_t>(lane);
        // lane = key: its page (of the last key that a row sees, for keys behind it)
        const int32_t e = static_cast<int32_t>(a.page.quot(static_cast<uint32_t>(min(key, seg.p_hi))));
        int32_t id = __shfl_sync(0xFFFFFFFFu, ids, e - e0);
        if (__shfl_sync(0xFFFFFFFFu, e, 31) >= e0 + 32) {  // (at most 32 entries a unit: these and the next)
          const int32_t other = __shfl_sync(0xFFFFFFFFu, ahead, e - e0 - 32);
          if (e >= e0 + 32) id = other;
          e0 += 32;
          ids = ahead;
          ahead = entries(e0 + 32);
        }
        const bool want = key <= seg.p_hi, have = static_cast<uint32_t>(id) < static_cast<uint32_t>(a.num_pages), live = want && have;
        if (want && !have) record_oob(a.err, static_cast<uint64_t>(seg.b));
        const uint32_t bits = __ballot_sync(0xFFFFFFFFu, live);
        const uint32_t off = static_cast<uint32_t>(key) - a.page.quot(static_cast<uint32_t>(key)) * a.page.d;
        // boxes of `box` groups of eight keys, which share a page
        const bool boxes = p.box > 0 && bits == ~0u;
        const int32_t page0 = __shfl_sync(0xFFFFFFFFu, id, 0), in0 = static_cast<int32_t>(__shfl_sync(0xFFFFFFFFu, off, 0) >> 3);
        const uint32_t bar = full_at + 8 * at.unit, part = FMT == KV_CACHE_SRC ? group_bytes : group_bytes / 2u;  // of eight keys
        const uint32_t dst = FMT == KV_CACHE_SRC ? ring + at.unit * unit_bytes : raw_ring + at.unit * raw_bytes;
        // (nothing that can be known before stands between a free unit and its boxes)
        if (n >= places) {
          if (waiting > 0u && !__all_sync(0xFFFFFFFFu, bar_try(empty_at + 8 * at.unit, at.phase ^ 1u))) hand_over(true);
          ok = __all_sync(0xFFFFFFFFu, bar_wait(empty_at + 8 * at.unit, at.phase ^ 1u, state));
          if (!ok) break;
          if constexpr (FMT != KV_CACHE_SRC) fence_async_shared();  // generic loads, and then boxes
        }
        if (boxes) {
          if constexpr (FMT == KV_CACHE_SRC) {
            if (waiting > 0u) hand_over(true);
          }
          if (p.box == 4 && p.box_chunks == p.chunks) {
            tma_rows(dst, &p.map, bar, 0, in0, page0);
          } else {
            for (int32_t g = 0; g < 4; g += p.box) {
              const int32_t page = __shfl_sync(0xFFFFFFFFu, id, 8 * g), in_page = static_cast<int32_t>(__shfl_sync(0xFFFFFFFFu, off, 8 * g) >> 3);
              for (int32_t c = 0; c < p.chunks; c += p.box_chunks)
                tma_rows(dst + g * part + c * (part / static_cast<uint32_t>(p.chunks)), &p.map, bar, 64 * c, in_page, page);
            }
          }
          if (lane == 0u) {
            (FMT == KV_CACHE_SRC ? sh_valid : sh_raw_valid)[at.unit] = bits;
            bar_arrive_expect(bar, 4u * part);  // (boxes that land before are counted already)
          }
        } else if (lane == 0u) {
          (FMT == KV_CACHE_SRC ? sh_valid : sh_raw_valid)[at.unit] = bits;
        }
        if constexpr (FMT != KV_CACHE_SRC)
          copy_async<4>(static_cast<uint32_t>(__cvta_generic_to_shared(sh_scale + (units + at.unit) * kLatKeys + lane)),
                        reinterpret_cast<const uint8_t*>(live ? lp.scales + (static_cast<int64_t>(id) * a.page.d + off) * lp.scale_slot : lp.scales),
                        live ? 4u : 0u);
        if (!boxes) {
          const int64_t row = live ? wide(id, p.page_stride) + wide(off, p.slot_stride) : -1;
          // pieces in turn, so that lanes copy neighbouring ones
          for (uint32_t i0 = 0; i0 < kLatKeys * pieces; i0 += 32u) {
            const uint32_t i = i0 + lane, kk = i / pieces, piece = i - kk * pieces;
            const int64_t r = __shfl_sync(0xFFFFFFFFu, row, kk);
            const uint32_t base = dst + (kk >> 3) * part;
            const uint32_t to = FMT == KV_CACHE_SRC ? base + (piece >> 3) * 1024u + (kk & 7u) * 128u + (((piece & 7u) ^ (kk & 7u)) << 4)
                                                    : base + (piece >> 2) * 512u + (kk & 7u) * 64u + ((piece & 3u) << 4);
            copy_async<16>(to, a.k + (r < 0 ? 0 : r + 16 * piece), r < 0 ? 0u : 16u);
          }
        }
        if constexpr (FMT == KV_CACHE_SRC) {
          if (!boxes) {
            commit_async();
            pending[waiting++] = at.unit;
            hand_over(false);
          }
        } else {
          bar_arrive_copies(bar);  // the scales, and rows
          if (!boxes && lane == 0u) bar_arrive(bar);
        }
        if (++at.unit == places) {
          at.unit = 0u;
          at.phase ^= 1u;
        }
      }
      hand_over(true);
      if (!ok) break;
    }
    wait_all_async();
    if (!ok)  // boxes in flight write shared memory: let them land before the CTA leaves it
      for (int i = 0; i < 1000; ++i) __nanosleep(1000);
  } else if constexpr (FMT != KV_CACHE_SRC) {
    // ======================================================================================
    // e4m3fn rows to fp16: a warp takes eight keys of a chunk at a time, 16 codes a lane
    // ======================================================================================
    const uint32_t w = warp - 9u, jobs = 4u * static_cast<uint32_t>(p.chunks);
    const uint32_t row = lane >> 2, q = lane & 3u;
    uint32_t k = 0u, n = 0u;
    Place at{0u, 0u}, from{0u, 0u};
    LatentSeg seg;
    while (take(k++, &seg)) {
      for (int32_t unit = seg.t0; unit < seg.t1; ++unit, ++n) {
        ok = __all_sync(0xFFFFFFFFu, bar_wait(raw_full + 8 * from.unit, from.phase, state));
        if (!ok) break;
        const uint32_t src = raw_ring + from.unit * raw_bytes;
        float scale = 0.0f;
        uint32_t bits = 0u;
        if (w == 0u) {
          scale = sh_scale[(units + from.unit) * kLatKeys + lane];
          bits = sh_raw_valid[from.unit];
        }
        if (n >= units) ok = __all_sync(0xFFFFFFFFu, bar_wait(empty + 8 * at.unit, at.phase ^ 1u, state));
        if (!ok) break;
        const uint32_t dst = ring + at.unit * unit_bytes;
#pragma unroll 1
        for (uint32_t i0 = w; i0 < jobs; i0 += 2u * kLatConverters) {
          uint4 v[2];
#pragma unroll
          for (uint32_t i = 0; i < 2u; ++i)
            if (i0 + kLatConverters * i < jobs) v[i] = ld_shared16(src + (i0 + kLatConverters * i) * 512u + lane * 16u);
#pragma unroll
          for (uint32_t i = 0; i < 2u; ++i) {
            if (i0 + kLatConverters * i < jobs) {
              const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
              uint32_t f[8];
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                f[2 * y] = f16x2_from_e4m3x2(x[y]);
                f[2 * y + 1] = f16x2_from_e4m3x2(x[y] >> 16);
              }
              const uint32_t to = dst + (i0 + kLatConverters * i) * 1024u + row * 128u;
              st_shared16(to + (((2u * q) ^ row) << 4), f[0], f[1], f[2], f[3]);
              st_shared16(to + (((2u * q + 1u) ^ row) << 4), f[4], f[5], f[6], f[7]);
            }
          }
        }
        __syncwarp();
        if (lane == 0u) bar_arrive(raw_empty + 8 * from.unit);
        if (++from.unit == raws) {
          from.unit = 0u;
          from.phase ^= 1u;
        }
        if (w == 0u) {
          sh_scale[at.unit * kLatKeys + lane] = scale;
          sh_log[at.unit * kLatKeys + lane] = fmaxf(lg2_fast(fabsf(scale)), -100.0f);
          if (lane == 0u) sh_valid[at.unit] = bits;
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0u) bar_arrive(full + 8 * at.unit);
        next_unit(&at);
      }
      if (!ok) break;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && state->ran_out()) {
    record_wait(a.err);
    if (p.split) p.head->gave_up = 1u;
  }
  if (warp == 4) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

constexpr int kLatJoinWarps = 16;

// Joins the parts of the items that were split, in the order of their keys: `wpr` warps of the CTA take
// 128 dims of one row.
template <int FMT, int NR>
__global__ void __launch_bounds__(32 * kLatJoinWarps) kv_attend_latent_join(const __grid_constant__ LatentTileParams p, const int32_t wpr) {
  __shared__ float4 sh_o[kLatJoinWarps][32];
  __shared__ float2 sh_ml[kLatJoinWarps];
  const LatentParams& lp = p.l;
  const AttendParams& a = lp.a;
  const uint32_t lane = threadIdx.x & 31u;
  const int32_t warp = static_cast<int32_t>(threadIdx.x >> 5), part = warp % wpr;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kLatJoinWarps / wpr) + warp / wpr;
  const int64_t row_of = unit / p.blocks;
  const int32_t block = static_cast<int32_t>(unit - row_of * p.blocks);
  const int32_t tok = static_cast<int32_t>(row_of / a.q_heads), h = static_cast<int32_t>(row_of - static_cast<int64_t>(tok) * a.q_heads);
  grid_handover();
  int32_t b = tok, c0 = 0, c1 = 0, r = 0, pos = 0;
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
      const LatentGeom geom = latent_geom<NR>(p, s);
      const int32_t row = (tok - s.q0) * a.q_heads + h, rb = row / NR;
      r = row % NR;
      pos = s.len - s.nq + (tok - s.q0);
      const int64_t s0 = p.meta[b] + static_cast<int64_t>(rb) * geom.steps;
      c0 = share_of(p.head, s0);
      c1 = share_of(p.head, s0 + geom.steps - 1);
      joined = c0 != c1;
      lost = p.head->gave_up != 0u;
    }
  }
  const int32_t width = 128 * p.blocks;
  float mm = -INFINITY, ll = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto merge = [&](float2 ml, float4 v) {
    const float mn = fmaxf(mm, ml.x), ref = mn == -INFINITY ? 0.0f : mn;
    const float ea = exp2_fast(mm - ref), eb = exp2_fast(ml.x - ref);
    mm = mn;
    ll = __fmaf_rn(ll, ea, ml.y * eb);
    acc.x = __fmaf_rn(acc.x, ea, v.x * eb);
    acc.y = __fmaf_rn(acc.y, ea, v.y * eb);
    acc.z = __fmaf_rn(acc.z, ea, v.z * eb);
    acc.w = __fmaf_rn(acc.w, ea, v.w * eb);
  };
  if (joined) {
    for (int32_t c = c0 + part; c <= c1; c += 4 * wpr) {
      float2 ml[4];
      float4 v[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int32_t cc = c + x * wpr;
        ml[x] = make_float2(-INFINITY, 0.0f);
        v[x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (cc <= c1) {
          const int64_t at = static_cast<int64_t>(2 * cc + (cc == c0 ? 1 : 0)) * p.part_rows + r;
          ml[x] = __ldcg(reinterpret_cast<const float2*>(p.part_ml + at * 2));
          v[x] = __ldcg(reinterpret_cast<const float4*>(p.part_o + at * width + 128 * block) + lane);
        }
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) merge(ml[x], v[x]);
    }
  }
  if (wpr > 1) {
    sh_o[warp][lane] = acc;
    if (lane == 0u) sh_ml[warp] = make_float2(mm, ll);
    __syncthreads();
    if (part != 0) return;
    for (int32_t w = warp + 1; w < warp + wpr; ++w) merge(sh_ml[w], sh_o[w][lane]);
  }
  const int32_t d = 128 * block + 4 * static_cast<int32_t>(lane);
  uint16_t* out = reinterpret_cast<uint16_t*>(a.out + tok * a.o_token + h * a.o_head);
  const bool lse = a.lse && block == 0 && lane == 0u;
  if (lost) {  // parts are missing, or whole rows: NaN, whatever was computed
    for (int i = 0; i < 4; ++i)
      if (d + i < lp.latent) out[d + i] = 0x7FFFu;
    if (lse) a.lse[static_cast<int64_t>(tok) * a.q_heads + h] = __uint_as_float(0x7FFFFFFFu);
    return;
  }
  if (!joined) return;
  const float inv = ll < INFINITY ? __fdiv_rn(1.0f, ll) : NAN;
  const float v[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
  bool fine = true;
#pragma unroll
  for (int i = 0; i < 4; ++i) fine = fine && (d + i >= lp.latent || fabsf(v[i]) < INFINITY);
  if (!__all_sync(0xFFFFFFFFu, fine)) {  // its dims alone: the row's others are other warps'
    attend_latent_row<FMT, 18>(lp, b, pos, tok, h, 128 * block, min(128 * block + 128, lp.latent));
    return;
  }
  if (d < lp.latent) *reinterpret_cast<uint2*>(out + d) = make_uint2(pack2(v[0], v[1], a.bf16), pack2(v[2], v[3], a.bf16));
  if (lse) a.lse[static_cast<int64_t>(tok) * a.q_heads + h] = (mm + log2f(ll)) * 0.6931471805599453f;
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------

template <int FMT, int NR, bool kBF16>
kv_status launch_latent_tile(LatentTileParams p, void* work, int64_t work_bytes, int64_t max_keys, cudaStream_t stream) {
  using S = LatentSmem<FMT, NR>;
  const AttendParams& a = p.l.a;
  auto* kernel = kv_attend_latent_tile<FMT, NR, kBF16>;
  constexpr int kMost = 227 * 1024;
  static SmemOptIn opt_in;
  kv_status st = opt_in(reinterpret_cast<const void*>(kernel), kMost);
  if (st != KV_OK) return st;
  int sms = 0;
  st = current_sm_count(&sms);
  if (st != KV_OK) return st;
  p.units = 3;
  if (FMT == KV_CACHE_SRC) {
    while (p.units < kLatMaxUnits && S::total(p.chunks, p.units + 1, 0) <= kMost) ++p.units;
  } else {
    p.raws = 2;
    if (S::total(p.chunks, 4, 4) <= kMost) p.units = 4;
    while (p.raws < 4 && S::total(p.chunks, p.units, p.raws + 1) <= kMost) ++p.raws;
    while (p.units < kLatMaxUnits && S::total(p.chunks, p.units + 1, p.raws) <= kMost) ++p.units;
    while (p.raws < kLatMaxRaws && S::total(p.chunks, p.units, p.raws + 1) <= kMost) ++p.raws;
  }
  const int smem = S::total(p.chunks, p.units, p.raws);
  const int64_t ctas = sms;
  const int64_t items = static_cast<int64_t>(a.num_q) * a.group.d / NR + a.num_seqs;  // at most
  const int64_t meta = (static_cast<int64_t>(a.num_seqs) + 31) / 32 * 256;
  p.part_rows = a.q_start || static_cast<int32_t>(a.group.d) > NR ? NR : static_cast<int32_t>(a.group.d);
  const int64_t slot = static_cast<int64_t>(p.part_rows) * (128 * p.blocks + 2) * 4;
  int64_t fit = work && work_bytes > kSplitHead + meta ? (work_bytes - kSplitHead - meta) / (2 * slot) : 0;
  if (fit > ctas) fit = ctas;
  p.split = items < 4 * ctas && max_keys > 8 * kLatKeys && 2 * fit >= ctas;
  int64_t grid = items < ctas ? items : ctas;
  if (p.split) {
    grid = fit < ctas ? fit : ctas;
    p.head = static_cast<SplitWork*>(work);
    p.meta = reinterpret_cast<int64_t*>(static_cast<uint8_t*>(work) + kSplitHead);
    p.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(work) + kSplitHead + meta);
    p.part_ml = p.part_o + 2 * fit * p.part_rows * 128 * p.blocks;
  }
  st = launch_chained(kernel, grid, kLatThreads<FMT>, smem, stream, p);
  if (st != KV_OK || !p.split) return st;
  // the fewer the rows, the more parts has each and the more warps take it
  const int64_t rows = static_cast<int64_t>(a.num_q) * a.q_heads * p.blocks;
  int32_t wpr = 1;
  while (wpr < kLatJoinWarps && rows * wpr < 16ll * sms) wpr *= 2;
  const int64_t per = kLatJoinWarps / wpr;
  return launch_chained(kv_attend_latent_join<FMT, NR>, (rows + per - 1) / per, 32 * kLatJoinWarps, 0, stream, p, wpr);
}

// The instantiations: 16-bit rows, and e4m3fn ones.
kv_status latent_tile_src(const LatentTileParams& p, bool few, void* work, int64_t work_bytes, int64_t max_keys, cudaStream_t stream);
kv_status latent_tile_e4m3(const LatentTileParams& p, bool few, void* work, int64_t work_bytes, int64_t max_keys, cudaStream_t stream);

}  // namespace kvimpl
