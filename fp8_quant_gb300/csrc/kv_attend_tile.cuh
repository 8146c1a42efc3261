// Attention for many query rows per sequence (prefill): tiles of 128 query
// rows against tiles of 128 keys on the tensor cores (tcgen05).
//
// Products bound it: 4 * head_dim operations a query row and visible key.  A
// CTA takes one KV head and up to two tiles of query rows, a row being a
// (query, head of the group) pair, so that a group's heads share K and V and a
// window's edge costs few keys.
//
//   warps 0-3, 4-7  the softmax of tile 0 and of tile 1, a thread a row: S from
//                   TMEM, running maximum and sum in registers, P back over S
//                   as 16-bit, O rescaled in TMEM.  A maximum that grew by less
//                   than 2^8 is kept, as the weights then stay below 2^8 (fp16: 2^15,
//                   so that small ones keep their bits): O is seldom touched.
//   warp  8         issues the products: S_t = Q_t K^T (both operands in shared
//                   memory), O_t += P_t V (P in TMEM, V as it lies: keys as
//                   rows, head dims contiguous).  While one tile's softmax runs
//                   the other tile's products do.
//   warps 9-15      bring K and V from their pages into a ring of shared memory,
//                   in the 128-byte swizzle that the products read.  16-bit
//                   tiles whose keys all exist go by TMA, a box for each 64 dims
//                   and page, or 16 keys of one (windows, and pages that 128 keys
//                   are no multiple of); others by cp.async, 16 bytes a lane, with
//                   zeros for keys that no row needs.  Quantised rows are copied
//                   as they are by warps 14 (V) and 15 (K) with cp.async, three
//                   (e4m3fn) or four K and V tiles ahead, and become fp16 on their way
//                   into the ring (exact; see kv_attend_split.cuh) by 9-13.
//
// Weights are rounded once to 16 bits, as the product's operand: 2^-9 (bf16) or
// 2^-12 of each at most, which is what the output's own rounding is; their sum
// is of the unrounded ones in fp32.
//
// Registers: 512 threads are launched with 128 each; the softmax warps take 176
// or 184 (a row's 128 scores stay in registers), the others leave 80 or 72.
//
// TMEM (512 columns): S_0/P_0, S_1/P_1 (128 each), O_0, O_1 (head_dim each).
// The products of one CTA run in the order of their issue, so S_t of the next
// keys may overwrite P_t behind O_t's product without a wait between.
//
// A CTA stays and takes item after item (one CTA an SM): the copies run ahead
// into the next item's keys and its queries are loaded while the last one's
// softmax ends and its rows are written.
//
// Measured on one GB300 (32 over 8 heads of 128): one causal prompt of 8,192
// fp16 tokens 415 us, 1.32 PFLOP/s, and over e4m3fn keys (bf16 queries) 472 us; prompts of
// 2,500 and 4,095 bf16 tokens in windows of 1,024 133 us, 0.83 PFLOP/s; chunks of 400 - 1,000
// fp16 tokens over windows of 4,096 4-bit keys 150 us, 0.94 PFLOP/s.  What bounds it is the chain of one tile:
// S's product, maximum and weights (0.9 us of a row's 128 scores in one thread), P V, next
// product: 2.0 us a pair of tiles and 128 keys against 1.1 of products.  Handing the weights
// over in two or three parts, or loading S while its first half's maximum is taken, gained
// less than their barriers and registers cost (whole 408, halves 413, thirds 465 us; 406
// against 399 us); the next queries by the copying warps cost 5 % in windows.  Items of equal
// length leave CTAs idle in the last round: 5.5 rounds of windows take 6.
//
// Every wait has a limit (kSpin); a CTA whose wait ran out records that in the
// error record, lets its copies and products end and leaves.
#pragma once

#include "kv_async.cuh"
#include "kv_attend_split.cuh"

namespace kvimpl {

struct TileParams {
  AttendParams a;
  int32_t k_page, k_slot, v_page, v_slot;      // byte strides, in 32 bits
  int32_t ks_page, ks_slot, vs_page, vs_slot;  // of the block scales
  int32_t scale_word;  // bytes of them that may be copied at once: 8, 4 or 1
  int32_t qpt;     // queries of a tile: 128 / group
  int32_t blocks;  // query blocks of the launch (an upper bound)
  int32_t box;     // keys of a TMA box (a page, 128 of one, or 16); 0: no TMA
  CUtensorMap k_map, v_map;
};

constexpr int kTileRows = 128, kTileKeys = 128;
constexpr int kTileThreads = 512;
constexpr int kCopyThreads = 224;

template <int FMT, int DP>
struct TileSmem {
  // Ring units, a K or a V tile in 16 bits: quantised caches take three, as raw tiles wait in front of
  // the ring: as many as there is room for.
  static constexpr int kUnits = FMT == KV_CACHE_SRC ? 4 : 3;
  static constexpr int kUnit = kTileKeys * DP * 2;
  static constexpr int kQ = kTileRows * DP * 2;
  // a lane's pieces of a unit: 8 dims (16-bit) or 16 (quantised) of every kStep-th key
  // 256 threads of each, of the 65,536 registers of the launch
  static constexpr int kSoftmaxRegs = FMT == KV_CACHE_SRC ? 176 : 184, kOtherRegs = FMT == KV_CACHE_SRC ? 80 : 72;
  static_assert(256 * (kSoftmaxRegs + kOtherRegs) <= 65536, "the registers of the launch");
  static constexpr int kFillers = FMT == KV_CACHE_SRC ? kCopyThreads : kCopyThreads - 64;
  static constexpr int kPieces = FMT == KV_CACHE_SRC ? DP / 8 : DP / 16;
  static constexpr int kStep = kFillers / kPieces;
  static_assert(kFillers % kPieces == 0, "a lane keeps its piece of the rows");
  static constexpr int kRaw = FMT == KV_CACHE_SRC ? 0 : FMT == KV_CACHE_E4M3FN ? DP : DP / 2;  // bytes of a quantised row
  static constexpr int kRawScales = FMT == KV_CACHE_E2M1 ? 8 : 0;
  static constexpr int kPer = (kTileKeys + kStep - 1) / kStep;
  static constexpr int kOffRing = 2 * kQ;
  static constexpr int kOutDims = FMT == KV_CACHE_SRC ? 64 : 32;  // of 32 rows for each softmax warp
  static constexpr int kOffOut = kOffRing + kUnits * kUnit;
  static constexpr int kOffRaw = kOffOut + 8 * 64 * kOutDims;  // K and V tiles in turn, as they lie in the cache
  static constexpr int kRaws = FMT == KV_CACHE_SRC ? 0 : FMT == KV_CACHE_E4M3FN ? 3 : 4;
  static constexpr int kRawTile = kTileKeys * (kRaw + kRawScales);
  static constexpr int kOffBars = kOffRaw + kRaws * kRawTile;
  static constexpr int kBars = 2 * kUnits + 21;
  static constexpr int kTotal = kOffBars + kBars * 8 + 1024;    // the base is aligned to 1,024
};

// -- tcgen05 ----------------------------------------------------------------------------------

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The products and their commits: executed by a whole, converged warp, issued by
// one lane of it, so that descriptors and addresses stay in uniform registers.
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xFFFFFFFF;\n\t"
               "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar) : "memory");
}

// D (TMEM) = or += A (shared memory) B (shared memory)
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile("{\n\t.reg .pred e, p;\n\telect.sync _|e, 0xFFFFFFFF;\n\tsetp.ne.b32 p, %4, 0;\n\t"
               "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
               ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u) : "memory");
}

// D (TMEM) = or += A (TMEM) B (shared memory)
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile("{\n\t.reg .pred e, p;\n\telect.sync _|e, 0xFFFFFFFF;\n\tsetp.ne.b32 p, %4, 0;\n\t"
               "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
               ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u) : "memory");
}

#define KV_R4(r, i) "=r"((r)[i]), "=r"((r)[(i) + 1]), "=r"((r)[(i) + 2]), "=r"((r)[(i) + 3])
#define KV_R16(r, i) KV_R4(r, i), KV_R4(r, (i) + 4), KV_R4(r, (i) + 8), KV_R4(r, (i) + 12)
#define KV_S4(r, i) "r"((r)[i]), "r"((r)[(i) + 1]), "r"((r)[(i) + 2]), "r"((r)[(i) + 3])
#define KV_S16(r, i) KV_S4(r, i), KV_S4(r, (i) + 4), KV_S4(r, (i) + 8), KV_S4(r, (i) + 12)

// Columns of the warp's 32 lanes: a lane's row, a register a column.  The wait
// is part of the statement: nothing may touch the registers before it.
__device__ __forceinline__ void tc_ld32(uint32_t (&r)[32], uint32_t addr) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
               "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
               "tcgen05.wait::ld.sync.aligned;"
               : KV_R16(r, 0), KV_R16(r, 16) : "r"(addr) : "memory");
}

__device__ __forceinline__ void tc_ld64(uint32_t* r, uint32_t addr) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x64.b32 "
               "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n\t"
               "tcgen05.wait::ld.sync.aligned;"
               : KV_R16(r, 0), KV_R16(r, 16), KV_R16(r, 32), KV_R16(r, 48) : "r"(addr) : "memory");
}

__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
               "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};"
               ::KV_S16(r, 0), KV_S16(r, 16), "r"(addr) : "memory");
}

__device__ __forceinline__ void tc_ld16(uint32_t (&r)[16], uint32_t addr) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
               "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
               "tcgen05.wait::ld.sync.aligned;"
               : KV_R16(r, 0) : "r"(addr) : "memory");
}

__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
               "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};"
               ::KV_S16(r, 0), "r"(addr) : "memory");
}

#undef KV_R4
#undef KV_R16
#undef KV_S4
#undef KV_S16

// Descriptor of an operand in shared memory, 128-byte swizzle: rows of 128 bytes, groups of eight
// rows 1,024 bytes apart.  `lead`: bytes from one 64-element column block to the next, where the
// contiguous dimension is not the summed one (V); unused otherwise.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(lead >> 4) << 16) |
         (static_cast<uint64_t>(1024u >> 4) << 32) | (uint64_t{1} << 46) | (uint64_t{2} << 61);
}

// kind::f16 instruction descriptor: fp32 accumulator, A and B bf16 or f16, B's contiguous dimension.
__device__ __forceinline__ uint32_t instr_desc(bool bf16, bool b_rows_summed, int n) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((b_rows_summed ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(kTileRows >> 4) << 24);
}

// Byte of 16-byte piece `piece` of row `row` in a tile of `rows` rows.
__device__ __forceinline__ uint32_t swizzled(uint32_t row, uint32_t piece, uint32_t rows) {
  return (piece >> 3) * (rows * 128u) + row * 128u + (((piece & 7u) ^ (row & 7u)) << 4);
}

__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// x * s + t and x + y for both lanes, in one instruction each.
__device__ __forceinline__ float2 fma2(float2 x, float s, float t) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, c, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\tmov.b64 c, {%5, %5};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y) : "f"(x.x), "f"(x.y), "f"(s), "f"(t));
  return r;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y) : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return r;
}

// The keys that a block of queries sees between them, in tiles of kTileKeys: the
// first ones (sinks), filled up to a multiple of 16, and behind them the others
// from a multiple of 16 on, so that a window's edges cost few keys beside it
// (4 sinks and a window of 1,024 are 9 tiles for 64 queries, at tiles of whole
// 128s 10.5 on average).  Place v of the list is key(v).
struct TileKeys {
  int32_t n;       // tiles
  int32_t lo_key;  // first key of the windows
  int32_t lead, shift;
  __device__ __forceinline__ int32_t key(int32_t v) const { return v + (v >= lead ? shift : 0); }
};

__device__ __forceinline__ TileKeys tile_keys(const AttendParams& a, int32_t p_lo, int32_t p_hi) {
  const KeyList k = visible_keys(a, p_lo, p_hi);
  TileKeys r;
  r.lo_key = k.lo;
  const int32_t lo = k.lo & ~15;
  r.lead = min((k.sinks + 15) & ~15, lo);
  r.shift = lo - r.lead;
  r.n = p_hi < 0 ? 0 : (p_hi + 1 - r.shift + kTileKeys - 1) / kTileKeys;
  return r;
}

// Whether a page id of the keys that some row needs is out of range; by a whole warp, once the CTA has met one.
__device__ __noinline__ inline bool bad_pages(const AttendParams& a, int32_t b, TileKeys list, int32_t p_hi, WaitState* state) {
  if ((threadIdx.x & 31u) == 0u) state->hold(1);
  const int32_t* table = a.table + static_cast<int64_t>(b) * a.table_stride;
  bool bad = false;
  for (int32_t v = static_cast<int32_t>(threadIdx.x & 31u); v < list.n * kTileKeys; v += 32) {
    const int32_t k = list.key(v);
    if (k > p_hi || (k < list.lo_key && k >= a.sinks)) continue;
    const int32_t id = __ldg(table + a.page.quot(static_cast<uint32_t>(k)));
    bad |= id < 0 || id >= a.num_pages;
  }
  bad = __any_sync(0xFFFFFFFFu, bad);
  if ((threadIdx.x & 31u) == 0u) state->hold(-1);
  return bad;
}

// One item: a block of up to 2 * qpt queries of a sequence, for one KV head.
struct TileItem {
  int32_t b, kvh, tiles;
  AttendSeq seq;
  int32_t q_first, nq;   // the block's first query in its sequence, and their number
  int32_t p_first, p_hi; // positions of the first and the last
  TileKeys list;
  int32_t have;
};

// The CTA's item of a round, by a whole warp; false behind the last.  Blocks of
// a sequence come with the last queries, which see the most keys, first, and
// every second round runs the other way, so that CTAs get long and short ones.
__device__ __forceinline__ bool tile_item(const TileParams& p, int32_t round, TileItem* it) {
  const AttendParams& a = p.a;
  const uint32_t lane = threadIdx.x & 31u;
  it->have = 0;
  const int64_t n = static_cast<int64_t>(round) * gridDim.x + ((round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
  if (n >= static_cast<int64_t>(p.blocks) * a.kv_heads) return false;
  const int32_t want = static_cast<int32_t>(n / a.kv_heads);
  it->kvh = static_cast<int32_t>(n - static_cast<int64_t>(want) * a.kv_heads);
  int32_t before = 0;
  for (int32_t b0 = 0; b0 < a.num_seqs; b0 += 32) {
    const int32_t b = b0 + static_cast<int32_t>(lane);
    const int32_t k = b < a.num_seqs ? (attend_seq(a, b, false).nq + 2 * p.qpt - 1) / (2 * p.qpt) : 0;
    int32_t incl = k;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= static_cast<uint32_t>(o)) incl += v;
    }
    const int32_t at = before + incl - k;
    const uint32_t hit = __ballot_sync(0xFFFFFFFFu, want >= at && want < at + k);
    if (hit != 0u) {
      const int src = __ffs(static_cast<int>(hit)) - 1;
      it->b = b0 + src;
      it->q_first = __shfl_sync(0xFFFFFFFFu, k - 1 - (want - at), src) * 2 * p.qpt;
      it->seq = attend_seq(a, it->b, false);
      it->nq = min(2 * p.qpt, it->seq.nq - it->q_first);
      it->tiles = it->nq > p.qpt ? 2 : 1;
      it->p_first = it->seq.len - it->seq.nq + it->q_first;
      it->p_hi = it->p_first + it->nq - 1;
      it->list = tile_keys(a, it->p_first, it->p_hi);
      it->have = 1;
      return true;
    }
    before += __shfl_sync(0xFFFFFFFFu, incl, 31);
  }
  return false;
}

template <int FMT, int DP, bool kBF16>
__global__ void __launch_bounds__(kTileThreads, 1) kv_attend_tile(const __grid_constant__ TileParams p) {
  using S = TileSmem<FMT, DP>;
  constexpr bool kApart = FMT == KV_CACHE_SRC;  // of the waits
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ uint32_t sh_tmem;
  __shared__ WaitState sh_waits;
  __shared__ volatile int sh_bad;     // a page id out of range was met, in this item or an earlier or later one
  __shared__ TileItem sh_item[2];     // the item of an odd and of an even round, for the softmax warps

  const AttendParams& a = p.a;
  const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u;
  const uint32_t smem = (static_cast<uint32_t>(__cvta_generic_to_shared(smem_raw)) + 1023u) & ~1023u;
  const int32_t G = static_cast<int32_t>(a.group.d);
  const uint32_t ring = smem + S::kOffRing;
  const uint32_t full = smem + S::kOffBars, empty = full + 8 * S::kUnits;
  const uint32_t q_full = empty + 8 * S::kUnits, s_full = q_full + 16, p_full = s_full + 16, o_full = p_full + 16, item_full = o_full + 16,
                 item_empty = item_full + 16, raw_full = item_empty + 16, raw_empty = raw_full + 32, done = raw_empty + 32;
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
        static_cast<uint32_t>(__cvta_generic_to_shared(&sh_tmem))) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    for (int i = 0; i < S::kUnits; ++i) {
      bar_init(full + 8 * i, S::kFillers);
      bar_init(empty + 8 * i, 1);
    }
    for (int t = 0; t < 2; ++t) {
      bar_init(q_full + 8 * t, kTileRows);
      bar_init(s_full + 8 * t, 1);
      bar_init(p_full + 8 * t, kTileRows);
      bar_init(o_full + 8 * t, 1);
      bar_init(item_full + 8 * t, 1);
      bar_init(item_empty + 8 * t, 8);
    }
    for (int i = 0; i < S::kRaws; ++i) {
      bar_init(raw_full + 8 * i, 32);
      bar_init(raw_empty + 8 * i, S::kFillers / 32);
    }
    bar_init(done, 1);
    sh_waits = WaitState{0, 0};
    sh_bad = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh_tmem;
  WaitState* const state = &sh_waits;
  grid_handover();
  if (blockIdx.x == 0 && warp == 15)  // lengths out of range, once
    for (int32_t b = static_cast<int32_t>(lane); b < a.num_seqs; b += 32) attend_seq(a, b, true);
  __syncwarp();

  // (all warps of a warpgroup execute the same one)
  if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kOtherRegs));
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kSoftmaxRegs));
    // ======================================================================================
    // softmax of tile t: a thread a row
    // ======================================================================================
    const int32_t t = static_cast<int32_t>(warp >> 2);
    const int32_t r = static_cast<int32_t>(tid & 127u);
    const int32_t qi = static_cast<int32_t>(a.group.quot(static_cast<uint32_t>(r)));
    const int32_t gh = r - qi * G, q_in = t * p.qpt + qi;  // head in the group, query in the block
    const float vscale = tensor_scale(a.v_scale);
    const float full_scale = a.scale_log2 * tensor_scale(a.k_scale);
    const uint32_t flip = full_scale < 0.0f ? 0x80008000u : 0u;  // the maximum is taken before the scale
    const uint32_t lanes = (warp & 3u) << 21;  // the warp's 32 lanes of TMEM
    const uint32_t s_at = tmem + lanes + t * 128, o_at = tmem + lanes + 256 + t * DP;
    bool ok = true;
    auto take_item = [&](int32_t round, TileItem* x) {
      ok = __all_sync(0xFFFFFFFFu, bar_wait<kApart>(item_full + 8 * (round & 1), static_cast<uint32_t>(round >> 1) & 1u, state));
      if (!ok) return;
      *x = sh_item[round & 1];
      __syncwarp();
      if (lane == 0u) bar_arrive(item_empty + 8 * (round & 1));
    };
    auto row_live = [&](const TileItem& x) { return t < x.tiles && qi < p.qpt && q_in < x.nq; };
    // A warp's queries: kQL lanes a row, 16 bytes each, so that a load meets few lines of 128 bytes.
    // Lane l's i-th piece is piece l % kQL of row row0 + i * (32 / kQL) + l / kQL.
    constexpr int kQL = DP / 8, kQR = 32 / kQL;
    const int32_t row0 = (static_cast<int32_t>(warp) & 3) * 32, q_row = static_cast<int32_t>(lane) / kQL, q_piece = static_cast<int32_t>(lane) % kQL;
    uint4 qw[kQL];
    auto load_q = [&](const TileItem& x) {
      const uint8_t* src = a.q + static_cast<int64_t>(x.seq.q0 + x.q_first + t * p.qpt) * a.q_token +
                           static_cast<int64_t>(x.kvh * G) * a.q_head + 16 * q_piece;
#pragma unroll
      for (int i = 0; i < kQL; ++i) {
        const int32_t row = row0 + i * kQR + q_row, y = static_cast<int32_t>(a.group.quot(static_cast<uint32_t>(row)));
        qw[i] = make_uint4(0u, 0u, 0u, 0u);
        if (t < x.tiles && y < p.qpt && t * p.qpt + y < x.nq && 8 * q_piece < a.head_dim)
          qw[i] = __ldg(reinterpret_cast<const uint4*>(src + y * a.q_token + (row - y * G) * a.q_head));
      }
    };
    // Queries to shared memory; the products that read this tile's queries before have ended, as
    // their scores were waited for.  Returns the row's factor of the scores.
    auto put_q = [&](const TileItem& x) {
      float scale = full_scale;
      if constexpr (FMT != KV_CACHE_SRC) {
        if (a.bf16) {  // into fp16's range: the row's largest element to 2^13 .. 2^14
          float row_f = 1.0f;
#pragma unroll
          for (int i = 0; i < kQL; ++i) {
            uint32_t y = absmax_pair<true>(absmax_pair<true>(absmax_pair<true>(absmax_pair<true>(0u, qw[i].x), qw[i].y), qw[i].z), qw[i].w);
#pragma unroll
            for (int o = 1; o < kQL; o <<= 1) y = absmax_pair<true>(y, __shfl_xor_sync(0xFFFFFFFFu, y, o));
            const uint32_t e = __float_as_uint(absmax_pair_value<true>(y)) >> 23;
            const float f = __uint_as_float(min(254u, 267u - e) << 23);
            auto shift = [&](uint32_t z) {
              const float2 v = widen2<true>(z);
              return pack2(v.x * f, v.y * f, false);
            };
            qw[i] = make_uint4(shift(qw[i].x), shift(qw[i].y), shift(qw[i].z), shift(qw[i].w));
            const float mine = __shfl_sync(0xFFFFFFFFu, f, (static_cast<int>(lane) % kQR) * kQL);
            if (static_cast<int>(lane) / kQR == i) row_f = mine;
          }
          scale *= __fdiv_rn(1.0f, row_f);
        }
      }
      if (t < x.tiles && x.list.n > 0) {
        const uint32_t dst = smem + t * S::kQ;
#pragma unroll
        for (int i = 0; i < kQL; ++i)
          st_shared16(dst + swizzled(static_cast<uint32_t>(row0 + i * kQR + q_row), q_piece, kTileRows),
                      qw[i].x ^ flip, qw[i].y ^ flip, qw[i].z ^ flip, qw[i].w ^ flip);
        fence_async_shared();
        bar_arrive(q_full + 8 * t);
      }
      scale = fabsf(scale);
      return scale == 0.0f ? __uint_as_float(1u) : scale;  // hidden scores (-inf) must stay -inf
    };
    float scale = full_scale;
    TileItem it;
    it.have = 0;
    take_item(0, &it);
    if (ok && it.have) {
      load_q(it);
      scale = put_q(it);
    }
    uint32_t waits = 0u, items = 0u;  // phases of s_full and p_full, and of q_full and o_full, that went by
    for (int32_t round = 0; ok && it.have;) {
      const bool mine = row_live(it);
      const int32_t pos = mine ? it.p_first + q_in : -1;
      const int32_t tok = it.seq.q0 + it.q_first + q_in, h = it.kvh * G + gh;
      const bool live = t < it.tiles && it.list.n > 0;
      // the maximum of scaled scores, as last used and less kSmall: weights begin at 2 to that
      constexpr float kSmall = kBF16 ? 0.0f : 7.0f;
      float m = -INFINITY, l = 0.0f;
      // positions of the tile's rows
      const int32_t t_lo = it.p_first + t * p.qpt, t_hi = min(t_lo + p.qpt - 1, it.p_hi);
      for (int32_t j = 0; live && j < it.list.n; ++j) {
        ok = __all_sync(0xFFFFFFFFu, bar_wait<kApart>(s_full + 8 * t, waits & 1u, state));
        if (!ok) break;
        tc_fence_after();
        uint32_t sw[kTileKeys];
        tc_ld64(sw, s_at);
        tc_ld64(sw + 64, s_at + 64);
        float s[kTileKeys];
#pragma unroll
        for (int i = 0; i < kTileKeys; ++i) s[i] = __uint_as_float(sw[i]);
        // mask
        const int32_t v0 = j * kTileKeys, v1 = v0 + kTileKeys - 1;
        if (!(it.list.key(v1) <= t_lo && (a.window == 0 || v1 < a.sinks || (v0 >= it.list.lead && it.list.key(v0) > t_hi - a.window)))) {
          // keys up to pos, and of those the window's or the sinks'
          auto upto = [](int32_t n) {  // n low bits set
            return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
          };
          auto seen = [&](int32_t k0) {  // of 16 keys from k0
            uint32_t see = upto(pos - k0 + 1);
            if (a.window > 0) see &= ~upto(pos - a.window - k0 + 1) | upto(a.sinks - k0);
            return see & 0xFFFFu;
          };
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t see = seen(it.list.key(v0 + 32 * c)) | seen(it.list.key(v0 + 32 * c + 16)) << 16;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if ((see & (1u << i)) == 0u) s[32 * c + i] = -INFINITY;
          }
        }
        float xs[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) xs[i] = fmaxf(s[i], s[i + 8]);
#pragma unroll
        for (int i = 16; i < kTileKeys; i += 16)
#pragma unroll
          for (int y = 0; y < 8; ++y) xs[y] = fmaxf(xs[y], fmaxf(s[i + y], s[i + 8 + y]));
        float x = fmaxf(fmaxf(fmaxf(xs[0], xs[1]), fmaxf(xs[2], xs[3])), fmaxf(fmaxf(xs[4], xs[5]), fmaxf(xs[6], xs[7])));
        x = __fmaf_rn(x, scale, -kSmall);
        // a maximum that grew little is kept (the weights stay below 2^(kSmall + 8))
        const bool grow = x > m + 8.0f || (m == -INFINITY && x > m);
        if (__any_sync(0xFFFFFFFFu, grow)) {
          const float mn = grow ? x : m;
          const float f = grow ? exp2_fast(m - (mn == -INFINITY ? 0.0f : mn)) : 1.0f;
          m = mn;
          if (j > 0) {
            l *= f;
#pragma unroll 1
            for (int c = 0; c < DP / 16; ++c) {  // (few registers: the scores are in them too)
              uint32_t w[16];
              tc_ld16(w, o_at + 16 * c);
#pragma unroll
              for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * f);
              tc_st16(o_at + 16 * c, w);
            }
          }
        }
        const float ref = m == -INFINITY ? 0.0f : m;
        // pairs of weights: one packed product and sum for both
        float2 sum[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) sum[y] = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t w[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float2 z = fma2(make_float2(s[64 * c + 2 * i], s[64 * c + 2 * i + 1]), scale, -ref);
            const float2 e = make_float2(exp2_fast(z.x), exp2_fast(z.y));
            sum[i & 3] = add2(sum[i & 3], e);
            w[i] = pack2(e.x, e.y, kBF16);
          }
          tc_st32(s_at + 32 * c, w);
        }
        tc_wait_st();
        tc_fence_before();
        bar_arrive(p_full + 8 * t);
        sum[0] = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
        l += sum[0].x + sum[0].y;
        ++waits;
      }
      if (!ok) break;
      // -- the next item's queries, so that its scores are there when this one's rows are written ---
      TileItem next;
      take_item(++round, &next);
      if (!ok) break;
      if (next.have) {
        load_q(next);
        scale = put_q(next);
      }
      if (t < it.tiles) {
        bool fine = l > 0.0f;
        if (live) {
          ok = __all_sync(0xFFFFFFFFu, bar_wait<kApart>(o_full + 8 * t, items & 1u, state));
          if (!ok) break;
          ++items;
          tc_fence_after();
          const float inv = __fdiv_rn(vscale, l);
          // kOutDims dims at a time through shared memory, so that neighbouring lanes write one row
          constexpr int kOL = S::kOutDims / 8, kOR = 32 / kOL;  // lanes a row, rows at once
          const uint32_t stage = smem + S::kOffOut + warp * (64u * S::kOutDims);
          auto staged = [&](uint32_t row, uint32_t piece) {
            return stage + row * (2u * S::kOutDims) + ((piece ^ (kOL == 8 ? row & 7u : row >> 1 & 3u)) << 4);
          };
          uint8_t* const out = a.out + static_cast<int64_t>(it.seq.q0 + it.q_first + t * p.qpt) * a.o_token +
                               static_cast<int64_t>(it.kvh * G) * a.o_head + 16 * (lane % kOL);
#pragma unroll
          for (int c = 0; c < DP / S::kOutDims; ++c) {
#pragma unroll
            for (int half = 0; half < S::kOutDims / 32; ++half) {
              uint32_t w[32];
              tc_ld32(w, o_at + S::kOutDims * c + 32 * half);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t o[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                  const float lo = __uint_as_float(w[8 * i + 2 * x]) * inv, hi = __uint_as_float(w[8 * i + 2 * x + 1]) * inv;
                  fine = fine && fabsf(lo) < INFINITY && fabsf(hi) < INFINITY;
                  o[x] = pack2(lo, hi, a.bf16);
                }
                st_shared16(staged(lane, 4 * half + i), o[0], o[1], o[2], o[3]);
              }
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 32 / kOR; ++i) {
              const uint32_t row = kOR * i + lane / kOL;
              const int32_t rr = row0 + static_cast<int32_t>(row), y = static_cast<int32_t>(a.group.quot(static_cast<uint32_t>(rr)));
              const uint4 v = ld_shared16(staged(row, lane % kOL));
              if (y < p.qpt && t * p.qpt + y < it.nq && static_cast<int32_t>(S::kOutDims * c + 8 * (lane % kOL)) < a.head_dim)
                *reinterpret_cast<uint4*>(out + y * a.o_token + (rr - y * G) * a.o_head + 2 * S::kOutDims * c) = v;
            }
            __syncwarp();
          }
        }
        // rows of an item with a page id out of range are done again: zeros stood for its keys
        const bool bad = __any_sync(0xFFFFFFFFu, sh_bad != 0) && bad_pages(a, it.b, it.list, it.p_hi, state);
        const bool done = mine && fine && !bad;
        if (done && a.lse)  // (a row without keys is not fine)
          a.lse[static_cast<int64_t>(tok) * a.q_heads + h] = (m + log2f(l)) * 0.6931471805599453f;
        uint32_t again = __ballot_sync(0xFFFFFFFFu, mine && !done);
        const bool hold = again != 0u && lane == 0u;
        if (hold) state->hold(1);
        while (again != 0u) {
          const int src = __ffs(static_cast<int>(again)) - 1;
          again &= again - 1u;
          attend_row<FMT, 8>(a, it.b, __shfl_sync(0xFFFFFFFFu, pos, src), __shfl_sync(0xFFFFFFFFu, tok, src),
                             __shfl_sync(0xFFFFFFFFu, h, src));
        }
        if (hold) state->hold(-1);
      }
      it = next;
    }
  } else if (warp == 8) {
    // ======================================================================================
    // the products
    // ======================================================================================
    const uint32_t qk_desc = instr_desc(kBF16, false, kTileKeys), pv_desc = instr_desc(kBF16, true, DP);
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
      if (ok) ok = __all_sync(0xFFFFFFFFu, bar_wait<kApart>(bar, parity, state));
      if (ok) tc_fence_after();
    };
    // descriptors of the operands' first pieces; the others are constant steps (in 16 bytes) away
    const uint64_t q_desc = smem_desc(smem, 16), k_desc = smem_desc(ring, 16), v_desc = smem_desc(ring, kTileKeys * 128);
    uint32_t unit = 0u;                              // ring units that went by
    uint32_t items0 = 0u, items1 = 0u, done0 = 0u, done1 = 0u;  // of each tile: items and products P V
    // the items, a round ahead of their use, for this warp and the softmax warps
    auto publish = [&](int32_t round, TileItem* x) {
      tile_item(p, round, x);
      if (round >= 2) wait(item_empty + 8 * (round & 1), static_cast<uint32_t>((round >> 1) - 1) & 1u);
      if (!ok) return;
      if (lane == 0u) {
        sh_item[round & 1] = *x;
        bar_arrive(item_full + 8 * (round & 1));
      }
      __syncwarp();
    };
    TileItem it, next;
    publish(0, &it);
    for (int32_t round = 0; ok && it.have; ++round, it = next) {
      const int32_t n = it.list.n, tiles = it.tiles;
      if (n == 0) {
        publish(round + 1, &next);
        continue;
      }
      auto wait_unit = [&](uint32_t u) { wait(full + 8 * (u % S::kUnits), (u / S::kUnits) & 1u); };
      auto scores = [&](int32_t t, uint32_t u) {  // S_t = Q_t K^T, K in unit u
        if (!ok) return;
        const uint64_t q = q_desc + static_cast<uint32_t>(t) * (S::kQ >> 4), k = k_desc + (u % S::kUnits) * (S::kUnit >> 4);
#pragma unroll
        for (int i = 0; i < DP / 16; ++i) {
          const uint32_t at = ((i / 4) * (kTileRows * 128) + (i % 4) * 32) >> 4;
          tc_mma_ss(tmem + t * 128, q + at, k + at, qk_desc, i > 0);
        }
        tc_commit(s_full + 8 * t);
        if (t == tiles - 1) tc_commit(empty + 8 * (u % S::kUnits));
      };
      for (int32_t t = 0; t < tiles; ++t) {
        wait(q_full + 8 * t, (t ? items1 : items0) & 1u);
        if (t == 0) wait_unit(unit);
        scores(t, unit);
      }
      if (ok) publish(round + 1, &next);
      for (int32_t j = 0; j < n && ok; ++j) {
        const uint32_t u = unit + 2 * j;
        for (int32_t t = 0; t < tiles; ++t) {
          const uint32_t parity = (t ? done1 : done0) & 1u;
          if (t == 0) {  // both before P, so that its two products follow each other
            wait_unit(u + 1);
            if (j + 1 < n) wait_unit(u + 2);
          }
          const uint64_t v = v_desc + ((u + 1) % S::kUnits) * (S::kUnit >> 4);
          wait(p_full + 8 * t, parity);
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < kTileKeys / 16; ++i)  // O_t += P_t V
            tc_mma_ts(tmem + 256 + t * DP, tmem + t * 128 + i * 8, v + i * (2048 >> 4), pv_desc, j > 0 || i > 0);
          if (t == tiles - 1) tc_commit(empty + 8 * ((u + 1) % S::kUnits));
          if (j == n - 1) tc_commit(o_full + 8 * t);
          if (t) ++done1; else ++done0;
          if (j + 1 < n) {
            scores(t, u + 2);
          }
        }
      }
      unit += 2 * n;
      ++items0;
      if (tiles > 1) ++items1;
    }
    if (!ok) {  // products still in flight read shared memory and write TMEM: let them end
      tc_commit(done);
      for (uint32_t i = 0; i < kSpin && !bar_try(done, 0); ++i) {}
    }
    __syncwarp();
  } else {
    // ======================================================================================
    // K and V into the ring
    // ======================================================================================
    const int32_t c = static_cast<int32_t>(tid) - (kTileThreads - kCopyThreads);
    const uint32_t row_bytes = static_cast<uint32_t>(a.head_dim) * (FMT == KV_CACHE_SRC ? 16 : FMT == KV_CACHE_E4M3FN ? 8 : 4) / 8;
    // Quantised rows of 128 dims: the lanes of the second 64 take the other key of a pair, so that the
    // eight lanes whose stores go together meet all banks.
    const uint32_t piece = static_cast<uint32_t>(c) % S::kPieces;
    const uint32_t key0 = static_cast<uint32_t>(c) / S::kPieces ^ (FMT != KV_CACHE_SRC && DP == 128 ? piece >> 2 : 0u);
    bool ok = true;
    uint32_t unit = 0u;  // ring units that went by
    auto wait_empty = [&](uint32_t u) {
      if (ok && u >= S::kUnits) ok = __all_sync(0xFFFFFFFFu, bar_wait<kApart>(empty + 8 * (u % S::kUnits), (u / S::kUnits - 1) & 1u, state));
    };
    // Which of the lane's keys of a tile a row needs, a bit each, and their pages.  What is loaded
    // is not looked at before it is used, a tile later (a select behind a load would wait for it),
    // and nothing branches: keys that are not needed read the last needed one's entry.
    auto pages_of = [&](const TileItem& it, int32_t j, int32_t (&id)[S::kPer]) -> uint32_t {
      uint32_t want = 0u;
      const int32_t* table = a.table + static_cast<int64_t>(it.b) * a.table_stride;
#pragma unroll
      for (int i = 0; i < S::kPer; ++i) {
        const uint32_t key = key0 + i * S::kStep;
        const int32_t k = it.list.key(j * kTileKeys + static_cast<int32_t>(key));
        const bool w = (kTileKeys % S::kStep == 0 || key < kTileKeys) && k <= it.p_hi && (k >= it.list.lo_key || k < a.sinks);
        want |= (w ? 1u : 0u) << i;
        id[i] = __ldg(table + a.page.quot(static_cast<uint32_t>(min(k, it.p_hi))));
      }
      return want;
    };
    // The bits of keys on pages that exist; the others are counted.
    auto checked = [&](const TileItem& it, uint32_t want, const int32_t (&id)[S::kPer]) -> uint32_t {
      uint32_t bad = 0u;
#pragma unroll
      for (int i = 0; i < S::kPer; ++i)
        bad |= (static_cast<uint32_t>(id[i]) >= static_cast<uint32_t>(a.num_pages) ? 1u : 0u) << i;
      bad &= want;
      if (bad != 0u) {
        sh_bad = 1;
        record_oob(a.err, static_cast<uint64_t>(it.b));
      }
      return want & ~bad;
    };
    auto offset_of = [&](const TileItem& it, int32_t j, int i) -> int32_t {  // in its page
      const uint32_t k = static_cast<uint32_t>(it.list.key(j * kTileKeys + static_cast<int32_t>(key0) + i * S::kStep));
      return static_cast<int32_t>(k - a.page.quot(k) * a.page.d);
    };
    TileItem it;
    if constexpr (FMT == KV_CACHE_SRC) {
      // TMA: lane i of warp 9 takes the tile's i-th page; every warp knows whether all are there
      const int32_t boxes = p.box > 0 ? kTileKeys / p.box : 0;
      for (int32_t round = 0; ok && tile_item(p, round, &it); ++round) {
        const int32_t* table = a.table + static_cast<int64_t>(it.b) * a.table_stride;
        const uint8_t* const kbase = a.k + it.kvh * a.k_head;
        const uint8_t* const vbase = a.v + it.kvh * a.v_head;
        auto first_page = [&](int32_t j) -> int32_t {
          if (j >= it.list.n || static_cast<int32_t>(lane) >= boxes) return 0;
          const int32_t k = it.list.key(j * kTileKeys + static_cast<int32_t>(lane) * p.box);
          return k < it.seq.len ? __ldg(table + a.page.quot(static_cast<uint32_t>(k))) : -1;
        };
        int32_t next = first_page(0);
        for (int32_t j = 0; j < it.list.n && ok; ++j, unit += 2) {
          const int32_t mine = next;
          next = first_page(j + 1);
          const bool whole = boxes > 0 && it.list.key(j * kTileKeys + kTileKeys - 1) < it.seq.len &&
                             __all_sync(0xFFFFFFFFu, mine >= 0 && mine < a.num_pages);
          if (whole) {
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
              wait_empty(unit + kv);
              if (!ok) break;
              const uint32_t slot = (unit + kv) % S::kUnits, bar = full + 8 * slot;
              if (c == 0) bar_arrive_expect(bar, S::kUnit); else bar_arrive(bar);
              __syncwarp();
              if (warp == 9 && static_cast<int32_t>(lane) < boxes) {
                const uint32_t k = static_cast<uint32_t>(it.list.key(j * kTileKeys + static_cast<int32_t>(lane) * p.box));
                const int32_t key = static_cast<int32_t>(k - a.page.quot(k) * a.page.d);
#pragma unroll
                for (int x = 0; x < DP / 64; ++x)
                  tma_box(ring + slot * S::kUnit + x * (kTileKeys * 128) + lane * static_cast<uint32_t>(p.box) * 128u,
                           kv ? &p.v_map : &p.k_map, bar, 64 * x, key, it.kvh, mine);
              }
            }
          } else {
            int32_t id[S::kPer];
            const uint32_t want = checked(it, pages_of(it, j, id), id);
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
              wait_empty(unit + kv);
              if (!ok) break;
              const uint8_t* base = kv ? vbase : kbase;
              const uint32_t at = ring + ((unit + kv) % S::kUnits) * S::kUnit;
#pragma unroll
              for (int i = 0; i < S::kPer; ++i) {
                const uint32_t key = key0 + i * S::kStep;
                if (kTileKeys % S::kStep != 0 && key >= kTileKeys) break;
                const bool w = (want >> i & 1u) != 0u && piece * 16 < row_bytes;
                const uint8_t* src = base + (w ? wide(id[i], kv ? p.v_page : p.k_page) +
                                                        wide(offset_of(it, j, i), kv ? p.v_slot : p.k_slot) + piece * 16 : 0);
                copy_async<16>(at + swizzled(key, piece, kTileKeys), src, w ? 16u : 0u);
              }
              commit_async();
            }
            if (ok) {
              wait_async<1>();
              fence_async_shared();
              bar_arrive(full + 8 * (unit % S::kUnits));
            }
            wait_async<0>();
            if (ok) {
              fence_async_shared();
              bar_arrive(full + 8 * ((unit + 1) % S::kUnits));
            }
          }
        }
      }
      if (!ok)  // boxes in flight write shared memory: let them land before the CTA leaves it
        for (int i = 0; i < 1000; ++i) __nanosleep(1000);
    } else if (warp >= 14) {
      // ====================================================================================
      // quantised rows as they lie into shared memory: lane l looks up keys l, l + 32, ..
      // ====================================================================================
      const int32_t kv = warp == 15 ? 0 : 1;
      const int32_t page_stride = kv ? p.v_page : p.k_page, slot_stride = kv ? p.v_slot : p.k_slot;
      constexpr int kKeys = kTileKeys / 32, kChunks = S::kRaw / 16, kRows = 32 / kChunks;
      int32_t round = 0, j = 0;
      bool have = tile_item(p, 0, &it);
      auto skip_empty = [&] {
        while (have && j >= it.list.n) {
          j = 0;
          have = tile_item(p, ++round, &it);
        }
      };
      int32_t id[kKeys];
      auto look = [&] {  // the pages of the cursor's tile; not looked at before a tile later
        const int32_t* table = a.table + static_cast<int64_t>(it.b) * a.table_stride;
#pragma unroll
        for (int i = 0; i < kKeys; ++i)
          id[i] = __ldg(table + a.page.quot(static_cast<uint32_t>(min(it.list.key(j * kTileKeys + 32 * i + static_cast<int32_t>(lane)), it.p_hi))));
      };
      skip_empty();
      if (have) look();
      for (uint32_t tile = 0u; have; ++tile) {
        // page and slot of the lane's keys; page -1: a key that no row needs
        int32_t pg[kKeys], of[kKeys];
        uint32_t bad = 0u;
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
          const int32_t k = it.list.key(j * kTileKeys + 32 * i + static_cast<int32_t>(lane));
          const bool want = k <= it.p_hi && (k >= it.list.lo_key || k < a.sinks);
          const bool page = static_cast<uint32_t>(id[i]) < static_cast<uint32_t>(a.num_pages);
          if (want && !page) bad = 1u;
          pg[i] = want && page ? id[i] : -1;
          of[i] = k - static_cast<int32_t>(a.page.quot(static_cast<uint32_t>(k)) * a.page.d);
        }
        if (bad != 0u) {
          sh_bad = 1;
          if (kv == 0) record_oob(a.err, static_cast<uint64_t>(it.b));
        }
        __syncwarp();
        const int32_t kvh = it.kvh;
        ++j;
        skip_empty();
        if (have) look();
        const uint32_t u = 2u * tile + static_cast<uint32_t>(kv), raw = u % S::kRaws;
        if (u >= S::kRaws) ok = __all_sync(0xFFFFFFFFu, bar_wait<kApart>(raw_empty + 8 * raw, (u / S::kRaws - 1u) & 1u, state));
        if (!ok) break;
        const uint32_t at = smem + S::kOffRaw + raw * S::kRawTile;
        const uint8_t* const base = kv ? a.v + kvh * a.v_head : a.k + kvh * a.k_head;
        // kChunks lanes a row, so that a copy meets few lines
        const uint32_t chunk = lane % kChunks;
        const int32_t bytes = min(max(static_cast<int32_t>(row_bytes) - 16 * static_cast<int32_t>(chunk), 0), 16);
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
          const int64_t off = pg[i] < 0 ? -1 : wide(pg[i], page_stride) + wide(of[i], slot_stride);
#pragma unroll
          for (int y = 0; y < 32 / kRows; ++y) {
            const int64_t o = __shfl_sync(0xFFFFFFFFu, off, y * kRows + lane / kChunks);
            const uint32_t key = 32 * i + y * kRows + lane / kChunks;
            const bool w = o != -1 && bytes > 0;
            copy_async<16>(at + key * S::kRaw + chunk * 16, base + (w ? o + 16 * chunk : 0), w ? static_cast<uint32_t>(bytes) : 0u);
          }
        }
        bool plain = false;
        if constexpr (FMT == KV_CACHE_E2M1) {
          const uint8_t* const sb = kv ? a.v_sc + kvh * a.vs_head : a.k_sc + kvh * a.ks_head;
          const int32_t sp = kv ? p.vs_page : p.ks_page, ss = kv ? p.vs_slot : p.ks_slot;
          const int32_t ds = a.head_dim / 16;
          plain = p.scale_word == 1;
#pragma unroll
          for (int i = 0; i < kKeys; ++i) {
            const bool w = pg[i] >= 0;
            const uint8_t* src = sb + (w ? wide(pg[i], sp) + wide(of[i], ss) : 0);
            const uint32_t dst = at + kTileKeys * S::kRaw + (32 * i + lane) * 8;
            if (p.scale_word == 8) {
              copy_async<8>(dst, src, w ? 8u : 0u);
            } else if (p.scale_word == 4) {
              copy_async<4>(dst, src, w ? 4u : 0u);
              copy_async<4>(dst + 4, w && ds > 4 ? src + 4 : src, w && ds > 4 ? static_cast<uint32_t>(min(ds - 4, 4)) : 0u);
            } else {
              uint32_t lo = 0u, hi = 0u;
              for (int32_t x = 0; x < ds && w; ++x) {
                const uint32_t v = __ldg(src + x);
                if (x < 4) lo |= v << (8 * x); else hi |= v << (8 * x - 32);
              }
              asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(dst), "r"(lo), "r"(hi) : "memory");
            }
          }
        }
        if (plain) {
          wait_all_async();
          bar_arrive(raw_full + 8 * raw);
        } else {
          bar_arrive_copies(raw_full + 8 * raw);
        }
      }
      wait_all_async();  // copies in flight write shared memory
    } else {
      // ====================================================================================
      // and from there, as fp16, into the ring
      // ====================================================================================
      constexpr int kWords = FMT == KV_CACHE_E4M3FN ? 4 : 2;
      for (int32_t round = 0; ok && tile_item(p, round, &it); ++round) {
#pragma unroll 1
        for (int32_t left = 2 * it.list.n; left > 0 && ok; --left, ++unit) {
          const uint32_t raw = unit % S::kRaws, from = smem + S::kOffRaw + raw * S::kRawTile;
          uint32_t w[S::kPer][kWords], sc[FMT == KV_CACHE_E2M1 ? S::kPer : 1];
          ok = __all_sync(0xFFFFFFFFu, bar_wait<kApart>(raw_full + 8 * raw, (unit / S::kRaws) & 1u, state));
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < S::kPer; ++i) {
            const uint32_t key = min(key0 + i * S::kStep, static_cast<uint32_t>(kTileKeys - 1));
            if constexpr (FMT == KV_CACHE_E4M3FN) {
              const uint4 v = ld_shared16(from + key * S::kRaw + piece * 16);
              w[i][0] = v.x; w[i][1] = v.y; w[i][2] = v.z; w[i][3] = v.w;
            } else {
              asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[i][0]), "=r"(w[i][1]) : "r"(from + key * S::kRaw + piece * 8) : "memory");
              asm volatile("ld.shared.u8 %0, [%1];" : "=r"(sc[i]) : "r"(from + kTileKeys * S::kRaw + key * 8 + piece) : "memory");
            }
          }
          __syncwarp();
          if (lane == 0u) bar_arrive(raw_empty + 8 * raw);
          wait_empty(unit);
          if (!ok) break;
          const uint32_t at = ring + (unit % S::kUnits) * S::kUnit;
#pragma unroll
          for (int i = 0; i < S::kPer; ++i) {
            const uint32_t key = key0 + i * S::kStep;
            if (kTileKeys % S::kStep != 0 && key >= kTileKeys) break;
            uint32_t f[8];
            if constexpr (FMT == KV_CACHE_E4M3FN) {
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                f[2 * x] = f16x2_from_e4m3x2(w[i][x]);
                f[2 * x + 1] = f16x2_from_e4m3x2(w[i][x] >> 16);
              }
            } else {
              const uint32_t s2 = f16x2_from_e4m3x2(sc[i] * 0x0101u);  // e2m1 codes are finite
              f16x2_from_e2m1x8(w[i][0], f);
              f16x2_from_e2m1x8(w[i][1], f + 4);
#pragma unroll
              for (int x = 0; x < 8; ++x) f[x] = mul_f16x2(f[x], s2);
            }
            st_shared16(at + swizzled(key, 2 * piece, kTileKeys), f[0], f[1], f[2], f[3]);
            st_shared16(at + swizzled(key, 2 * piece + 1, kTileKeys), f[4], f[5], f[6], f[7]);
          }
          fence_async_shared();
          bar_arrive(full + 8 * (unit % S::kUnits));
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && state->ran_out()) record_wait(a.err);
  if (warp == 8) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------

template <int FMT, int DP, bool kBF16>
kv_status launch_tile(TileParams p, cudaStream_t stream) {
  auto* kernel = kv_attend_tile<FMT, DP, kBF16>;
  constexpr int kSmem = TileSmem<FMT, DP>::kTotal;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static SmemOptIn opt_in;
  const kv_status st = opt_in(reinterpret_cast<const void*>(kernel), kSmem);
  if (st != KV_OK) return st;
  int sms = 0;
  const kv_status sc = current_sm_count(&sms);
  if (sc != KV_OK) return sc;
  const int64_t items = static_cast<int64_t>(p.blocks) * p.a.kv_heads;
  const int64_t grid = items < sms ? items : sms;
  return launch_chained(kernel, grid, kTileThreads, kSmem, stream, p);
}

// The instantiations: 16-bit caches, and quantised ones.
kv_status tile_src(const TileParams& p, cudaStream_t stream);
kv_status tile_quant(const TileParams& p, kv_cache_format format, cudaStream_t stream);

}  // namespace kvimpl
