// Attention over a paged cache of latent rows on the tensor cores (tcgen05).
//
// All query heads share one row of D dims per key, L of them values, so a key's
// bytes meet HQ rows a query: 4 * HQ * (D + L) / (4 * D) operations a byte, 60
// for 32 heads of 576 / 512. One query a sequence is bound by the cache's
// bytes, from about four queries on by the products.
//
// A CTA takes up to NR = 64 or 32 query rows, a row being a (query, head)
// pair, and goes over tiles of 64 keys:
//   S [rows][keys] = Q K^T       M = 64 (Q, shared memory), N = 64 keys, all D dims;
//   O^T [dims][rows] += V^T P^T  M = 128 dims, N = NR rows: the tile's first L
//                                dims as they lie (dims contiguous), P in
//                                shared memory.
// O^T of 512 dims then is 4 x NR columns of TMEM (256 of 512 for 64 rows; with
// rows as M it would be all of it), a key tile is brought in once for both
// products, and the rows that do not fill M = 128 cost nothing.
//
//   warps 0-3  the softmax: S by 16x256b loads (a thread has 16 keys of two rows),
//              running maximum and sums in registers, P to shared memory. O^T is
//              rescaled only when a row's maximum grew by 2^8 or more. They also
//              bring the queries in and write the outputs.
//   warp  4    issues the products S, up to four tiles ahead of
//   warp  6    P V (a product takes 31 clocks to issue and 25 to 48 to run: one warp for both was the bound).
//   warp  5    cuts the work: finds the CTA's next items and hands them to the others.
//   others     bring the tiles: 16-bit rows by TMA, a box for each 64 dims and
//              run of keys within a page, where all 64 keys exist, else by cp.async; e4m3fn rows
//              through registers, a tile ahead, as fp16 (exact).
//   A stage (tile) is waited for in chunks of 64 dims, so that S follows the copies,
//   and given back by 128 dims, as P V goes over them: two stages of 576 dims and the
//   queries fill the shared memory.
//
// Weights are rounded once to 16 bits, as the product's operand; their sums are
// of the unrounded ones in fp32. An e4m3fn row's scale f multiplies its scores,
// and its weights p before they are rounded: the running reference is the
// maximum of score + log2 f, so that p f, not p, begins at 2^7.
//
// Few long sequences are split over the CTAs by keys, in steps of a tile, counted
// on the device: one share for each CTA and smaller ones for those that are done first;
// parts are joined in the order of the keys by a second kernel.
//
// Every wait has a limit (kSpin); a CTA whose wait ran out records that in the
// error record and in the workspace's head, lets its copies and products end and leaves.
#pragma once

#include "kv_attend_latent.cuh"
#include "kv_attend_tile.cuh"

namespace kvimpl {

constexpr int kLatKeys = 32;        // keys of a tile
constexpr int kLatChunk = kLatKeys * 128;  // bytes of its keys x 64 dims of 16 bits
constexpr int kLatMaxChunks = 9;    // row dims up to 576
constexpr int kLatMaxStages = 8;
constexpr int kLatScores = 4;       // tiles whose scores may be in TMEM

struct LatentTileParams {
  LatentParams l;
  CUtensorMap map;
  int32_t box;       // keys of a TMA box; 0: no TMA
  int32_t page_stride, slot_stride;  // of the cache, bytes in 32 bits
  int32_t chunks;    // 64-dim chunks of a row, the last perhaps cut
  int32_t ksteps;    // 16-dim steps of a row
  int32_t blocks;    // 128-dim blocks of the values
  int32_t stages;
  int32_t split;     // 0: an item is one CTA's
  int32_t min_steps, max_shares;
  int32_t part_rows;
  SplitWork* head;
  int64_t* meta;     // [num_seqs]: first step of each sequence
  float *part_o, *part_ml;  // [2 * max_shares][part_rows] x 128 * blocks and x 2
};

// Loader warps: e4m3fn rows are converted by them.
template <int FMT>
constexpr int kLatLoaders = FMT == KV_CACHE_SRC ? 4 : 8;
template <int FMT>
constexpr int kLatThreads = 32 * (7 + kLatLoaders<FMT>);

// A CTA's next piece of work.
struct LatentSeg {
  int32_t b, q0, nq, p_first;  // sequence, its first query row and their number, position of the first
  int32_t row0, nrows;         // rows of the item: (query, head) pairs of the sequence
  int32_t t0, t1;              // tiles
  int32_t part;                // -1: the item is whole; else the part's place
  int32_t stop;
};

template <int NR>
struct LatentSmem {  // behind the stages
  static constexpr int kP = NR * 128;
  static constexpr int kBars = 40;
  static constexpr int kSeg = 2;
  static __host__ __device__ constexpr int q_bytes(int chunks) { return chunks * NR * 128; }
  // offsets behind Q and P
  static constexpr int kOffBars = 0, kOffSegs = kOffBars + kBars * 8, kOffAlpha = kOffSegs + kSeg * 64,
                       kOffInv = kOffAlpha + 2 * NR * 4, kOffQf = kOffInv + NR * 4, kOffPlace = kOffQf + NR * 4,
                       kOffMisc = kOffPlace + kLatKeys * 8, kOffValid = kOffMisc + 64, kOffScale = kOffValid + kLatMaxStages * 4;
  static __host__ __device__ constexpr int total(int chunks, int stages) {
    return stages * (chunks * kLatChunk + kLatKeys * 4) + q_bytes(chunks) + kP + kOffScale;
  }
};
static_assert(sizeof(LatentSeg) <= 64, "segments");
static_assert(LatentSmem<64>::total(kLatMaxChunks, 4) <= 227 * 1024, "four stages of the widest rows fit");
static_assert(2 * kLatMaxStages + 2 * kLatScores + 12 <= LatentSmem<64>::kBars, "barriers");

// Rows of the sequence's queries in blocks of NR, and tiles of each (an upper bound, at least one).
struct LatentGeom {
  int32_t blocks, steps;
};

template <int NR>
__device__ __forceinline__ LatentGeom latent_geom(const AttendParams& a, const AttendSeq& s) {
  LatentGeom g;
  g.blocks = static_cast<int32_t>((static_cast<uint32_t>(s.nq) * a.group.d + NR - 1) / NR);
  g.steps = max((s.len + kLatKeys - 1) / kLatKeys, 1);
  return g;
}

template <int NR>
__device__ __forceinline__ int64_t latent_units(const LatentTileParams& p, int32_t b, bool record) {
  const LatentGeom g = latent_geom<NR>(p.l.a, attend_seq(p.l.a, b, record));
  return static_cast<int64_t>(g.blocks) * (p.split ? g.steps : 1);
}

// One share of 88 % of an equal part for each CTA, and the rest in shares of a quarter of what is left for each.
constexpr int kLatFirst = 88;

__device__ __forceinline__ int32_t latent_cut(int64_t total, int32_t ctas, int32_t max_shares, int32_t min_steps, ShareLevel (&level)[2],
                                              int32_t* shares) {
  int64_t each = (total + ctas - 1) / ctas;
  if (each < min_steps) each = min_steps;
  const int64_t size = each * kLatFirst / 100, left = total - size * ctas;
  int64_t small = (left + 2 * ctas - 1) / (2 * ctas);
  if (small < min_steps) small = min_steps;
  if (left <= 0 || each < 6 * min_steps || max_shares < ctas + (left + small - 1) / small) {
    level[0] = ShareLevel{0, static_cast<int32_t>(each), 0};
    *shares = static_cast<int32_t>((total + each - 1) / each);
    return 1;
  }
  level[0] = ShareLevel{0, static_cast<int32_t>(size), 0};
  level[1] = ShareLevel{size * ctas, static_cast<int32_t>(small), ctas};
  *shares = ctas + static_cast<int32_t>((left + small - 1) / small);
  return 2;
}

// 16 lanes x 32 columns over the warp: thread (g, t) = (lane / 4, lane % 4) gets columns 8 i + 2 t, + 1 of
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

// N products D (TMEM) = or += A B (shared memory), by a whole, converged warp as tc_mma_ss: the operands' descriptors
// step by AS and BS (in 16 bytes), whose low words alone change.  One election for all, and no carries: a product then
// takes 31 clocks to issue, 40 each on its own.
template <int N, int AS, int BS>
__device__ __forceinline__ void tc_mma_run(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  static_assert(N == 2 || N == 4, "products");
  const uint32_t al = static_cast<uint32_t>(a), ah = static_cast<uint32_t>(a >> 32), bl = static_cast<uint32_t>(b), bh = static_cast<uint32_t>(b >> 32);
#define KV_FIRST "{\n\t.reg .pred e, p;\n\t.reg .b64 x, y;\n\t.reg .b32 u, v;\n\telect.sync _|e, 0xFFFFFFFF;\n\tsetp.ne.b32 p, %6, 0;\n\t" \
  "mov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %4};\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, p;\n\t"
#define KV_NEXT(i, j) "add.u32 u, %1, %" #i ";\n\tadd.u32 v, %3, %" #j ";\n\tmov.b64 x, {u, %2};\n\tmov.b64 y, {v, %4};\n\t" \
  "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, 1;\n\t"
  if constexpr (N == 4) {
    asm volatile(KV_FIRST KV_NEXT(7, 8) KV_NEXT(9, 10) KV_NEXT(11, 12) "}"
                 ::"r"(d), "r"(al), "r"(ah), "r"(bl), "r"(bh), "r"(idesc), "r"(acc ? 1u : 0u), "n"(AS), "n"(BS), "n"(2 * AS), "n"(2 * BS), "n"(3 * AS), "n"(3 * BS)
                 : "memory");
  } else {
    asm volatile(KV_FIRST KV_NEXT(7, 8) "}"
                 ::"r"(d), "r"(al), "r"(ah), "r"(bl), "r"(bh), "r"(idesc), "r"(acc ? 1u : 0u), "n"(AS), "n"(BS) : "memory");
  }
#undef KV_FIRST
#undef KV_NEXT
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
template <int FMT, int NR, bool kBF16>
__global__ void __launch_bounds__(kLatThreads<FMT>, 1) kv_attend_latent_tile(const __grid_constant__ LatentTileParams p) {
  using S = LatentSmem<NR>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const LatentParams& lp = p.l;
  const AttendParams& a = lp.a;
  const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31u;
  // (no static shared memory: the dynamic part begins at a multiple of 1,024, which the swizzle wants)
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem_raw));
  const int32_t HQ = static_cast<int32_t>(a.group.d);
  const uint32_t stage_bytes = static_cast<uint32_t>(p.chunks) * kLatChunk;
  const uint32_t q_at = ring + static_cast<uint32_t>(p.stages) * stage_bytes;
  const uint32_t p_at = q_at + static_cast<uint32_t>(S::q_bytes(p.chunks));
  const uint32_t small = p_at + S::kP;
  uint8_t* const small_ptr = smem_raw + (small - ring);
  const uint32_t full = small + S::kOffBars, empty = full + 8 * kLatMaxStages, q_full = empty + 8 * kLatMaxStages, s_full = q_full + 8,
                 s_free = s_full + 8 * kLatScores, p_full = s_free + 8 * kLatScores, pv_done = p_full + 16, seg_full = pv_done + 16, seg_empty = seg_full + 16, done = seg_empty + 16,
                 load_bar = done + 16;
  LatentSeg* const segs = reinterpret_cast<LatentSeg*>(small_ptr + S::kOffSegs);
  float* const sh_alpha = reinterpret_cast<float*>(small_ptr + S::kOffAlpha);   // [2][NR]
  float* const sh_inv = reinterpret_cast<float*>(small_ptr + S::kOffInv);
  float* const sh_qf = reinterpret_cast<float*>(small_ptr + S::kOffQf);
  int64_t* const sh_place = reinterpret_cast<int64_t*>(small_ptr + S::kOffPlace);
  float* const sh_scale = reinterpret_cast<float*>(small_ptr + S::kOffScale);   // [stages][kLatKeys]
  uint32_t* const sh_valid = reinterpret_cast<uint32_t*>(small_ptr + S::kOffValid);  // of a stage's keys, a bit each
  WaitState* const state = reinterpret_cast<WaitState*>(small_ptr + S::kOffMisc);
  uint32_t* const sh_tmem = reinterpret_cast<uint32_t*>(small_ptr + S::kOffMisc + 16);
  unsigned long long* const sh_bad = reinterpret_cast<unsigned long long*>(small_ptr + S::kOffMisc + 24);
  constexpr int kLoaders = kLatLoaders<FMT>;

  if (warp == 4) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
        static_cast<uint32_t>(__cvta_generic_to_shared(sh_tmem))) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    for (int i = 0; i < p.stages; ++i) {
      bar_init(full + 8 * i, 1);
      bar_init(empty + 8 * i, 1);
    }
    bar_init(q_full, 128);
    for (int i = 0; i < kLatScores; ++i) {
      bar_init(s_full + 8 * i, 1);
      bar_init(s_free + 8 * i, NR / 16);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(p_full + 8 * i, 128);
      bar_init(pv_done + 8 * i, 1);
      bar_init(seg_full + 8 * i, 1);
      bar_init(seg_empty + 8 * i, 6 + kLoaders);
    }
    bar_init(done, 1);
    bar_init(done + 8, 1);
    bar_init(load_bar, kLoaders);
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
  const uint32_t tm_s = tmem + 4 * NR;  // S, kLatScores buffers of kLatKeys columns, behind O^T

  if (warp < 4) {
    // ======================================================================================
    // the softmax
    // ======================================================================================
    const uint32_t g = lane >> 2, t = lane & 3u;
    const bool has_rows = warp < NR / 16;
    const int32_t r0 = static_cast<int32_t>(16u * warp + g);  // and r0 + 8
    const uint32_t lanes = warp << 21;
    const uint32_t flip = a.scale_log2 < 0.0f ? 0x80008000u : 0u;  // the maximum is taken before the scale
    constexpr float kSmall = kBF16 ? 0.0f : 7.0f;
    // Queries into shared memory: a warp has NR / 4 rows, four at a time. (All products that read the
    // last ones have ended, as their scores were waited for.)
    auto load_q = [&](const LatentSeg& s) {
      constexpr int kRows = NR / 4, kAt = 4, kPer = (kLatMaxChunks * 8 + 31) / 32;
      const uint32_t pieces = static_cast<uint32_t>(a.head_dim) / 8u;
      for (int i0 = 0; i0 < kRows; i0 += kAt) {
        uint4 w[kAt][kPer];
#pragma unroll
        for (int y = 0; y < kAt; ++y) {
          const int32_t r = static_cast<int32_t>(warp) * kRows + i0 + y;
          const bool live = r < s.nrows;
          const int32_t qi = static_cast<int32_t>(a.group.quot(static_cast<uint32_t>(s.row0 + (live ? r : 0))));
          const int32_t h = s.row0 + (live ? r : 0) - qi * HQ;
          const uint8_t* src = a.q + static_cast<int64_t>(s.q0 + qi) * a.q_token + static_cast<int64_t>(h) * a.q_head;
#pragma unroll
          for (int x = 0; x < kPer; ++x) {
            const uint32_t piece = lane + 32u * x;
            w[y][x] = make_uint4(0u, 0u, 0u, 0u);
            if (live && piece < pieces) w[y][x] = __ldg(reinterpret_cast<const uint4*>(src + 16u * piece));
          }
        }
#pragma unroll
        for (int y = 0; y < kAt; ++y) {
          const uint32_t r = warp * kRows + i0 + y;
          if constexpr (FMT != KV_CACHE_SRC) {
            float f = 1.0f;
            if (a.bf16) {  // into fp16's range: the row's largest element to 2^13 .. 2^14
              uint32_t m = 0u;
#pragma unroll
              for (int x = 0; x < kPer; ++x)
                m = absmax_pair<true>(absmax_pair<true>(absmax_pair<true>(absmax_pair<true>(m, w[y][x].x), w[y][x].y), w[y][x].z), w[y][x].w);
              const uint32_t e = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(absmax_pair_value<true>(m))) >> 23;
              f = __uint_as_float(min(254u, 267u - e) << 23);
              auto shift = [&](uint32_t z) {
                const float2 v = widen2<true>(z);
                return pack2(v.x * f, v.y * f, false);
              };
#pragma unroll
              for (int x = 0; x < kPer; ++x)
                w[y][x] = make_uint4(shift(w[y][x].x), shift(w[y][x].y), shift(w[y][x].z), shift(w[y][x].w));
            }
            if (lane == 0u) sh_qf[r] = __fdiv_rn(1.0f, f);
          }
#pragma unroll
          for (int x = 0; x < kPer; ++x) {
            const uint32_t piece = lane + 32u * x;
            if (piece < pieces)
              st_shared16(q_at + (piece >> 3) * (NR * 128u) + r * 128u + (((piece & 7u) ^ (r & 7u)) << 4), w[y][x].x ^ flip,
                          w[y][x].y ^ flip, w[y][x].z ^ flip, w[y][x].w ^ flip);
          }
        }
      }
      fence_async_shared();
      bar_arrive(q_full);
      sync_softmax();  // sh_qf
    };
    uint32_t k = 0u, T = 0u;  // segments and tiles that went by
    uint32_t stage = 0u, phase = 0u;
    LatentSeg seg, next;
    bool have = take(k++, &seg);
    const bool lost = any_of_softmax(!ok);
    if (!lost && have && seg.t1 > seg.t0) load_q(seg);
    while (!lost && have) {
      const int32_t pos[2] = {seg.p_first + static_cast<int32_t>(a.group.quot(static_cast<uint32_t>(seg.row0 + min(r0, seg.nrows - 1)))),
                              seg.p_first + static_cast<int32_t>(a.group.quot(static_cast<uint32_t>(seg.row0 + min(r0 + 8, seg.nrows - 1))))};
      const int32_t p_lo = seg.p_first + static_cast<int32_t>(a.group.quot(static_cast<uint32_t>(seg.row0)));
      float rs[2], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        rs[c] = fabsf(a.scale_log2);
        if constexpr (FMT != KV_CACHE_SRC) rs[c] *= has_rows ? sh_qf[r0 + 8 * c] : 1.0f;
        if (rs[c] == 0.0f) rs[c] = __uint_as_float(1u);  // hidden scores (-inf) must stay -inf
      }
      for (int32_t j = seg.t0; j < seg.t1; ++j, ++T) {
        ok = ok && __all_sync(0xFFFFFFFFu, bar_wait(full + 8 * stage, phase, state));
        const uint32_t valid = sh_valid[stage];
        ok = ok && __all_sync(0xFFFFFFFFu, bar_wait(s_full + 8 * (T % kLatScores), (T / kLatScores) & 1u, state));
        tc_fence_after();
        float s[16], kf[8], alpha[2] = {1.0f, 1.0f};  // scores, their keys' scales, factors of the rows' sums
        bool grew = false;
        if (has_rows && ok) {
          tc_ld_rows(s, tm_s + kLatKeys * (T % kLatScores) + lanes);
          tc_fence_before();
          if (lane == 0u) bar_arrive(s_free + 8 * (T % kLatScores));
          if constexpr (FMT != KV_CACHE_SRC) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 f = *reinterpret_cast<const float2*>(sh_scale + stage * kLatKeys + 8 * i + 2 * t);
              kf[2 * i] = f.x;
              kf[2 * i + 1] = f.y;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] *= kf[2 * (i / 4) + (i & 1)] * rs[(i >> 1) & 1];
          }
          if (j * kLatKeys + kLatKeys - 1 > p_lo || valid != ~0u) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int32_t n = pos[c] - j * kLatKeys + 1;  // the first n keys
              const uint32_t see = ((n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u) & valid) >> (2 * t);
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                  if ((see >> (8 * i + x) & 1u) == 0u) s[4 * i + 2 * c + x] = -INFINITY;
            }
          }
          float lv[8];
          if constexpr (FMT != KV_CACHE_SRC) {
#pragma unroll
            for (int i = 0; i < 8; ++i) lv[i] = fmaxf(lg2_fast(fabsf(kf[i])), -100.0f);
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float x[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int y = 0; y < 2; ++y) x[y] = fmaxf(x[y], FMT == KV_CACHE_SRC ? s[4 * i + 2 * c + y] : s[4 * i + 2 * c + y] + lv[2 * i + y]);
            float top = fmaxf(x[0], x[1]);
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            top = FMT == KV_CACHE_SRC ? __fmaf_rn(top, rs[c], -kSmall) : top - kSmall;
            // a maximum that grew little is kept (the weights stay below 2^(kSmall + 8))
            if (top > m[c] + 8.0f || (m[c] == -INFINITY && top > m[c])) {
              alpha[c] = exp2_fast(m[c] - top);
              m[c] = top;
              grew = true;
            }
          }
          if (t == 0u) {
            sh_alpha[(T & 1u) * NR + r0] = alpha[0];
            sh_alpha[(T & 1u) * NR + r0 + 8] = alpha[1];
          }
        }
        // O^T is all warps': whether any row of the CTA grew
        const bool rescale = any_of_softmax((grew && j > seg.t0) || !ok);
        if (rescale && any_of_softmax(!ok)) {  // (a warp that gave up still comes here: all leave together)
          ok = false;
          break;
        }
        uint32_t pw[8];
        if (has_rows) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float ref = m[c] == -INFINITY ? 0.0f : m[c];
            float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float2 z = make_float2(s[4 * i + 2 * c], s[4 * i + 2 * c + 1]);
              if constexpr (FMT == KV_CACHE_SRC) z = fma2(z, rs[c], -ref); else z = add2(z, make_float2(-ref, -ref));
              float2 e = make_float2(exp2_fast(z.x), exp2_fast(z.y));
              sum[i & 1] = add2(sum[i & 1], e);
              if constexpr (FMT != KV_CACHE_SRC) {
                e.x *= kf[2 * i];
                e.y *= kf[2 * i + 1];
              }
              pw[2 * i + c] = pack2(e.x, e.y, kBF16);
            }
            sum[0] = add2(sum[0], sum[1]);
            l[c] = __fmaf_rn(l[c], alpha[c], sum[0].x + sum[0].y);
          }
        }
        if (T > 1u)  // P V of the last tile but one has read its P
          ok = __all_sync(0xFFFFFFFFu, bar_wait(pv_done + 8 * (T & 1u), ((T >> 1) - 1u) & 1u, state));
        if (rescale && ok) {  // and that of the last one has written O^T
          ok = __all_sync(0xFFFFFFFFu, bar_wait(pv_done + 8 * ((T - 1u) & 1u), ((T - 1u) >> 1) & 1u, state));
          tc_fence_after();
          const float* f = sh_alpha + (T & 1u) * NR;
          for (int32_t b = 0; b < p.blocks; ++b)
#pragma unroll 1
            for (int c = 0; c < NR / 16; ++c) {
              uint32_t w[16];
              tc_ld16(w, tmem + lanes + b * NR + 16 * c);
#pragma unroll
              for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * f[16 * c + i]);
              tc_st16(tmem + lanes + b * NR + 16 * c, w);
            }
          tc_wait_st();
        }
        if (has_rows && ok) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t r = static_cast<uint32_t>(r0 + 8 * c);
#pragma unroll
            for (int i = 0; i < 4; ++i)  // tiles take turns in the halves of P's rows
              asm volatile("st.shared.u32 [%0], %1;" ::"r"(p_at + r * 128u + (((i + 4u * (T & 1u)) ^ (r & 7u)) << 4) + 4u * t), "r"(pw[2 * i + c]) : "memory");
          }
        }
        fence_async_shared();
        tc_fence_before();
        bar_arrive(p_full + 8 * (T & 1u));
        if (++stage == static_cast<uint32_t>(p.stages)) {
          stage = 0u;
          phase ^= 1u;
        }
      }
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
        if (has_rows && t == 0u) sh_inv[r0 + 8 * c] = l[c] < INFINITY ? __fdiv_rn(1.0f, l[c]) : NAN;
      }
      if (live) {
        ok = __all_sync(0xFFFFFFFFu, bar_wait(pv_done + 8 * ((T - 1u) & 1u), ((T - 1u) >> 1) & 1u, state));
        tc_fence_after();
      }
      if (any_of_softmax(!ok)) break;
      const int32_t L = lp.latent;
      if (seg.part < 0) {
        unsigned long long bad = 0ull;
        for (int32_t b = 0; b < p.blocks; ++b) {
          const int32_t d = 128 * b + static_cast<int32_t>(tid);
          for (int32_t c = 0; 16 * c < seg.nrows; ++c) {
            uint32_t w[16];
            if (live) {
              tc_ld16(w, tmem + lanes + b * NR + 16 * c);
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) w[i] = 0u;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int32_t r = 16 * c + i;
              if (r >= seg.nrows) break;
              const int32_t qi = static_cast<int32_t>(a.group.quot(static_cast<uint32_t>(seg.row0 + r))), h = seg.row0 + r - qi * HQ;
              uint16_t* out = reinterpret_cast<uint16_t*>(a.out + static_cast<int64_t>(seg.q0 + qi) * a.o_token + static_cast<int64_t>(h) * a.o_head);
              const float v = live ? __uint_as_float(w[i]) * sh_inv[r] : 0.0f;
              if (d < L) {
                if (!(fabsf(v) < INFINITY)) bad |= 1ull << r;
                out[d] = round16(v, a.bf16);
              }
            }
          }
        }
        const uint32_t lo = __reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(bad)), hi = __reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(bad >> 32));
        if (lane == 0u && (lo | hi) != 0u) atomicOr(sh_bad, static_cast<unsigned long long>(hi) << 32 | lo);
        sync_softmax();
        unsigned long long again = *const_cast<volatile unsigned long long*>(sh_bad);
        if (a.lse && has_rows && t == 0u) {
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
            attend_latent_row<FMT, 18>(lp, seg.b, seg.p_first + qi, seg.q0 + qi, h, 0, L);
          }
          if (lane == 0u) state->hold(-1);
          sync_softmax();
          if (tid == 0u) *sh_bad = 0ull;
        }
      } else {
        const int64_t at = static_cast<int64_t>(seg.part) * p.part_rows;
        const int32_t width = 128 * p.blocks;
        for (int32_t b = 0; b < p.blocks; ++b)
          for (int32_t c = 0; 16 * c < seg.nrows; ++c) {
            uint32_t w[16];
            if (live) {
              tc_ld16(w, tmem + lanes + b * NR + 16 * c);
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) w[i] = 0u;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (16 * c + i < seg.nrows) p.part_o[(at + 16 * c + i) * width + 128 * b + tid] = __uint_as_float(w[i]);
          }
        if (has_rows && t == 0u) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
            if (r0 + 8 * c < seg.nrows) *reinterpret_cast<float2*>(p.part_ml + (at + r0 + 8 * c) * 2) = make_float2(m[c], l[c]);
        }
      }
      tc_fence_before();
      seg = next;
    }
  } else if (warp == 4 || warp == 6) {
    // ======================================================================================
    // the products: warp 4 S = Q K^T, warp 6 O^T += V^T P^T
    // ======================================================================================
    auto wait = [&](uint32_t bar, uint32_t parity) {
      if (ok) ok = __all_sync(0xFFFFFFFFu, bar_wait(bar, parity, state));
      tc_fence_after();
    };
    // Descriptors and addresses are to be in uniform registers: a reduction's result is in one, loops end by the
    // parameters alone, and products stand in straight lines. (Of the 36 + 8 products of a tile of 576 / 512 dims each takes
    // 25 to 48 clocks to run; with descriptors in any register 70 to 140 to issue.)
    auto same = [](uint32_t x) { return __reduce_or_sync(0xFFFFFFFFu, x); };
    const uint32_t ring0 = same(ring);
    uint32_t k = 0u, T = 0u, stage = 0u, phase = 0u;
    LatentSeg seg;
    auto advance = [&] {
      ++T;
      if (++stage == static_cast<uint32_t>(p.stages)) {
        stage = 0u;
        phase ^= 1u;
      }
    };
    if (warp == 4) {
      const uint32_t desc = (1u << 4) | (kBF16 ? 1u << 7 | 1u << 10 : 0u) | ((static_cast<uint32_t>(kLatKeys) >> 3) << 17) | ((64u >> 4) << 24);
      const uint32_t s_at = same(tm_s);
      const uint64_t q_desc = smem_desc(same(q_at), 16);
      uint32_t items = 0u;
      while (take(k++, &seg)) {
        if (seg.t1 <= seg.t0) continue;
        wait(q_full, items++ & 1u);
        for (int32_t j = seg.t0; j < seg.t1; ++j) {
          const uint32_t u = same(stage | (T % kLatScores) << 8), st = u & 255u, buf = u >> 8;
          const uint64_t kd = smem_desc(ring0 + st * stage_bytes, 16);
          const uint32_t d = s_at + kLatKeys * buf;
          if (T >= kLatScores) wait(s_free + 8 * (T % kLatScores), (T / kLatScores - 1u) & 1u);
          wait(full + 8 * stage, phase);
          if (!ok) break;
          auto chunk = [&](int32_t c) {
            tc_mma_run<4, 2, 2>(d, q_desc + c * (NR * 128 >> 4), kd + c * (kLatChunk >> 4), desc, c > 0);
          };
#pragma unroll
          for (int c = 0; c < kLatMaxChunks; c += 3) {
            if (p.ksteps >= 4 * c + 12) {
              chunk(c); chunk(c + 1); chunk(c + 2);
            } else {
#pragma unroll 1
              for (int32_t y = c; 4 * y + 4 <= p.ksteps; ++y) chunk(y);
              if (p.ksteps >= 4 * c)
#pragma unroll 1
                for (int32_t i = p.ksteps & ~3; i < p.ksteps; ++i)
                  tc_mma_ss(d, q_desc + ((i / 4) * (NR * 128 >> 4) + (i % 4) * 2), kd + ((i / 4) * (kLatChunk >> 4) + (i % 4) * 2), desc, i > 0);
              break;
            }
          }
          tc_commit(s_full + 8 * buf);
          advance();
        }
        if (!ok) break;
      }
    } else {
      const uint32_t desc = (1u << 4) | (kBF16 ? 1u << 7 | 1u << 10 : 0u) | (1u << 15) | ((static_cast<uint32_t>(NR) >> 3) << 17) | ((128u >> 4) << 24);
      const uint32_t o_at = same(tmem), free0 = same(empty);
      const uint64_t p_desc = smem_desc(same(p_at), 16);
      while (take(k++, &seg)) {
        for (int32_t j = seg.t0; j < seg.t1; ++j) {
          const uint32_t u = same(stage | (T & 1u) << 8 | (j > seg.t0 ? 512u : 0u)), st = u & 255u, odd = u >> 8 & 1u, old = u >> 9;
          const uint64_t v = smem_desc(ring0 + st * stage_bytes, kLatChunk), pd = p_desc + 4 * odd;
          wait(full + 8 * stage, phase);
          wait(p_full + 8 * (T & 1u), (T >> 1) & 1u);
          if (!ok) break;
          auto block = [&](int32_t b) {
            tc_mma_run<kLatKeys / 16, (2048 >> 4), 2>(o_at + b * NR, v + b * (2 * kLatChunk >> 4), pd, desc, old != 0u);
          };
          if (p.blocks == 4) {
            block(0); block(1); block(2); block(3);
          } else {
#pragma unroll 1
            for (int32_t b = 0; b < p.blocks; ++b) block(b);
          }
          tc_commit(free0 + 8 * st);
          tc_commit(pv_done + 8 * odd);
          advance();
        }
        if (!ok) break;
      }
    }
    if (!ok) {  // products still in flight read shared memory and write TMEM: let them end
      const uint32_t bar = warp == 4 ? done : done + 8;
      tc_commit(bar);
      for (uint32_t i = 0; i < kSpin && !bar_try(bar, 0); ++i) {}
    }
    __syncwarp();
  } else if (warp == 5) {
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
    ShareLevel level[2] = {};
    int32_t shares = 0, levels = 1;
    const int32_t ctas = static_cast<int32_t>(gridDim.x);
    if (p.split) {
      levels = latent_cut(total, ctas, p.max_shares, p.min_steps, level, &shares);
      if (blockIdx.x == 0 && lane == 0u) {
        p.head->level[0] = level[0];
        p.head->level[1] = level[1];
        p.head->levels = levels;
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
    int32_t share = static_cast<int32_t>(blockIdx.x);
    while (ok) {
      int64_t pos, end;
      if (p.split) {
        if (share >= shares) break;
        const int32_t lv = levels > 1 && share >= level[1].first ? 1 : 0;
        pos = level[lv].start + static_cast<int64_t>(share - level[lv].first) * level[lv].size;
        end = min(lv + 1 < levels ? level[1].start : total, pos + level[lv].size);
      } else {  // items in turn, every second round the other way
        pos = static_cast<int64_t>(round) * ctas + ((round & 1) ? ctas - 1 - static_cast<int32_t>(blockIdx.x) : static_cast<int32_t>(blockIdx.x));
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
        const LatentGeom geom = latent_geom<NR>(a, seq);
        const int32_t unit = p.split ? geom.steps : 1;
        int32_t item = static_cast<int32_t>(local / unit);
        const int32_t s_in = static_cast<int32_t>(local - static_cast<int64_t>(item) * unit);
        const int32_t s_out = static_cast<int32_t>(min(static_cast<int64_t>(unit), s_in + (end - pos)));
        pos += s_out - s_in;
        if (!p.split) item = geom.blocks - 1 - item;  // the last queries, which see the most keys, first
        s.q0 = seq.q0;
        s.nq = seq.nq;
        s.p_first = seq.len - seq.nq;
        s.row0 = item * NR;
        s.nrows = min(NR, seq.nq * HQ - s.row0);
        const int32_t p_hi = s.p_first + static_cast<int32_t>(a.group.quot(static_cast<uint32_t>(s.row0 + s.nrows - 1)));
        const int32_t tiles = p_hi < 0 ? 0 : p_hi / kLatKeys + 1;
        s.t0 = p.split ? min(s_in, tiles) : 0;
        s.t1 = p.split ? min(s_out, tiles) : tiles;
        s.part = s_out - s_in == unit ? -1 : 2 * share + (s_in == 0 ? 1 : 0);
        publish(s);
      }
      if (p.split) {
        int32_t after = 0;
        if (lane == 0u) after = static_cast<int32_t>(gridDim.x + atomicAdd(&p.head->next, 1u));
        share = __shfl_sync(0xFFFFFFFFu, after, 0);
      }
    }
    LatentSeg s = {};
    s.stop = 1;
    publish(s);
  } else {
    // ======================================================================================
    // the tiles
    // ======================================================================================
    constexpr uint32_t kN = 32u * kLoaders;
    const uint32_t lt = tid - 7u * 32u;  // of the loaders
    uint32_t k = 0u, T = 0u, stage = 0u, phase = 0u;
    LatentSeg seg;
    // the stage is free: all that read it has ended
    auto wait_empty = [&] {
      if (ok && T >= static_cast<uint32_t>(p.stages)) ok = __all_sync(0xFFFFFFFFu, bar_wait(empty + 8 * stage, phase ^ 1u, state));
    };
    auto advance = [&] {
      ++T;
      if (++stage == static_cast<uint32_t>(p.stages)) {
        stage = 0u;
        phase ^= 1u;
      }
    };
    // the loaders wait for one another, with the limit of all waits
    uint32_t syncs = 0u;
    auto sync_loaders = [&] {
      __syncwarp();
      if (lane == 0u) bar_arrive(load_bar);
      ok = ok && __all_sync(0xFFFFFFFFu, bar_wait(load_bar, syncs++ & 1u, state));
    };
    const uint32_t per_row = static_cast<uint32_t>(a.head_dim) / (FMT == KV_CACHE_SRC ? 8u : 16u);  // 16-byte pieces
    while (take(k++, &seg)) {
      const int32_t* table = a.table + static_cast<int64_t>(seg.b) * a.table_stride;
      const int32_t p_hi = seg.p_first + static_cast<int32_t>(a.group.quot(static_cast<uint32_t>(seg.row0 + seg.nrows - 1)));
      // the page of key j of a tile (of its last key a row sees, for keys behind it)
      auto page_at = [&](int32_t j) { return __ldg(table + a.page.quot(static_cast<uint32_t>(min(j, p_hi)))); };
      // by the first loader warp, a key a lane: where its row lies (-1: no row needs it), into sh_place; the others do nothing
      auto place = [&](int32_t tile, int32_t id) {
        const int32_t j = tile * kLatKeys + static_cast<int32_t>(lt);
        const bool want = j <= p_hi, have = static_cast<uint32_t>(id) < static_cast<uint32_t>(a.num_pages);
        if (want && !have) record_oob(a.err, static_cast<uint64_t>(seg.b));
        const uint32_t off = static_cast<uint32_t>(j) - a.page.quot(static_cast<uint32_t>(j)) * a.page.d;
        sh_place[lt] = want && have ? wide(id, p.page_stride) + wide(off, p.slot_stride) : -1;
        return want && have ? off : 0xFFFFFFFFu;
      };
      if constexpr (FMT == KV_CACHE_SRC) {
        const int32_t boxes = p.box > 0 ? kLatKeys / p.box : 0;
        const uint32_t box_bytes = static_cast<uint32_t>(p.box) * 128u;
        // lane i: the page of the tile's i-th box; every loader warp knows whether all are there
        auto box_page = [&](int32_t tile) -> int32_t {
          if (tile >= seg.t1 || static_cast<int32_t>(lane) >= boxes) return 0;
          return page_at(tile * kLatKeys + static_cast<int32_t>(lane) * p.box);
        };
        int32_t next_box = box_page(seg.t0), next_id = seg.t0 < seg.t1 && lt < kLatKeys ? page_at(seg.t0 * kLatKeys + static_cast<int32_t>(lt)) : 0;
        for (int32_t tile = seg.t0; tile < seg.t1 && ok; ++tile) {
          const int32_t page = next_box, id = next_id;
          next_box = box_page(tile + 1);
          if (lt < kLatKeys && tile + 1 < seg.t1) next_id = page_at((tile + 1) * kLatKeys + static_cast<int32_t>(lt));
          const bool whole = boxes > 0 && tile * kLatKeys + kLatKeys - 1 <= p_hi &&
                             __all_sync(0xFFFFFFFFu, static_cast<int32_t>(lane) >= boxes || (page >= 0 && page < a.num_pages));
          if (whole) {
            const uint32_t key = static_cast<uint32_t>(tile * kLatKeys + static_cast<int32_t>(lane) * p.box);
            const int32_t in_page = static_cast<int32_t>(key - a.page.quot(key) * a.page.d);
            wait_empty();
            if (ok && lt < 32u) {
              const uint32_t bar = full + 8 * stage;
              if (lane == 0u) {
                sh_valid[stage] = ~0u;
                bar_arrive_expect(bar, stage_bytes);
              }
              __syncwarp();
              if (static_cast<int32_t>(lane) < boxes)
                for (int32_t c = 0; c < p.chunks; ++c)
                  tma_box(ring + stage * stage_bytes + c * kLatChunk + lane * box_bytes, &p.map, bar, 64 * c, in_page, 0, page);
            }
          } else {
            wait_empty();
            if (lt < kLatKeys) {
              const bool have = place(tile, id) != 0xFFFFFFFFu;
              const uint32_t bits = __ballot_sync(0xFFFFFFFFu, have);
              if (lane == 0u && ok) sh_valid[stage] = bits;
            }
            sync_loaders();
            const uint32_t at = ring + stage * stage_bytes;
            if (ok)
              for (uint32_t i = lt; i < kLatKeys * per_row; i += kN) {
                const uint32_t key = i / per_row, piece = i - key * per_row;
                const int64_t off = sh_place[key];
                copy_async<16>(at + (piece >> 3) * kLatChunk + key * 128u + (((piece & 7u) ^ (key & 7u)) << 4),
                               a.k + (off < 0 ? 0 : off + 16 * piece), off < 0 ? 0u : 16u);
              }
            wait_all_async();
            fence_async_shared();
            sync_loaders();
            if (lt == 0u && ok) bar_arrive(full + 8 * stage);
          }
          if (ok) advance();
        }
      } else {
        constexpr int kPer = (kLatKeys * kLatMaxChunks * 4 + static_cast<int>(kN) - 1) / static_cast<int>(kN);  // pieces of a thread
        const uint32_t pieces = kLatKeys * per_row;
        uint4 w[2][kPer];
        float sc[2] = {0.0f, 0.0f};
        uint32_t have[2] = {0u, 0u};
        int32_t next_id = seg.t0 < seg.t1 && lt < kLatKeys ? page_at(seg.t0 * kLatKeys + static_cast<int32_t>(lt)) : 0;
        auto load = [&](int32_t tile, uint4 (&v)[kPer], float* scale, uint32_t* bits) {
          sync_loaders();  // sh_place has been read
          if (lt < kLatKeys) {
            const int32_t id = next_id;
            if (tile + 1 < seg.t1) next_id = page_at((tile + 1) * kLatKeys + static_cast<int32_t>(lt));
            const uint32_t off = place(tile, id);
            *scale = 0.0f;
            if (off != 0xFFFFFFFFu) *scale = row_scale(lp, id, off);
            *bits = __ballot_sync(0xFFFFFFFFu, off != 0xFFFFFFFFu);
          }
          sync_loaders();
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const uint32_t n = lt + i * kN, key = n / per_row, piece = n - key * per_row;
            v[i] = make_uint4(0u, 0u, 0u, 0u);
            if (n < pieces) {
              const int64_t off = sh_place[key];
              if (off >= 0) v[i] = __ldg(reinterpret_cast<const uint4*>(a.k + off + 16 * piece));
            }
          }
        };
        auto put = [&](const uint4 (&v)[kPer], float scale, uint32_t bits) {
          wait_empty();
          const uint32_t at = ring + stage * stage_bytes;
          if (ok) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
              const uint32_t n = lt + i * kN, key = n / per_row, piece = n - key * per_row;
              if (n < pieces) {
                const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                uint32_t f[8];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  f[2 * y] = f16x2_from_e4m3x2(x[y]);
                  f[2 * y + 1] = f16x2_from_e4m3x2(x[y] >> 16);
                }
                // pieces of two neighbouring chunks take turns, so that eight lanes meet all banks
                const uint32_t row = at + (piece >> 2) * kLatChunk + key * 128u, first = piece >> 2 & 1u;
                const uint32_t at0 = row + (((2u * (piece & 3u) + first) ^ (key & 7u)) << 4), at1 = row + (((2u * (piece & 3u) + 1u - first) ^ (key & 7u)) << 4);
                st_shared16(at0, first ? f[4] : f[0], first ? f[5] : f[1], first ? f[6] : f[2], first ? f[7] : f[3]);
                st_shared16(at1, first ? f[0] : f[4], first ? f[1] : f[5], first ? f[2] : f[6], first ? f[3] : f[7]);
              }
            }
            if (lt < kLatKeys) {
              sh_scale[stage * kLatKeys + lt] = scale;
              if (lane == 0u) sh_valid[stage] = bits;
            }
          }
          fence_async_shared();
          sync_loaders();
          if (lt == 0u && ok) bar_arrive(full + 8 * stage);
          if (ok) advance();
        };
        if (seg.t0 < seg.t1) load(seg.t0, w[0], &sc[0], &have[0]);
        for (int32_t tile = seg.t0; tile < seg.t1 && ok; tile += 2) {
          if (tile + 1 < seg.t1) load(tile + 1, w[1], &sc[1], &have[1]);
          put(w[0], sc[0], have[0]);
          if (tile + 1 < seg.t1) {
            if (tile + 2 < seg.t1) load(tile + 2, w[0], &sc[0], &have[0]);
            put(w[1], sc[1], have[1]);
          }
        }
      }
      if (!ok) break;
    }
    if (!ok) {  // copies in flight write shared memory: let them land before the CTA leaves it
      wait_all_async();
      for (int i = 0; i < 1000; ++i) __nanosleep(1000);
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
  if (blockIdx.x == 0 && threadIdx.x == 0) p.head->next = 0u;
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
      const LatentGeom geom = latent_geom<NR>(a, s);
      const int32_t row = (tok - s.q0) * a.q_heads + h, rb = row / NR;
      r = row - rb * NR;
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

constexpr int kLatMinSteps = 8;  // tiles of a share at least

template <int FMT, int NR, bool kBF16>
kv_status launch_latent_tile(LatentTileParams p, void* work, int64_t work_bytes, int64_t max_keys, cudaStream_t stream) {
  using S = LatentSmem<NR>;
  const AttendParams& a = p.l.a;
  auto* kernel = kv_attend_latent_tile<FMT, NR, kBF16>;
  constexpr int kMost = 227 * 1024;
  static SmemOptIn opt_in;
  kv_status st = opt_in(reinterpret_cast<const void*>(kernel), kMost);
  if (st != KV_OK) return st;
  int sms = 0;
  st = current_sm_count(&sms);
  if (st != KV_OK) return st;
  p.stages = 2;
  while (p.stages < kLatMaxStages && S::total(p.chunks, p.stages + 1) <= kMost) ++p.stages;
  const int64_t items = static_cast<int64_t>(a.num_q) * a.group.d / NR + a.num_seqs;  // at most
  const int64_t meta = (static_cast<int64_t>(a.num_seqs) + 31) / 32 * 256;
  p.part_rows = a.q_start || static_cast<int32_t>(a.group.d) > NR ? NR : static_cast<int32_t>(a.group.d);
  const int64_t slot = static_cast<int64_t>(p.part_rows) * (128 * p.blocks + 2) * 4;
  int64_t fit = work && work_bytes > kSplitHead + meta ? (work_bytes - kSplitHead - meta) / (2 * slot) : 0;
  if (fit > 8 * sms) fit = 8 * sms;
  p.min_steps = kLatMinSteps;
  p.split = items < 4 * sms && max_keys > kLatMinSteps * kLatKeys && 2 * fit >= sms;
  int64_t grid = items < sms ? items : sms;
  if (p.split) {
    grid = fit < sms ? fit : sms;
    p.max_shares = static_cast<int32_t>(fit);
    p.head = static_cast<SplitWork*>(work);
    p.meta = reinterpret_cast<int64_t*>(static_cast<uint8_t*>(work) + kSplitHead);
    p.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(work) + kSplitHead + meta);
    p.part_ml = p.part_o + 2 * fit * p.part_rows * 128 * p.blocks;
  }
  st = launch_chained(kernel, grid, kLatThreads<FMT>, S::total(p.chunks, p.stages), stream, p);
  if (st != KV_OK || !p.split) return st;
  // the fewer the rows, the more parts has each and the more warps take it
  const int64_t units = static_cast<int64_t>(a.num_q) * a.q_heads * p.blocks;
  int32_t wpr = 1;
  while (wpr < kLatJoinWarps && units * wpr < 16ll * sms) wpr *= 2;
  const int64_t per = kLatJoinWarps / wpr;
  return launch_chained(kv_attend_latent_join<FMT, NR>, (units + per - 1) / per, 32 * kLatJoinWarps, 0, stream, p, wpr);
}

// The instantiations: 16-bit rows, and e4m3fn ones.
kv_status latent_tile_src(const LatentTileParams& p, bool few, void* work, int64_t work_bytes, int64_t max_keys, cudaStream_t stream);
kv_status latent_tile_e4m3(const LatentTileParams& p, bool few, void* work, int64_t work_bytes, int64_t max_keys, cudaStream_t stream);

}  // namespace kvimpl
