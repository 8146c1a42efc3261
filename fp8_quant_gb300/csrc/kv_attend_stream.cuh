// Attention for few query rows per sequence over much cache: the work and the
// products of kv_attend_split.cuh, fed by TMA.
//
// What bounds it is the memory's bandwidth, and what kept the cp.async form
// from it were the ends of shares (a CTA's ring ran empty there) and, for
// quantised caches, the instructions of the copies.  Here
//  * one warp per CTA does nothing but bring units (the K or the V rows of a
//    step: TW keys of every head of the CTA, or of `subs` neighbouring tiles where
//    there are few heads) into a ring, by one or two boxes a tile; it goes through the
//    CTA's shares without a stop and tells the others by a few words per step which
//    rows of which item a unit belongs to;
//  * eight other warps, one for each head or tile, only multiply.  A unit lies as [tile][box][128 bytes of a row][head][key] in
//    the swizzle of TMA; the lanes' pieces of a row are chosen so that the eight (or
//    sixteen) lanes that read together meet all banks: K pieces 2t and 2t + 1
//    of a 128-byte row for lane (g, t), V piece g of rows 2t.
//  * boxes in which no row sees a key (beside the sinks, before a window, behind
//    the last query) are not copied, nor are their pages looked up; other keys behind a
//    sequence's end are not hidden from TMA.  The scores of both are masked and
//    their V rows (e2m1: scales) are zeroed in shared memory, by the warp
//    that is about to use them.  Pages out of range are fetched as zeros.
//  * the products' loads and TMA's writes are accesses of different proxies: the copy
//    warp puts a fence between an empty unit's last arrival and its next box.
// Every wait has a limit; a CTA whose wait ran out records that, for the join too, and leaves.
//
// Measured on one GB300 (one query a sequence, 32 over 8 heads of 128): 128
// windows of 4,096 16-bit keys 317 us, 6.7 TB/s; 32 sequences of 16,000 - 32,768
// e4m3fn keys 248 us, 6.4 TB/s (99 and 95 % of a copy's rate), with four queries each
// 312 us; 64 such sequences of 4-bit keys 401 us, 4.5 TB/s, and one of 131,071 keys 48 us.  The 4-bit ones are
// bound by the eight warps' conversions and products, not by memory; 12 or 16
// warps with fewer registers each took 670 us and more.
#pragma once

#include "kv_async.cuh"
#include "kv_attend_split.cuh"

namespace kvimpl {

// A run of bytes (both ends and the length multiples of 16).
__device__ __forceinline__ void copy_run(uint32_t dst, const uint8_t* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

// Keys of a tile of a 4-bit cache, whose softmax would cost as much as their products otherwise
// (64 sequences of 24,000 keys: 427 us at 64, 480 at 32).
constexpr int kStreamFp4Tile = 64;

struct StreamParams {
  SplitParams s;
  int32_t box;   // keys of a TMA box: a tile's, or 32 or 16 of them
  int32_t flat_scales;  // e2m1: the scales of neighbouring keys and all heads are one run of bytes
  CUtensorMap k_map, v_map, ks_map, vs_map;
};

template <int FMT, int DP, int NB>
struct StreamLayout {
  using L = Layout<FMT, DP>;
  static constexpr int TW = FMT == KV_CACHE_E2M1 ? kStreamFp4Tile : L::TW;
  static constexpr int kHeads = kSplitWarps;                     // heads, or tiles of fewer, of a CTA: a warp each
  static constexpr int kWarps = kHeads;
  static constexpr int kThreads = 32 * (kWarps + 4);             // and a warpgroup of which one warp copies
  static constexpr int kLaunchRegs = 168, kRegs = 208, kCopyRegs = 88;
  static_assert(32 * kWarps * kRegs + 128 * kCopyRegs <= kThreads * kLaunchRegs, "the registers of the launch");
  static constexpr int W = L::kRow > 128 ? 128 : L::kRow;        // bytes of a row of a box
  static constexpr int kSpans = L::kRow > 128 ? L::kRow / 128 : 1;  // boxes of a head's row
  static constexpr int kCodes = kHeads * TW * L::kRow;
  static constexpr int kUnit = kCodes + (FMT == KV_CACHE_E2M1 ? (kHeads * TW * (DP / 16) + 1023) / 1024 * 1024 : 0);
  static constexpr int kFrag = (NB * (L::VN * L::VD / 2) * 4 + 4 * NB) * 128;  // a warp's sums and statistics
  static constexpr int kJoin = kWarps / 2 * kFrag;                // at most half of them write at a time
  static constexpr int kFit = (219 * 1024 - 3072 - kJoin) / kUnit;      // 8 KB are left to the static part
  static constexpr int kUnits = kFit > 20 ? 20 : kFit;
  static constexpr int kOffJoin = kUnits * kUnit;
  static constexpr int kOffBars = kOffJoin + kJoin;
  static constexpr int kOffDesc = kOffBars + (2 * kUnits + 1) * 8 + 8;
  static constexpr int kTotal = kOffDesc + kUnits * 32 + 1024;
  static_assert(kUnits >= 4 && kUnit % 1024 == 0, "ring");
};

// What a step belongs to, written by the copy warp.
struct StreamStep {
  int32_t b, item, step, flags;
  int32_t share, pad[3];
};
// of an item's steps in a share: the first, the last; the share has all of them, or the item's first; no more
// steps; a page id of the step's is out of range
constexpr int kFirst = 1, kLast = 2, kWhole = 4, kBegins = 8, kStop = 16, kBadPage = 32;

// kDimsFit (4-bit caches): head_dim is DP, so that every piece of a lane has its block scales (64
// sequences of 16,000 - 32,768 keys 420 us; 456 with the other form's selection).
template <int FMT, int DP, int NB, bool kBF16, bool kDimsFit>
__global__ void __launch_bounds__(StreamLayout<FMT, DP, NB>::kThreads, 1)
    kv_attend_stream(const __grid_constant__ StreamParams sp) {
  using L = Layout<FMT, DP>;
  using S = StreamLayout<FMT, DP, NB>;
  constexpr int TW = S::TW, MB = TW / 16, W = S::W, QP = DP / 8, OM = L::VN * L::VD / 2;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ int64_t sh_scan[S::kThreads / 32];
  __shared__ int64_t sh_excl[S::kThreads + 1];  // first step of each thread's sequences; the total
  __shared__ SplitWork sh_work;
  __shared__ WaitState sh_waits;

  const SplitParams& p = sp.s;
  const AttendParams& a = p.a;
  const uint32_t tid = threadIdx.x, lane = tid & 31u, warp = tid >> 5;
  const uint32_t raw = static_cast<uint32_t>(__cvta_generic_to_shared(smem_raw));
  const uint32_t ring = (raw + 1023u) & ~1023u;
  uint8_t* const smem_ptr = smem_raw + (ring - raw);
  const uint32_t full = ring + S::kOffBars, empty = full + 8 * S::kUnits, join_bar = empty + 8 * S::kUnits;
  StreamStep* const steps = reinterpret_cast<StreamStep*>(smem_ptr + S::kOffDesc);
  if (tid == 0) {
    for (int i = 0; i < S::kUnits; ++i) {
      bar_init(full + 8 * i, 1);
      bar_init(empty + 8 * i, S::kWarps);
    }
    bar_init(join_bar, S::kWarps);
    sh_waits = WaitState{0, 0};
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  grid_handover();

  // -- the shares ---------------------------------------------------------------------------
  const int32_t per_thread = (a.num_seqs + S::kThreads - 1) / S::kThreads;
  {
    const int32_t b0 = min(static_cast<int32_t>(tid) * per_thread, a.num_seqs), b1 = min(b0 + per_thread, a.num_seqs);
    int64_t mine = 0;
    for (int32_t b = b0; b < b1; ++b) mine += seq_units<TW>(p, b, blockIdx.x == 0);
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= static_cast<uint32_t>(o)) incl += v;
    }
    if (lane == 31u) sh_scan[warp] = incl;
    __syncthreads();
    int64_t excl = incl - mine, total = 0;
    for (uint32_t w = 0; w < S::kThreads / 32; ++w) {
      if (w < warp) excl += sh_scan[w];
      total += sh_scan[w];
    }
    sh_excl[tid] = excl;
    if (tid == 0) sh_excl[S::kThreads] = total;
    if (p.split && blockIdx.x == 0) {  // for the join
      for (int32_t b = b0; b < b1; ++b) {
        p.meta[b] = excl;
        excl += seq_units<TW>(p, b, false);
      }
    }
  }
  __syncthreads();
  if (tid == 0) {
    if (p.split) {
      cut_shares(sh_excl[S::kThreads], static_cast<int32_t>(gridDim.x), p.max_shares, p.min_steps, &sh_work);
      if (blockIdx.x == 0) {
        for (int i = 0; i < sh_work.levels; ++i) p.head->level[i] = sh_work.level[i];
        p.head->levels = sh_work.levels;
      }
    } else {
      sh_work.level[0] = ShareLevel{0, 1, 0};
      sh_work.levels = 1;
      sh_work.shares = static_cast<int32_t>(sh_excl[S::kThreads]);
    }
  }
  __syncthreads();
  WaitState* const waits = &sh_waits;
  const int32_t G = static_cast<int32_t>(a.group.d);

  // (all warps of a warpgroup execute the same one)
  if (warp >= S::kWarps) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kCopyRegs));
  if (warp == S::kWarps) {
    // ======================================================================================
    // the copies
    // ======================================================================================
    const int32_t nbox = TW / sp.box;                  // boxes of a tile
    const int32_t sub = static_cast<int32_t>(lane) / nbox, part = static_cast<int32_t>(lane) - sub * nbox;
    const bool mine = sub < p.subs;                    // the lane has a box of every step
    const uint32_t box_bytes = static_cast<uint32_t>(sp.box * p.hw) * W;
    const uint32_t sc_bytes = FMT == KV_CACHE_E2M1 ? static_cast<uint32_t>(sp.box * p.hw * (a.head_dim / 16)) : 0u;
    const uint32_t at_codes = static_cast<uint32_t>(sub) * (p.hw * TW * L::kRow) + static_cast<uint32_t>(part) * S::kSpans * box_bytes;
    const uint32_t at_scales = S::kCodes + static_cast<uint32_t>(sub * nbox + part) * sc_bytes;
    uint32_t unit = 0u;
    bool ok = true;
    // Ends with a fence between proxies: the products' loads are generic accesses, still under way for all that
    // an arrival tells TMA, which writes past them. (Without it units were overwritten under a warp
    // that was late while the others stored their sums.)
    auto wait_empty = [&](uint32_t u) {
      if (ok && u >= S::kUnits) ok = __all_sync(0xFFFFFFFFu, bar_wait(empty + 8 * (u % S::kUnits), (u / S::kUnits - 1) & 1u, waits));
      fence_async_shared();
    };
    const int32_t shares = sh_work.shares;
    int32_t share = static_cast<int32_t>(blockIdx.x);
    while (ok && share < shares) {
      int32_t after = share + static_cast<int32_t>(gridDim.x);  // without a split: one item a share
      if (p.split) {  // asked for early: the answer is needed at this share's end
        if (lane == 0u) after = static_cast<int32_t>(gridDim.x + atomicAdd(&p.head->next, 1u));
      }
      int32_t level = sh_work.levels - 1;
      while (level > 0 && sh_work.level[level].first > share) --level;
      int64_t pos = sh_work.level[level].start + static_cast<int64_t>(share - sh_work.level[level].first) * sh_work.level[level].size;
      const int64_t end = min(sh_excl[S::kThreads], pos + sh_work.level[level].size);
      int32_t lo = 0, hi = S::kThreads - 1;  // the thread whose sequences hold the first step
      while (lo < hi) {
        const int32_t mid = (lo + hi + 1) >> 1;
        if (sh_excl[mid] <= pos) lo = mid; else hi = mid - 1;
      }
      int32_t b = lo * per_thread;
      int64_t base = sh_excl[lo];
      while (ok && pos < end && b < a.num_seqs) {
        const AttendSeq seq = attend_seq(a, b, false);
        const SplitGeom geom = split_geom<TW>(p, seq);
        const int32_t unit_steps = p.split ? geom.steps : 1;
        const int64_t local = pos - base, all = static_cast<int64_t>(geom.blocks) * p.hgroups * unit_steps;
        if (local >= all) {
          base += all;
          ++b;
          continue;
        }
        const int32_t item = static_cast<int32_t>(local / unit_steps);
        const int32_t s_in = static_cast<int32_t>(local - static_cast<int64_t>(item) * unit_steps);
        const int32_t s_out = static_cast<int32_t>(min(static_cast<int64_t>(unit_steps), s_in + (end - pos)));
        pos += s_out - s_in;
        const int32_t step0 = p.split ? s_in : 0, step1 = p.split ? s_out : geom.steps;
        const int32_t rb = item / p.hgroups, hg = item - rb * p.hgroups, row0 = rb * p.rows;
        const int32_t nrows = min(p.rows, seq.nq * G - row0), p_first = seq.len - seq.nq;
        const int32_t p_lo = p_first + static_cast<int32_t>(a.group.quot(static_cast<uint32_t>(row0)));
        const int32_t p_hi = p_first + static_cast<int32_t>(a.group.quot(static_cast<uint32_t>(row0 + nrows - 1)));
        const TileList list = visible_tiles<TW>(a, p_lo, p_hi);
        const int32_t* table = a.table + static_cast<int64_t>(b) * a.table_stride;
        // First key of the lane's box; -1: none, or none that a row sees (its page may be gone).
        auto key_of = [&](int32_t step) -> int32_t {
          const int32_t li = step * p.subs + sub;
          if (!mine || step >= step1 || li >= list.n) return -1;
          const int32_t k = list.tile(li) * TW + part * sp.box;
          return k > p_hi || (k >= a.sinks && k + sp.box <= list.lo_key) ? -1 : k;
        };
        int32_t key = key_of(step0);
        int32_t id = key >= 0 ? __ldg(table + a.page.quot(static_cast<uint32_t>(key))) : 0;
        for (int32_t step = step0; step < step1; ++step) {
          const bool has = key >= 0;
          const uint32_t boxes = static_cast<uint32_t>(__popc(__ballot_sync(0xFFFFFFFFu, has)));
          int32_t page = id;
          const bool bad = has && (id < 0 || id >= a.num_pages);
          if (bad) {
            page = a.num_pages;  // outside the map: zeros
            record_oob(a.err, static_cast<uint64_t>(b));
          }
          const bool any_bad = __any_sync(0xFFFFFFFFu, bad);
          const uint32_t in_page = has ? static_cast<uint32_t>(key) - a.page.quot(static_cast<uint32_t>(key)) * a.page.d : 0u;
          key = key_of(step + 1);
          id = key >= 0 ? __ldg(table + a.page.quot(static_cast<uint32_t>(key))) : 0;
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const uint32_t u = unit + kv, slot = u % S::kUnits, bar = full + 8 * slot, at = ring + slot * S::kUnit;
            wait_empty(u);
            if (!ok) break;
            if (lane == 0u) {
              if (kv == 0) {
                StreamStep& d = steps[slot];
                d.b = b;
                d.item = item;
                d.step = step;
                d.flags = (step == step0 ? kFirst : 0) | (step == step1 - 1 ? kLast : 0) | (s_out - s_in == unit_steps ? kWhole : 0) | (step0 == 0 ? kBegins : 0) | (any_bad ? kBadPage : 0);
                d.share = share;
              }
              bar_arrive_expect(bar, boxes * (S::kSpans * box_bytes + sc_bytes));
            }
            __syncwarp();
            if (has) {
#pragma unroll
              for (int x = 0; x < S::kSpans; ++x)
                tma_box(at + at_codes + x * box_bytes, kv ? &sp.v_map : &sp.k_map, bar, x * W, static_cast<int32_t>(in_page), hg * p.hw, page);
              if constexpr (FMT == KV_CACHE_E2M1) {
                if (sp.flat_scales)
                  copy_run(at + at_scales, (kv ? a.v_sc : a.k_sc) + (page == a.num_pages ? 0 : wide(page, kv ? p.vs_page : p.ks_page) +
                                               wide(in_page, kv ? p.vs_slot : p.ks_slot)), sc_bytes, bar);
                else
                  tma_box(at + at_scales, kv ? &sp.vs_map : &sp.ks_map, bar, hg * p.hw * (a.head_dim / 16), static_cast<int32_t>(in_page), 0, page);
              }
            }
          }
          if (!ok) break;
          unit += 2;
        }
      }
      share = __shfl_sync(0xFFFFFFFFu, after, 0);
    }
    wait_empty(unit);
    if (ok && lane == 0u) {
      steps[unit % S::kUnits].flags = kStop;
      bar_arrive(full + 8 * (unit % S::kUnits));
    }
    if (!ok)  // boxes in flight write shared memory: let them land before the CTA leaves it
      for (int i = 0; i < 1000; ++i) __nanosleep(1000);
  } else if (warp < S::kWarps) {
    // ======================================================================================
    // the products
    // ======================================================================================
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kRegs));
    const uint32_t g = lane >> 2, t = lane & 3u;
    const bool used = static_cast<int32_t>(warp) < p.hw * p.subs;
    const int32_t hl = static_cast<int32_t>(warp) % p.hw, sub = static_cast<int32_t>(warp) / p.hw;
    // Row g of a product is key gk of its eight: lanes that read together then meet rows of both
    // parities and of both halves of the swizzle.
    const uint32_t gk = g ^ ((g & 1u) << 2);
    const float kscale = a.scale_log2 * tensor_scale(a.k_scale);
    const float vscale = tensor_scale(a.v_scale);
    const uint32_t ds = static_cast<uint32_t>(a.head_dim) / 16;
    // where the warp's rows are in a unit
    const uint32_t head_at = static_cast<uint32_t>(sub) * (p.hw * TW * L::kRow) + static_cast<uint32_t>(hl * sp.box) * W;
    const uint32_t span_step = static_cast<uint32_t>(p.hw * sp.box) * W;
    // where 16 keys begin: boxes of a tile lie one behind the other
    const uint32_t box_step = S::kSpans * span_step;
    const int per_box = sp.box / 16;  // 1, 2 or 4
    auto mb_at = [&](int mb) -> uint32_t {
      return per_box == 1 ? mb * box_step : per_box == 2 ? (mb >> 1) * box_step + (mb & 1) * 16u * W : mb * 16u * W;
    };
    const uint32_t sc_row = static_cast<uint32_t>(p.hw) * ds;
    const uint32_t sc_at = S::kCodes + static_cast<uint32_t>(sub * TW) * sc_row + static_cast<uint32_t>(hl) * ds;
    // The lane's block scales of a K and of a V row: where they are, and which bits count. A piece behind
    // head_dim has none (its codes are 0; the next bytes are another head's or key's, and may be NaN).
    const uint32_t k_block = t * (L::KD / kFp4Block), v_block = g * L::VD / kFp4Block;
    const uint32_t k_sc = kDimsFit || k_block < ds ? k_block : 0u, k_bits = kDimsFit || k_block < ds ? 0xFFFFu : 0u;
    const uint32_t v_sc = kDimsFit || v_block < ds ? v_block : 0u, v_bits = kDimsFit || v_block < ds ? 0xFFu : 0u;
    static_assert(FMT != KV_CACHE_E2M1 || (L::KN == 1 && L::VN == 1 && L::VD <= kFp4Block), "a lane has one piece of a 4-bit row");
    float* const frag = reinterpret_cast<float*>(smem_ptr + S::kOffJoin);

    uint32_t qf[NB][QP];
    float rs[NB][2], o[NB][OM][4], m[NB][2], l[NB][2];
    AttendSeq seq{0, 0, 0};
    TileList list{0, 0, 0, 0};
    int32_t b = 0, kvh = 0, row0 = 0, nrows = 0, p_lo = 0, p_hi = 0;
    uint32_t joins = 0u;
    bool ok = true;
    auto join_wait = [&] {
      __syncwarp();
      if (lane == 0u) bar_arrive(join_bar);
      if (ok) ok = __all_sync(0xFFFFFFFFu, bar_wait(join_bar, joins & 1u, waits));
      ++joins;
    };
    for (uint32_t n = 0u; ok; ++n) {
      const uint32_t ks = (2u * n) % S::kUnits, vs = (2u * n + 1u) % S::kUnits;
      ok = __all_sync(0xFFFFFFFFu, bar_wait(full + 8 * ks, ((2u * n) / S::kUnits) & 1u, waits));
      if (!ok) break;
      const volatile StreamStep& d = steps[ks];
      const int32_t flags = d.flags, step = d.step;
      if ((flags & kStop) != 0) break;
      if ((flags & kFirst) != 0) {
        // -- a new item -------------------------------------------------------------------
        b = d.b;
        const int32_t item = d.item, rb = item / p.hgroups;
        kvh = (item - rb * p.hgroups) * p.hw + hl;
        seq = attend_seq(a, b, false);
        row0 = rb * p.rows;
        nrows = min(p.rows, seq.nq * G - row0);
        p_lo = seq.len - seq.nq + static_cast<int32_t>(a.group.quot(static_cast<uint32_t>(row0)));
        p_hi = seq.len - seq.nq + static_cast<int32_t>(a.group.quot(static_cast<uint32_t>(row0 + nrows - 1)));
        list = visible_tiles<TW>(a, p_lo, p_hi);
        // lane (g, t)'s K pieces: 2t and 2t + 1 of each 128 bytes; piece t of shorter rows
        load_queries<FMT, DP, NB>(a, seq, kvh, row0, nrows, kscale,
                                  [&](int i) {
                                    const int pc = 2 * i / L::KD, rem = 2 * i % L::KD;
                                    return L::kRow >= 128 ? ((pc >> 1) * 8 + 2 * static_cast<int>(t) + (pc & 1)) * L::KD + rem
                                                    : static_cast<int>(t) * L::KD + rem;
                                  }, qf, rs);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
          for (int i = 0; i < OM; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[nb][i][c] = 0.0f;
          m[nb][0] = m[nb][1] = -INFINITY;
          l[nb][0] = l[nb][1] = 0.0f;
        }
      }
      const int32_t share = d.share;
      const int32_t li = step * p.subs + sub, j0 = list.tile(li) * TW;
      const bool work = used && li < list.n;
      uint32_t pt[MB][NB][2], pl[MB][NB][2];
      if (work) {
        // S^T = K Q^T
        float s[MB][NB][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int c = 0; c < 4; ++c) s[mb][nb][c] = 0.0f;
        const uint32_t kat = ring + ks * S::kUnit + head_at + gk * W;
        const uint32_t scat = ring + ks * S::kUnit + sc_at + gk * sc_row;
#pragma unroll
        for (int i = 0; i < L::KN; ++i) {
          // rows gk and gk + 8 share a swizzle
          const uint32_t piece = L::kRow >= 128 ? ((2u * t + (i & 1)) ^ gk) << 4
                                 : W == 64      ? (t ^ ((gk >> 1) & 3u)) << 4
                                                : t * L::KC;
          uint32_t w[MB][2][L::KC / 4], sc[MB][2];
#pragma unroll
          for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int rh = 0; rh < 2; ++rh) {
              ld_own<L::KC>(w[mb][rh], kat + mb_at(mb) + (L::kRow >= 128 ? i >> 1 : 0) * span_step + rh * 8 * W + piece);
              sc[mb][rh] = 0u;
              if constexpr (FMT == KV_CACHE_E2M1) {
                const uint32_t at = scat + (mb * 16 + rh * 8) * sc_row + k_sc;
                sc[mb][rh] = (L::KD > kFp4Block ? ld_shared_u16(at) : ld_shared_u8(at)) & k_bits;
              }
            }
          k_products<FMT, DP, NB, kBF16>(s, w, sc, qf, i * (L::KD / 2));
        }
        __syncwarp();
        if (lane == 0u) bar_arrive(empty + 8 * ks);
        const bool bad = (flags & kBadPage) != 0;
        if (bad || !(j0 + TW - 1 <= p_lo && (a.window == 0 || j0 > p_hi - a.window || j0 + TW - 1 < a.sinks)))
          hide_scores<NB, MB>(a, a.table + static_cast<int64_t>(b) * a.table_stride, j0, p_hi, bad, seq.len - seq.nq, row0, gk, s);
        if constexpr (FMT == KV_CACHE_E2M1) {  // before the softmax, for one stretch of code without a wait
          ok = __all_sync(0xFFFFFFFFu, bar_wait(full + 8 * vs, ((2u * n + 1u) / S::kUnits) & 1u, waits));
          if (!ok) break;
        }
        softmax_step<FMT, NB, MB, OM, kBF16>(s, rs, m, l, o, pt, pl);
      } else {
        __syncwarp();
        if (lane == 0u) bar_arrive(empty + 8 * ks);
      }

      // O^T += V^T P^T
      if (FMT != KV_CACHE_E2M1 || !work)
        ok = __all_sync(0xFFFFFFFFu, bar_wait(full + 8 * vs, ((2u * n + 1u) / S::kUnits) & 1u, waits));
      if (!ok) break;
      if (work) {
        const uint32_t unit_at = ring + vs * S::kUnit, vat = unit_at + head_at;
        // Rows behind the sequence's end and in boxes that were not copied may hold anything, and a weight of 0
        // must not meet a NaN: rows r0 .. r1 - 1 of the tile are cleared.
        auto clear = [&](int32_t r0, int32_t r1) {
          for (int32_t r = r0; r < r1; ++r) {
            if constexpr (FMT == KV_CACHE_E2M1) {
              for (uint32_t x = lane; x < ds; x += 32u)
                asm volatile("st.shared.u8 [%0], %1;" ::"r"(unit_at + sc_at + static_cast<uint32_t>(r) * sc_row + x), "h"(static_cast<uint16_t>(0)) : "memory");
            } else {
              const uint32_t at = vat + mb_at(r >> 4) + static_cast<uint32_t>(r & 15) * W;
#pragma unroll
              for (int x = 0; x < S::kSpans; ++x)
                if (lane < W / 16) {
                  asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at + x * span_step + lane * 16u), "r"(0u) : "memory");
                }
            }
          }
        };
        const int32_t in_box = sp.box - 1;  // boxes are 16, 32 or 64 keys
        const int32_t there = min(seq.len, (p_hi | in_box) + 1);                               // keys from here on are not,
        const int32_t gap0 = (a.sinks + in_box) & ~in_box, gap1 = list.lo_key & ~in_box;       // nor those between these two
        if (j0 + TW > there || (gap0 < gap1 && j0 < gap1 && j0 + TW > gap0)) {
          clear(max(there - j0, 0), TW);
          clear(max(gap0 - j0, 0), min(gap1 - j0, TW));
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before TMA fills the unit again
          __syncwarp();
        }
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
#pragma unroll
          for (int i = 0; i < L::VN; ++i) {
            uint32_t w[4][L::VC / 4], sc[2][2] = {{0u, 0u}, {0u, 0u}};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint32_t r = (x & 1) ? (2u * t + 1u) ^ 4u : 2u * t, row = 8u * (x >> 1) + r;
              const uint32_t piece = L::kRow >= 128 ? (g ^ r) << 4
                                     : W == 64      ? (((g >> 1) ^ ((r >> 1) & 3u)) << 4) + (g & 1u) * 8u
                                                    : g * L::VC;
              ld_own<L::VC>(w[x], vat + mb_at(mb) + i * span_step + row * W + piece);
              if constexpr (FMT == KV_CACHE_E2M1) {
                const uint32_t at = unit_at + sc_at + (mb * 16 + row) * sc_row + v_sc;
                sc[x >> 1][0] |= (ld_shared_u8(at) & v_bits) << (8 * (x & 1));
              }
            }
            v_products<FMT, DP, NB, kBF16>(o, w, sc, pt[mb], pl[mb], i * (L::VD / 2));
          }
        }
      }
      __syncwarp();
      if (lane == 0u) bar_arrive(empty + 8 * vs);
      if ((flags & kLast) == 0) continue;

      // -- the item's end: the warps of a head join, the first writes -------------------------
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
      for (int32_t many = p.subs; many > 1; many = (many + 1) / 2) {
        const int32_t half = (many + 1) / 2;  // subs half .. many - 1 hand theirs to 0 .. many - half - 1
        float* const at = frag + ((sub >= half ? sub - half : sub) * p.hw + hl) * (S::kFrag / 4) + lane;  // a float a lane
        if (used && sub >= half && sub < many) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int i = 0; i < OM; ++i)
#pragma unroll
              for (int c = 0; c < 4; ++c) at[((nb * OM + i) * 4 + c) * 32] = o[nb][i][c];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              at[(NB * OM * 4 + nb * 4 + c) * 32] = m[nb][c];
              at[(NB * OM * 4 + nb * 4 + 2 + c) * 32] = l[nb][c];
            }
          }
        }
        join_wait();
        if (used && sub < many - half) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float mo = at[(NB * OM * 4 + nb * 4 + c) * 32], mn = fmaxf(m[nb][c], mo), ref = mn == -INFINITY ? 0.0f : mn;
              const float ea = exp2_fast(m[nb][c] - ref), eb = exp2_fast(mo - ref);
              m[nb][c] = mn;
              l[nb][c] = __fmaf_rn(l[nb][c], ea, at[(NB * OM * 4 + nb * 4 + 2 + c) * 32] * eb);
#pragma unroll
              for (int i = 0; i < OM; ++i)
#pragma unroll
                for (int y = 0; y < 2; ++y)
                  o[nb][i][2 * y + c] = __fmaf_rn(o[nb][i][2 * y + c], ea, at[((nb * OM + i) * 4 + 2 * y + c) * 32] * eb);
            }
        }
        join_wait();
      }
      if (ok && used && sub == 0) {
        if ((flags & kWhole) != 0) {
          write_rows<FMT, DP, NB>(a, b, seq, kvh, row0, nrows, vscale, o, m, l, waits);
        } else {
          // a part that begins its item is the second of its share, one that does not the first
          write_part<FMT, DP, NB>(p, (static_cast<int64_t>(2 * share + ((flags & kBegins) != 0 ? 1 : 0)) * p.hw + hl) * p.part_rows, nrows, o, m, l);
        }
      }
    }
  }
  __syncthreads();
  if (tid == 0 && waits->ran_out()) {
    record_wait(a.err);
    if (p.split) p.head->gave_up = 1u;
  }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------

// Launches the kernel of one format and padded head dim.
template <int FMT, int DP, int NB, bool kBF16, bool kDimsFit>
kv_status launch_stream(StreamParams sp, void* work, int64_t work_bytes, int64_t max_keys, cudaStream_t stream) {
  using S = StreamLayout<FMT, DP, NB>;
  auto* kernel = kv_attend_stream<FMT, DP, NB, kBF16, kDimsFit>;
  static_assert(S::kTotal <= 227 * 1024 - 8 * 1024, "shared memory, with the static part");
  int sms = 0;
  kv_status st = current_sm_count(&sms);
  if (st != KV_OK) return st;
  static SmemOptIn opt_in;
  st = opt_in(reinterpret_cast<const void*>(kernel), S::kTotal);
  if (st != KV_OK) return st;
  int64_t grid = set_up_split<DP>(sp.s, S::kHeads, 8 * NB, S::TW, sms, work, work_bytes, max_keys);
  if (!sp.s.split && grid > sms) grid = sms;  // CTAs go on to further items by themselves
  const kv_status ls = launch_chained(kernel, grid, S::kThreads, S::kTotal, stream, sp);
  if (ls != KV_OK || !sp.s.split) return ls;
  return launch_join<FMT, DP, S::TW>(sp.s, sms, stream);
}

template <int FMT, int DP, bool kBF16>
kv_status launch_stream_dim(const StreamParams& sp, bool wide, void* work, int64_t work_bytes, int64_t max_keys,
                            cudaStream_t stream) {
  if constexpr (FMT == KV_CACHE_E2M1) {
    if (sp.s.a.head_dim != DP)
      return wide ? launch_stream<FMT, DP, 2, kBF16, false>(sp, work, work_bytes, max_keys, stream)
                  : launch_stream<FMT, DP, 1, kBF16, false>(sp, work, work_bytes, max_keys, stream);
  }
  return wide ? launch_stream<FMT, DP, 2, kBF16, true>(sp, work, work_bytes, max_keys, stream)
              : launch_stream<FMT, DP, 1, kBF16, true>(sp, work, work_bytes, max_keys, stream);
}

template <int FMT, bool kBF16>
kv_status launch_stream_fmt(const StreamParams& sp, bool wide, void* work, int64_t work_bytes, int64_t max_keys,
                            cudaStream_t stream) {
  return sp.s.a.head_dim <= 64 ? launch_stream_dim<FMT, 64, kBF16>(sp, wide, work, work_bytes, max_keys, stream)
                               : launch_stream_dim<FMT, 128, kBF16>(sp, wide, work, work_bytes, max_keys, stream);
}

// The formats' instantiations, a translation unit each.
kv_status stream_bf16(const StreamParams& p, bool wide, void* work, int64_t work_bytes, int64_t max_keys, cudaStream_t stream);
kv_status stream_f16(const StreamParams& p, bool wide, void* work, int64_t work_bytes, int64_t max_keys, cudaStream_t stream);
kv_status stream_e4m3(const StreamParams& p, bool wide, void* work, int64_t work_bytes, int64_t max_keys, cudaStream_t stream);
kv_status stream_e2m1(const StreamParams& p, bool wide, void* work, int64_t work_bytes, int64_t max_keys, cudaStream_t stream);

}  // namespace kvimpl
