// fa_paged.cu — attention of a few new tokens over a paged key/value cache:
// one token, a chain, or a tree of drafted tokens for each sequence.
//
// New token i of sequence b (c_b places cached before, n_b new) sees place p iff
// p < c_b, or p = c_b + j with j < n_b and, in a chain, j <= i, in a tree, bit j
// of the token's mask set.  What a token does not see contributes nothing,
// whatever it holds; a token that sees nothing gets O = 0 and LSE = -inf.
#include <cuda_bf16.h>

#include <cmath>

#include "fa_paged.h"
#include "paged_seq.h"
#include "ptx.cuh"

namespace fa {
namespace {

// Work.  A unit is one key tile (bn places) of one item; an item is one (sequence,
// HB adjacent kv heads, row group), a row group being QT tiles of TB * G rows (TB
// tokens with the G query heads that share a kv head).  The units of all items stand
// in one line, each item's after `lead` units without a tile that stand for its other
// costs (fetching its Q, writing its result), cut into equal stretches for the blocks,
// so that ragged batches keep all SMs busy; the lengths are known on the device only,
// so every block sums them up itself.  A block that gets only a part of an item writes
// its unnormalised O with the row maxima and sums; paged_combine_kernel joins the
// parts.
struct PagedParams {
  CUtensorMap tm_q;  // [total, Hkv, G, d]: box 64 columns x G heads x TB tokens
  CUtensorMap tm_k, tm_v;  // [num_pages, page_size, Hkv, d]: box 64 columns x min(page_size, BN) rows of one head
  const __nv_bfloat16 *q, *v_pages;
  const int *cu;
  const unsigned long long *mask;  // [total, words] or nullptr: a chain
  __nv_bfloat16 *o;
  float *lse;
  float *part_o;      // [2 * blocks, d, rows] fp32, rows of an item token by token
  float2 *part_ml;    // [2 * blocks, rows]: row maximum (scaled log2 units) and sum
  long long *prefix;  // [B + 1] units before each sequence
  unsigned *status;
  PageGeom g;
  int words, max_new, total, H, Hkv, G, TB;
  int bn_log2, QT, HB;  // places in a tile; row tiles and kv heads of an item
  int heads, groups;    // Hkv / HB; row groups of max_new tokens
  int min_units;        // a block's stretch is no shorter
  int lead;             // units that stand for what an item costs beside its tiles
  bool by_warp;         // up to 32 sequences, whose units fit 31 bits
  int join, join_y;     // the join: warps that share a task, blocks of a row group that is not the last
  float scale_log2;
};

// Head dim 64: the rings of an SM's blocks hold 128 KB.  With all that fits (176 to 192 KB)
// the many short rows in flight cost bandwidth: 16 x 8000 places, one token, 16 heads 86.5
// against 83.7 us, 8 x 16000, 40 tokens 98 against 90.  (Dim 256, few rows, wants all: 192 KB
// 154 us, 128 KB 165, for 32 x 8000 places, 4 heads.)
constexpr int kNarrowRing = 128 * 1024;

template <int D, int BN_, int QT_>
struct PagedCfg {
  static constexpr int kBoxes = D / 64;
  static constexpr int kQBytes = 128 * D * 2;     // one row tile: kBoxes boxes of 128 rows
  static constexpr int kTileBytes = BN_ * D * 2;  // one tile of K or V
  static constexpr int kBoxBytes = BN_ * 128;     // its 64-column box
  static constexpr int kMinBlocks = (QT_ == 1 && D <= 128) ? 2 : 1;
  static constexpr int kSmemMax = kMinBlocks == 2 ? 113 * 1024 : 227 * 1024;
  static constexpr int kStagesFit = (kSmemMax - 1024 - 512 - QT_ * kQBytes) / kTileBytes;
  static constexpr int kStages = D == 64 ? kNarrowRing / kMinBlocks / kTileBytes : kStagesFit;
  static_assert(kStages >= 4 && kStages <= kStagesFit, "ring");
  static constexpr int kThreads = 128 * QT_ + 64;  // softmax warps, MMA warp, TMA warp
  static constexpr int kMmaWarp = 4 * QT_, kLoadWarp = 4 * QT_ + 1;
  // S of row tile t: 128 columns from 128 t (two tiles of 64 places, or one of 128), then O
  static constexpr int kOCol = 128 * QT_;
  static constexpr int kTmemNeed = QT_ * (128 + D);
  static constexpr bool kPair = BN_ == 128;
  static_assert(BN_ == 64 || BN_ == 128, "");
  static constexpr int kTmemCols = kTmemNeed <= 128 ? 128 : kTmemNeed <= 256 ? 256 : 512;
  static_assert(kTmemNeed <= 512 && kMinBlocks * kTmemCols <= 512, "TMEM budget");
  static constexpr int kOffQ = 0, kOffRing = QT_ * kQBytes, kOffBar = kOffRing + kStages * kTileBytes;
  // barriers: full[S], empty[S], q_full, q_free, s_full[QT][2], p_full[QT][2], pv[QT], o_full[QT], drain.
  // Warps of a row tile may be a buffer apart: two barriers each, by buffer.
  static constexpr int kNumBars = 2 * kStages + 3 + 6 * QT_;
  static constexpr int kOffMisc = kOffBar + 8 * kNumBars;
  static constexpr int kSmemBytes = kOffMisc + 256 + 1024;
  static_assert(kSmemBytes <= kSmemMax, "shared memory budget");
};

// Ring slots of tile j's K and V within an item of nt tiles, in the order the MMA
// warp takes them: K_0 V_0 K_1 V_1 ... where a tile is a pair of halves, else (S a
// tile ahead) K_0 K_1 V_0 K_2 V_1 ... V_last.
template <bool PAIR>
__device__ __forceinline__ int k_fill(int j) {
  return PAIR ? 2 * j : j == 0 ? 0 : 2 * j - 1;
}
template <bool PAIR>
__device__ __forceinline__ int v_fill(int j, int nt) {
  return PAIR ? 2 * j + 1 : j + 1 < nt ? 2 * j + 2 : 2 * nt - 1;
}

FA_STALL_FLAG_DECL

enum PagedSite : int {
  kPSiteQ = 31, kPSiteKFull = 32, kPSiteVFull = 33, kPSitePFull = 34, kPSiteEmpty = 35,
  kPSiteSFull = 36, kPSiteOFull = 37, kPSiteDrain = 38, kPSiteQFree = 39, kPSiteVTail = 40
};

// EARLY: before the kernel's grid_wait (the join's), from L2, so that no line is used which an
// SM's L1 still holds from before these arrays were written.
template <bool EARLY = false>
__device__ __forceinline__ PagedSeq paged_seq(const PagedParams &p, int b) {
  auto at = [](const int *x) { return EARLY ? __ldcg(x) : *x; };
  return paged_seq_of(at(p.cu + b), at(p.cu + b + 1), at(p.g.cache_lens + b), p.total, p.max_new,
                      p.g.max_pages * p.g.page_size);
}
__device__ __forceinline__ void paged_units(const PagedParams &p, const PagedSeq &s, int &tiles, int &groups) {
  tiles = (s.keys + (1 << p.bn_log2) - 1) >> p.bn_log2;
  groups = p.max_new <= p.TB * p.QT ? 1 : (s.n + p.TB * p.QT - 1) / (p.TB * p.QT);
}
// a / b for a >= 0, b > 0, in 32 bits where both fit (nearly always)
__device__ __forceinline__ long long quot(long long a, long long b) {
  if (((a | b) >> 32) == 0) return (long long)((unsigned)a / (unsigned)b);
  return a / b;
}
// Units of a block's stretch.
__device__ __forceinline__ long long stretch_units(const PagedParams &p, long long total, int blocks) {
  return max(quot(total + blocks - 1, blocks), (long long)p.min_units);
}

__device__ __forceinline__ long long units_of(const PagedParams &p, const PagedSeq &s) {
  if (s.n == 0) return 0;
  int tiles, groups;
  paged_units(p, s, tiles, groups);
  return (long long)(tiles + p.lead) * groups * p.heads;
}
__device__ __forceinline__ long long warp_scan(long long x) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if ((threadIdx.x & 31) >= o) x += y;
  }
  return x;
}

// A block's stretch [begin, end) of all units, the sequence it begins in (b < 0
// where there is none) and that one's first unit.
struct PagedStart {
  long long begin, end, base;
  PagedSeq s;
  int b;
};

// Up to 32 sequences whose units surely fit 31 bits (p.by_warp): every warp sums
// them up by itself, a lane each.
struct WarpUnits {
  PagedSeq s;
  unsigned before, after, total;
};
template <bool EARLY = false>
__device__ __forceinline__ WarpUnits warp_units(const PagedParams &p) {
  const int lane = threadIdx.x & 31;
  WarpUnits w;
  w.s = {0, 0, 0, 0};
  if (lane < p.g.B) w.s = paged_seq<EARLY>(p, lane);
  const unsigned x = (unsigned)units_of(p, w.s);
  w.after = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(0xffffffffu, w.after, o);
    if (lane >= o) w.after += y;
  }
  w.before = w.after - x;
  w.total = __shfl_sync(0xffffffffu, w.after, 31);
  return w;
}
__device__ __forceinline__ PagedStart warp_stretch(const PagedParams &p) {
  const WarpUnits w = warp_units(p);
  const unsigned per = max((w.total + gridDim.x - 1) / gridDim.x, (unsigned)p.min_units);
  const unsigned begin = min(per * blockIdx.x, w.total);  // per * blocks < total + 2 * blocks
  const unsigned here = __ballot_sync(0xffffffffu, begin >= w.before && begin < w.after);
  PagedStart r;
  r.b = __ffs(here) - 1;
  const int from = max(r.b, 0);
  r.begin = begin;
  r.end = min(begin + per, w.total);
  r.base = __shfl_sync(0xffffffffu, w.before, from);
  r.s.start = __shfl_sync(0xffffffffu, w.s.start, from);
  r.s.n = __shfl_sync(0xffffffffu, w.s.n, from);
  r.s.len = __shfl_sync(0xffffffffu, w.s.len, from);
  r.s.keys = __shfl_sync(0xffffffffu, w.s.keys, from);
  return r;
}

// More: the block together, through *at (b = -1 on entry), which holds the result
// after the caller's next barrier.  Block 0 also leaves every sequence's first unit
// in p.prefix for the join.
template <int THREADS>
__device__ __forceinline__ void block_stretch(const PagedParams &p, long long *s_sums, PagedStart *at) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  PagedSeq s;
  auto units = [&](int b) -> long long {
    if (b >= p.g.B) return 0;
    s = paged_seq(p, b);
    return units_of(p, s);
  };
  auto block_scan = [&](long long x, long long &total) -> long long {  // exclusive
    const long long sum = warp_scan(x);
    __syncthreads();
    if (lane == 31) s_sums[warp] = sum;
    __syncthreads();
    long long before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      const long long y = s_sums[w];
      if (w < warp) before += y;
      total += y;
    }
    return before + sum - x;
  };
  long long total_units = 0;
  for (int b0 = 0; b0 < p.g.B; b0 += THREADS) {
    long long sum;
    block_scan(units(b0 + (int)threadIdx.x), sum);
    total_units += sum;
  }
  const long long per = stretch_units(p, total_units, gridDim.x);
  const long long begin = min(per * blockIdx.x, total_units);
  long long done = 0;
  for (int b0 = 0; b0 < p.g.B; b0 += THREADS) {
    const int b = b0 + (int)threadIdx.x;
    long long sum;
    const long long x = units(b), before = done + block_scan(x, sum);
    if (b < p.g.B && begin >= before && begin < before + x) {
      at->begin = begin;
      at->end = min(begin + per, total_units);
      at->base = before;
      at->s = s;
      at->b = b;
    }
    if (blockIdx.x == 0 && b < p.g.B) p.prefix[b] = before;
    done += sum;
    if (blockIdx.x != 0 && done > begin) break;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) p.prefix[p.g.B] = total_units;
}

// A stretch of units, item by item; every warp of a block walks its own copy.
struct PagedWalk {
  long long u, end, base;
  int b, tiles, groups;
  PagedSeq s;
  int items;  // so far
  // the current item
  int kh, rg, j0, j1;
  bool whole, first;

  __device__ void start(const PagedParams &p, const PagedStart &at) {
    u = at.b < 0 ? 0 : at.begin;
    end = at.b < 0 ? 0 : at.end;
    items = 0;
    base = at.base;
    b = at.b;
    s = at.s;
    paged_units(p, s, tiles, groups);
  }
  __device__ void load(const PagedParams &p) {
    for (; b < p.g.B; ++b) {
      s = paged_seq(p, b);
      if (s.n > 0) break;
    }
    if (b < p.g.B) paged_units(p, s, tiles, groups);
  }
  __device__ bool next(const PagedParams &p) {
    while (u < end) {
      const unsigned span = (unsigned)(tiles + p.lead);
      if ((unsigned)(u - base) >= span * groups * p.heads) {
        base = u;
        ++b;
        load(p);
        if (b >= p.g.B) return false;
        continue;
      }
      const unsigned r = (unsigned)(u - base);  // a sequence's units fit 31 bits (checked by the host)
      const int item = (int)(r / span), at = (int)(r - (unsigned)item * span);
      const int stop = end - u < (int)span - at ? at + (int)(end - u) : (int)span;
      u += stop - at;
      j0 = max(at - p.lead, 0);
      j1 = stop - p.lead;
      if (j1 <= j0) continue;  // the units without a tile only
      kh = groups == 1 ? item : item / groups;
      rg = item - kh * groups;
      whole = j0 == 0 && j1 == tiles;
      first = items++ == 0;
      return true;
    }
    return false;
  }
};

// Which of the 32 new tokens from j0 on (j0 may be negative) token i of the sequence sees.
__device__ __forceinline__ unsigned seen_bits(const unsigned long long *words, int i, int n, int j0) {
  if (j0 >= n || j0 <= -32) return 0;
  unsigned bits;
  if (words == nullptr) {
    const int m = i - j0;  // the last one seen
    bits = m < 0 ? 0u : m >= 31 ? 0xffffffffu : (2u << m) - 1u;
  } else {
    const int a = max(j0, 0);
    unsigned long long w = words[a >> 6] >> (a & 63);
    if ((a & 63) > 32 && (a >> 6) + 1 <= (n - 1) >> 6) w |= words[(a >> 6) + 1] << (64 - (a & 63));
    bits = (unsigned)w;
    if (j0 < 0) bits <<= -j0;
  }
  if (n - j0 < 32) bits &= (1u << (n - j0)) - 1u;
  if (j0 < 0) bits &= 0xffffffffu << -j0;
  return bits;
}

// bf16 pairs: infinities and NaNs made zero.
__device__ __forceinline__ uint32_t finite_pair(uint32_t w) {
  if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
  if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
  return w;
}

// The V rows of a tile that not every row of S sees.  Past the sequence's end
// they hold anything, and 0 * NaN is NaN: cleared.  Among the new tokens
// non-finite values are cleared too, and the epilogue adds them to the rows that
// see them.  By the 128 threads of row tile 0's softmax, before they hand over the
// tile's first P (which the MMA warp takes before any other row tile's); returns
// whether this warp cleared a new token's value.  Rows from the last page's end on
// are zeros already.
template <int D, int BN>
__device__ __forceinline__ bool clear_unseen(uint8_t *tile, const PagedSeq &s, int kv0, int page_size) {
  const int r0 = max(s.len - kv0, 0), r1 = min((s.keys + page_size - 1) / page_size * page_size - kv0, BN);
  const int chunk = threadIdx.x & 7;
  bool any = false;
#pragma unroll 1
  for (int bx = 0; bx < D / 64; ++bx) {
#pragma unroll 2
    for (int r = r0 + ((threadIdx.x & 127) >> 3); r < r1; r += 16) {
      uint4 *at = reinterpret_cast<uint4 *>(tile + bx * (BN * 128) + r * 128 + ((chunk ^ (r & 7)) * 16));
      if (kv0 + r >= s.keys) {
        *at = make_uint4(0, 0, 0, 0);
        continue;
      }
      const uint4 was = *at;
      const uint4 x = make_uint4(finite_pair(was.x), finite_pair(was.y), finite_pair(was.z), finite_pair(was.w));
      if (x.x != was.x || x.y != was.y || x.z != was.z || x.w != was.w) {
        *at = x;
        any = true;
      }
    }
  }
  fence_proxy_async_smem();
  return __any_sync(0xffffffffu, any);
}

// Sums into x the non-finite values, in columns [col, col + count), of the new
// tokens that a row sees at places [p0, p1): their weights are positive, so the
// sum belongs to that row's O.
__device__ __noinline__ void add_unfinite(const PagedParams &p, const PagedSeq &s, int b, int kh,
                                          const unsigned long long *words, int i, int p0, int p1, int D, int col,
                                          int count, float *x) {
  for (int e = 0; e < count; ++e) x[e] = 0.f;
  for (int j = max(p0 - s.len, 0); j < min(p1, s.keys) - s.len; ++j) {
    if (!(seen_bits(words, i, s.keys - s.len, j) & 1u)) continue;
    const int page = page_of(p.g, b, (long long)s.len + j);
    if (page < 0) continue;
    const __nv_bfloat16 *v =
        p.v_pages + (((size_t)page * p.g.page_size + (s.len + j) % p.g.page_size) * p.Hkv + kh) * D + col;
    for (int e = 0; e < count; ++e) {
      const float y = __bfloat162float(v[e]);
      if (!isfinite(y)) x[e] += y;
    }
  }
}

// Softmax with one pass over the keys: per row the running maximum m and sum l of
// exp2(c2 S - m), O rescaled only where m grows by more than kRescaleTau.  Warps: 4 QT
// of softmax (a thread to a row), one that issues tcgen05 MMAs, one that fetches tiles
// page by page.  A byte of the cache meets `rows` FLOPs (an element 2 * rows), so up to some
// 280 rows HBM is the bound, and from 128 rows on the softmax: each place of a row costs an
// ex2.  P goes to P V in bf16, the type that V has there: each weight within 2^-8 of itself
// (half a step), relative to the row's maximum.  The row sum takes the unrounded weights, so
// that rounding does not shift it too.  O's error against 64 bits is 0.0023 of its norm, where
// fp32 weights with one rounding at the end have 0.0017; they would need V widened in shared
// memory and half the MMA rate.
// One row tile: two blocks on an SM (head dims 64 and 128), tiles of 64 places, S one
// tile ahead of the softmax.  Two: one block, 128 places (at 64 columns an MMA step costs
// what it costs at 128), the softmax 64 columns at a time with one maximum for all 128
// (the first half is read twice; 128 columns in a thread's registers spilled 600 bytes,
// a maximum for each half took 3.3 us more below), one issuing warp that
// alternates between the row tiles (with one for each, both softmaxes ran in phase: 4100
// instead of 3500 cycles for 128 places at that time; 3100 now, of which MMAs 2048).
// Measured with the join: 16 ragged sequences of up to 7000 places, trees of up to 33
// tokens, 4 kv heads of dim 256: 49 us, 4.7 TB/s; one of 32768 places, 64 tokens, 32 on 8
// heads of dim 128: 37 us, 930 TFLOP/s; of both 13 to 14 us are set-up, the first tiles, the
// parts' way out and the join.
template <int D, int BN, int QT>
__global__ void __launch_bounds__(PagedCfg<D, BN, QT>::kThreads, PagedCfg<D, BN, QT>::kMinBlocks)
    paged_fwd_kernel(const __grid_constant__ PagedParams p) {
  using C = PagedCfg<D, BN, QT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::kOffBar;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (C::kStages + s); };
  const uint32_t q_bar = bar0 + 8u * (2 * C::kStages), qfree_bar = q_bar + 8u;
  auto s_bar = [&](int t, int buf) { return q_bar + 8u * (2 + 2 * t + buf); };
  auto p_bar = [&](int t, int buf) { return q_bar + 8u * (2 + 2 * QT + 2 * t + buf); };
  auto pv_bar = [&](int t) { return q_bar + 8u * (2 + 4 * QT + t); };
  auto o_bar = [&](int t) { return q_bar + 8u * (2 + 5 * QT + t); };
  const uint32_t drain_bar = q_bar + 8u * (2 + 6 * QT);
  uint8_t *misc = smem + C::kOffMisc;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(misc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(misc + 4);
  PagedStart *at = reinterpret_cast<PagedStart *>(misc + 192);  // 48 bytes
  volatile int *odd = reinterpret_cast<volatile int *>(misc + 248);  // [QT] the last item with cleared V values
  volatile int *tail_hit = reinterpret_cast<volatile int *>(misc + 244);  // the same, as row tile 0's softmax finds them
  volatile unsigned *bad = reinterpret_cast<volatile unsigned *>(misc + 32);  // [16] granules without a page, by tile
  long long *s_sums = reinterpret_cast<long long *>(misc + 96);               // [kThreads / 32] <= 11
  const WaitCtx wctx{abort_flag, p.status};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kNumBars; ++i) {
      const uint32_t bar = bar0 + 8u * i;
      mbar_init(bar, bar >= p_bar(0, 0) && bar < pv_bar(0) ? 4u : 1u);
    }
    *abort_flag = 0;
    odd[0] = odd[1] = *tail_hit = 0;
    at->b = -1;
    fence_mbar_init();
  }
  if (warp == C::kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  if (warp == C::kLoadWarp && lane == 0) {
    prefetch_tmap(&p.tm_q);
    prefetch_tmap(&p.tm_k);
    prefetch_tmap(&p.tm_v);
  }
  grid_wait();
  grid_go();  // only now: the join reads the call's inputs without a wait of its own
  if (!p.by_warp) block_stretch<C::kThreads>(p, s_sums, at);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  PagedWalk walk;
  walk.start(p, p.by_warp ? warp_stretch(p) : *at);

  auto tile_tokens = [&](int t) { return max(0, min(p.TB, walk.s.n - (walk.rg * QT + t) * p.TB)); };

  if (warp < 4 * QT) {
    // ===================================================== softmax warpgroups
    const int t = warp >> 2;
    const int r = threadIdx.x & 127;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t o_tm = tmem + lane_off + C::kOCol + (uint32_t)(D * t);
    const float c2 = p.scale_log2;
    const int tok = r / p.G, head = r - tok * p.G;
    int tile_no = 0, o_no = 0, pv_no = 0;  // tiles, items, and items of several tiles of this row tile so far
    int tiles = 0, item = 0;               // tiles and items of the block
    bool ok = true;
    while (ok && walk.next(p)) {
      ++item;
      const int tokens = tile_tokens(t), nt = walk.j1 - walk.j0;
      const int i = (walk.rg * QT + t) * p.TB + tok;  // this row's token in its sequence
      const bool live = (warp & 3) * 32 < tokens * p.G;
      const bool row = r < tokens * p.G;
      if (tokens > 0) {
        const unsigned long long *words =
            p.mask && row ? p.mask + (size_t)(walk.s.start + i) * p.words : nullptr;
        float m_ref = -INFINITY, l_sum = 0.f;
        for (int j = 0; j < nt && ok; ++j, ++tile_no) {
          const int kv0 = (walk.j0 + j) * BN;
          const bool tail = kv0 + BN > walk.s.len;
          unsigned see[BN / 32];  // the places this row sees, while the tile is being multiplied
#pragma unroll
          for (int w = 0; w < BN / 32; ++w) {
            see[w] = 0xffffffffu;
            if (tail) {
              const int at = kv0 + 32 * w, pre = walk.s.len - at;
              see[w] = pre >= 32 ? 0xffffffffu : pre <= 0 ? 0u : (1u << pre) - 1u;
              if (pre < 32) see[w] |= seen_bits(words, i, walk.s.keys - walk.s.len, at - walk.s.len);
            }
          }
          const int buf = C::kPair ? 0 : tile_no & 1;
          const uint32_t s_tm = tmem + lane_off + (uint32_t)(64 * (2 * t + buf));
          ok = mbar_wait_warp(s_bar(t, buf), (C::kPair ? tile_no : tile_no >> 1) & 1, wctx, kPSiteSFull);
          if (!ok) break;
          tc_fence_after();
          float s[64];  // of one half
          const unsigned gone = bad[(tiles + j) & 15];
          const bool masked = tail || gone;
          if (gone) {
#pragma unroll
            for (int w = 0; w < BN / 32; ++w) {
              if ((gone >> (2 * w)) & 1) see[w] &= 0xffff0000u;
              if ((gone >> (2 * w)) & 2) see[w] &= 0x0000ffffu;
            }
          }
          auto read_s = [&](int half) {
            uint32_t sr[2][32];
            tmem_ld_32x32b_x32(s_tm + 64 * half, sr[0]);
            tmem_ld_32x32b_x32(s_tm + 64 * half + 32, sr[1]);
            tmem_wait_ld(sr[0]);
            reg_tie(sr[1]);
#pragma unroll
            for (int c = 0; c < 64; ++c) s[c] = __uint_as_float(sr[c >> 5][c & 31]);
            if (masked) {
#pragma unroll
              for (int c = 0; c < 64; ++c)
                if (!((see[2 * half + (c >> 5)] >> (c & 31)) & 1)) s[c] = -INFINITY;
            }
          };
          auto max_s = [&] {
            float mx0 = s[0], mx1 = s[1], mx2 = s[2], mx3 = s[3];
#pragma unroll
            for (int c = 4; c < 60; c += 8) {
              mx0 = fmax3(mx0, s[c], s[c + 1]);
              mx1 = fmax3(mx1, s[c + 2], s[c + 3]);
              mx2 = fmax3(mx2, s[c + 4], s[c + 5]);
              mx3 = fmax3(mx3, s[c + 6], s[c + 7]);
            }
            mx0 = fmax3(mx0, s[60], s[61]);
            mx1 = fmax3(mx1, s[62], s[63]);
            return fmax3(mx0, mx1, fmaxf(mx2, mx3)) * c2;
          };
          float neg_m = 0.f;
          auto weigh = [&](int half) {  // P over the half's S
            float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
            uint32_t pk[32];
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
              float x[4], e[4];
              ffma2(x[0], x[1], s[c], s[c + 1], c2, c2, neg_m, neg_m);
              ffma2(x[2], x[3], s[c + 2], s[c + 3], c2, c2, neg_m, neg_m);
#pragma unroll
              for (int u = 0; u < 4; ++u) e[u] = ex2_mufu(x[u]);
              fadd2(l0, l1, l0, l1, e[0], e[1]);
              fadd2(l2, l3, l2, l3, e[2], e[3]);
              pk[c >> 1] = pack_bf16x2(e[0], e[1]);
              pk[(c >> 1) + 1] = pack_bf16x2(e[2], e[3]);
            }
            tmem_st_32x32b_x32(s_tm + 64 * half, pk);
            l_sum += (l0 + l1) + (l2 + l3);
            tmem_wait_st();
            tc_fence_before();
          };
          if (live) {
            read_s(0);
            float m_blk = max_s();
            if (C::kPair) {  // the second half stays in registers and is weighed first
              read_s(1);
              m_blk = fmaxf(m_blk, max_s());
            }
            if (j == 0) {
              m_ref = m_blk;
            } else if (__any_sync(0xffffffffu, row && (m_blk - m_ref) > kRescaleTau)) {
              // O is read once the P V before is done.  A pair's S follows it; else S of the next tile follows
              // it, and where there is no next tile it has a barrier.
              if (!C::kPair && j + 1 < nt)
                ok = mbar_wait_warp(s_bar(t, buf ^ 1), ((tile_no + 1) >> 1) & 1, wctx, kPSiteOFull);
              else if (!C::kPair)
                ok = mbar_wait_warp(pv_bar(t), pv_no & 1, wctx, kPSiteOFull);
              if (!ok) break;
              tc_fence_after();
              const float m_new = fmaxf(m_ref, m_blk);
              const float alpha = m_ref == m_new ? 1.f : ex2_mufu(m_ref - m_new);
              m_ref = m_new;
              l_sum *= alpha;
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld_32x32b_x32(o_tm + 32 * c, o);
                tmem_wait_ld(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                tmem_st_32x32b_x32(o_tm + 32 * c, o);
              }
            }
            neg_m = m_ref == -INFINITY ? 0.f : -m_ref;  // nothing seen yet: all weights 0
            weigh(C::kPair ? 1 : 0);
          }
          if (t == 0 && tail) {
            const int fv = 2 * tiles + v_fill<C::kPair>(j, nt), sv = fv % C::kStages;
            ok = mbar_wait_warp(full_bar(sv), (fv / C::kStages) & 1, wctx, kPSiteVTail);
            if (!ok) break;
            if (clear_unseen<D, BN>(smem + C::kOffRing + sv * C::kTileBytes, walk.s, kv0, p.g.page_size) && lane == 0)
              *tail_hit = item;
          }
          if (C::kPair) {
            mbar_arrive_warp(p_bar(t, 1));
            if (live) {
              read_s(0);
              weigh(0);
            }
          }
          if (!(FA_STALL(4) && tile_no == 0 && t == 0)) mbar_arrive_warp(p_bar(t, buf));
        }
        // ----------------------------------------------------- epilogue
        if (ok) ok = mbar_wait_warp(o_bar(t), o_no & 1, wctx, kPSiteOFull);
        ++o_no;
        pv_no += nt > 1;
        tc_fence_after();
        if (ok && live) {
          const int odd_item = odd[t];
          const int q_row = walk.s.start + i, h = walk.kh * p.G + head;
          const int all = QT * p.TB * p.G;
          const size_t slot = ((size_t)blockIdx.x * 2 + (walk.first ? 0 : 1)) * all;
          const float inv_l = walk.whole ? (l_sum == 0.f ? 0.f : 1.0f / l_sum) : 1.0f;
          uint4 *orow = reinterpret_cast<uint4 *>(p.o + ((size_t)q_row * p.H + h) * D);
          float *part = p.part_o + slot * D + t * p.TB * p.G + r;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(o_tm + 32 * c, o);
            tmem_wait_ld(o);
            if (row && odd_item == item) {
              float x[32];
              add_unfinite(p, walk.s, walk.b, walk.kh, words, i, walk.j0 * BN, walk.j1 * BN, D, 32 * c, 32, x);
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) + x[e]);
            }
            if (row && walk.whole) {
#pragma unroll
              for (int k4 = 0; k4 < 4; ++k4) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  w[e] = pack_bf16x2(__uint_as_float(o[8 * k4 + 2 * e]) * inv_l, __uint_as_float(o[8 * k4 + 2 * e + 1]) * inv_l);
                orow[4 * c + k4] = make_uint4(w[0], w[1], w[2], w[3]);
              }
            } else if (row) {
#pragma unroll
              for (int e = 0; e < 32; ++e) part[(size_t)(32 * c + e) * all] = __uint_as_float(o[e]);
            }
            __syncwarp();
          }
          if (row && walk.whole) {
            if (p.lse != nullptr)
              p.lse[(size_t)h * p.total + q_row] = (m_ref + __log2f(l_sum)) * 0.69314718055994531f;
          } else if (row) {
            p.part_ml[slot + t * p.TB * p.G + r] = make_float2(m_ref, l_sum);
          }
          tc_fence_before();
        }
      }
      tiles += nt;
    }
  } else if (warp == C::kMmaWarp) {
    // ===================================================== MMA issue (whole warp; the elected lane issues)
    // One warp for both row tiles: their S and P V alternate in the pipe, so that one tile's softmax runs
    // under the other's products.
    constexpr uint32_t idesc_s = make_idesc_bf16(128, BN, false, false);
    constexpr uint32_t idesc_pv = make_idesc_bf16(128, D, false, true);
    auto slot_of = [&](int f) { return f % C::kStages; };
    auto par_of = [&](int f) { return (uint32_t)((f / C::kStages) & 1); };
    const uint64_t q_desc = make_sdesc_sw128(sbase + C::kOffQ, 0, 1024);
    const uint64_t ring_desc_k = make_sdesc_sw128(sbase + C::kOffRing, 0, 1024);
    const uint64_t ring_desc_v = make_sdesc_sw128(sbase + C::kOffRing, C::kBoxBytes, 1024);
    auto issue_s = [&](int t, int buf, int slot) {
      const uint64_t kd = ring_desc_k + (uint64_t)((slot * C::kTileBytes) >> 4);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        mma_ss(tmem + 128u * t + 64u * buf, q_desc + (uint32_t)((t * C::kQBytes + (kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
               kd + (uint32_t)(((kk >> 2) * C::kBoxBytes + (kk & 3) * 32) >> 4), idesc_s, kk > 0);
    };
    // P V of the 64 places whose P is in buffer `buf`, rows 64 * half on of the tile (of a pair the second
    // half is ready first)
    auto issue_pv = [&](int t, int buf, int half, int slot, bool acc) {
      const uint64_t vd = ring_desc_v + (uint64_t)((slot * C::kTileBytes + half * 64 * 128) >> 4);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        mma_ts(tmem + C::kOCol + (uint32_t)(D * t), tmem + 128u * t + 64u * buf + 8u * kk, vd + (uint64_t)(kk * 128),
               idesc_pv, (acc || kk > 0));
    };
    // Two row tiles: a tile's S fills both buffers at once (128 columns an instruction),
    //   S_0 | PV_0a PV_0b S_1 | ... for each;
    // one row tile: S runs one tile ahead of the softmax, S_0 S_1 | PV_0 S_2 | PV_1 S_3 | ...
    constexpr int kAhead = C::kPair ? 1 : 2;
    int fill = 0, seg = 0;      // ring slots, items
    int s_no[QT] = {}, p_no[QT] = {};  // tiles through S and through P V, by row tile
    bool ok = true;
    while (ok && walk.next(p)) {
      const int nt = walk.j1 - walk.j0;
      bool act[QT];
#pragma unroll
      for (int t = 0; t < QT; ++t) act[t] = tile_tokens(t) > 0;
      ok = mbar_wait_warp(q_bar, seg & 1, wctx, kPSiteQ);
      if (!ok) break;
      ++seg;
      auto multiply_s = [&](int t, int slot) {
        const int buf = C::kPair ? 0 : s_no[t] & 1;
        if (elect_one()) {
          issue_s(t, buf, slot);
          tc_commit(s_bar(t, buf));
        }
        __syncwarp();
        ++s_no[t];
      };
      auto wait_k = [&](int j) {
        const int f = fill + k_fill<C::kPair>(j);
        ok = mbar_wait_warp(full_bar(slot_of(f)), par_of(f), wctx, kPSiteKFull);
        tc_fence_after();
        return slot_of(f);
      };
      for (int j = 0; j < kAhead && j < nt && ok; ++j) {
        const int sk = wait_k(j);
        if (!ok) break;
#pragma unroll
        for (int t = 0; t < QT; ++t)
          if (act[t]) multiply_s(t, sk);
        if (elect_one()) {
          tc_commit(empty_bar(sk));
          if (j == nt - 1) tc_commit(qfree_bar);
        }
        __syncwarp();
      }
      for (int j = 0; j < nt && ok; ++j) {
        const int fv = fill + v_fill<C::kPair>(j, nt), sv = slot_of(fv);
        ok = mbar_wait_warp(full_bar(sv), par_of(fv), wctx, kPSiteVFull);
        if (!ok) break;
        bool cleared = false;
        int sk = -1;
#pragma unroll
        for (int t = 0; t < QT; ++t) {
          if (!act[t] || !ok) continue;
          const int buf = C::kPair ? 0 : p_no[t] & 1, par = C::kPair ? p_no[t] & 1 : (p_no[t] >> 1) & 1;
          ok = mbar_wait_warp(p_bar(t, C::kPair ? 1 : buf), par, wctx, kPSitePFull);
          if (!ok) break;
          tc_fence_after();
          // Row tile 0's warps have cleared what they had to; this one's have left the epilogue of every
          // earlier item.
          if (t == 0) cleared = *tail_hit == seg;
          if (cleared && lane == 0) odd[t] = seg;
          __syncwarp();
          if (elect_one()) {
            issue_pv(t, C::kPair ? 1 : buf, C::kPair ? 1 : 0, sv, j > 0);
            if (!C::kPair && j == nt - 2) tc_commit(pv_bar(t));
          }
          __syncwarp();
          if (C::kPair) {
            ok = mbar_wait_warp(p_bar(t, 0), par, wctx, kPSitePFull);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) issue_pv(t, 0, 0, sv, true);
            __syncwarp();
          }
          ++p_no[t];
          if (j == nt - 1) {
            if (elect_one()) tc_commit(o_bar(t));
            __syncwarp();
          } else if (j + kAhead < nt) {  // into the columns that P just left (the tensor pipe runs in order)
            if (sk < 0) sk = wait_k(j + kAhead);
            if (!ok) break;
            multiply_s(t, sk);
          }
        }
        if (elect_one()) {
          tc_commit(empty_bar(sv));
          if (sk >= 0) tc_commit(empty_bar(sk));
          if (sk >= 0 && j + kAhead == nt - 1) tc_commit(qfree_bar);
        }
        __syncwarp();
      }
      fill += 2 * nt;
    }
    // Drain: every MMA this warp issued completes before TMEM is released.
    if (seg > 0) {
      if (elect_one()) tc_commit(drain_bar);
      __syncwarp();
      if (!mbar_wait_warp(drain_bar, 0, wctx, kPSiteDrain) && *abort_flag) {
        const uint64_t t0 = global_timer_ns();
        while (!mbar_test(drain_bar, 0) && global_timer_ns() - t0 < kWaitLimitNs) {}
      }
    }
  } else {
    // ===================================================== TMA producer (whole warp; one lane per page of a tile)
    const uint64_t once = policy_evict_first();
    const int box_rows = min(p.g.page_size, BN), boxes = BN / box_rows;
    const int shift = 31 - __clz(p.g.page_size);
    const uint32_t ring = sbase + C::kOffRing;
    int fill = 0, seg = 0, tile = 0;
    bool ok = true;
    while (ok && walk.next(p)) {
      const int nt = walk.j1 - walk.j0;
      const int *row = p.g.page_table + (size_t)walk.b * p.g.max_pages;
      auto page_at = [&](int j) {  // this lane's page of tile j: -2 where the sequence has ended, -1 where there is none
        const int pos = j * BN + lane * box_rows;
        if (lane >= boxes || pos >= walk.s.keys) return -2;
        const int page = row[pos >> shift];
        return page >= 0 && page < p.g.num_pages ? page : -1;
      };
      // in the order of k_fill and v_fill
      auto load = [&](const CUtensorMap *map, int j, int page) {
        const int s = fill % C::kStages;
        ok = mbar_wait_warp(empty_bar(s), ((fill / C::kStages) & 1) ^ 1, wctx, kPSiteEmpty);
        if (!ok) return;
        if (lane == 0) mbar_arrive_expect_tx(full_bar(s), C::kTileBytes);
        __syncwarp();
        if (lane < boxes) {
          const int r0 = ((walk.j0 + j) * BN + lane * box_rows) & (p.g.page_size - 1);
#pragma unroll
          for (int bx = 0; bx < C::kBoxes; ++bx)
            tma_load_4d_hint(ring + s * C::kTileBytes + bx * C::kBoxBytes + lane * box_rows * 128, map, full_bar(s), bx * 64,
                             walk.kh, r0, max(page, -1), once);
        }
        ++fill;
      };
      int page = page_at(walk.j0), page_v = -2;
      for (int j = 0; j < nt + !C::kPair && ok; ++j) {
        const int page_next = j + 1 < nt ? page_at(walk.j0 + j + 1) : -2;
        if (j < nt) {
          unsigned gone = page == -1 ? ((1u << (box_rows / 16)) - 1u) << (lane * (box_rows / 16)) : 0u;
          gone = __reduce_or_sync(0xffffffffu, gone);
          if (lane == 0) bad[tile & 15] = gone;
          ++tile;
          load(&p.tm_k, j, page);
          if (!ok) break;
        }
        if (j == 0) {
          // Q after the first K tile: it may have to wait for the previous item's last S
          if (seg > 0) ok = mbar_wait_warp(qfree_bar, (seg - 1) & 1, wctx, kPSiteQFree);
          if (!ok) break;
          if (lane == 0) {
            int active = 0;
            for (int t = 0; t < QT; ++t) active += tile_tokens(t) > 0;
            mbar_arrive_expect_tx(q_bar, active * C::kBoxes * p.TB * p.G * 128);
            for (int t = 0; t < QT; ++t)
              if (tile_tokens(t) > 0)
                for (int bx = 0; bx < C::kBoxes; ++bx)
                  tma_load_4d_hint(sbase + C::kOffQ + t * C::kQBytes + bx * 16384, &p.tm_q, q_bar, bx * 64, 0, walk.kh,
                                   walk.s.start + (walk.rg * QT + t) * p.TB, once);
          }
          ++seg;
          __syncwarp();
        }
        if (C::kPair) load(&p.tm_v, j, page);
        else if (j > 0) load(&p.tm_v, j - 1, page_v);
        page_v = page;
        page = page_next;
      }
    }
    // Every copy issued lands before the block exits (normally they already have).
    const uint64_t t0 = global_timer_ns();
    for (int f = max(0, fill - C::kStages); f < fill; ++f)
      while (!mbar_test(full_bar(f % C::kStages), (f / C::kStages) & 1) && global_timer_ns() - t0 < kWaitLimitNs) {}
    if (seg > 0)
      while (!mbar_test(q_bar, (seg - 1) & 1) && global_timer_ns() - t0 < kWaitLimitNs) {}
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ------------------------------------------------------------------ few rows
// All rows of a kv head (new tokens x G heads) in one 16-row fragment: a decoding
// step, a short chain.  The cache is read once and each byte of it
// meets few multiplications, so HBM is the bound and the work around the tiles is
// what has to be small.  mma.sync.m16n8k16 fits: a warp takes 16 places of a
// tile through S, softmax and P V in its own registers (running maximum, sum and O
// of all rows over its own places), so warps only meet in the ring's barriers and,
// where several of them share a kv head, at an item's end.  The tcgen05 kernel pads
// the rows to 128 and passes S and P between warps for every tile.
//
// A tile is 64 / HB places of HB adjacent kv heads, four warps' work in any case.
// A head's row is only 128 to 512 bytes of the cache; fetching adjacent heads
// together keeps DRAM pages and 256-byte L2 lines whole, and with HB = 4 each warp
// has a head to itself and nothing to join.
// Measured with the join: 64 sequences of up to 8192 places, one token each, 32 on 8
// heads of dim 128: 154 to 156 us, 6.6 TB/s (the tcgen05 kernel: 164); 32 of up to 2500,
// chains of up to 7, 16 heads of dim 64: 33 us, 5.0 TB/s, of which some 8 are set-up,
// the first tiles and the join.
template <int D>
struct FewCfg {
  static constexpr int kWarps = 4, kBoxes = D / 64;
  static constexpr int kThreads = 32 * (kWarps + 1);
  static constexpr int kTileBytes = 16 * kWarps * D * 2;  // K or V of a tile
  static constexpr int kMinBlocks = D <= 128 ? 2 : 1;
  static constexpr int kSmemMax = kMinBlocks == 2 ? 113 * 1024 : 227 * 1024;
  static constexpr int kJoinBytes = (kWarps / 2) * 16 * D * 4;
  static constexpr int kStagesFit = (kSmemMax - 1024 - 1024 - kJoinBytes) / (2 * kTileBytes);
  static constexpr int kStages = D == 64 ? kNarrowRing / kMinBlocks / (2 * kTileBytes) : kStagesFit;
  static_assert(kStages >= 2 && kStages <= kStagesFit, "ring");
  static constexpr int kOffRing = 0, kOffJoin = 2 * kStages * kTileBytes, kOffBar = kOffJoin + kJoinBytes;
  static constexpr int kOffMisc = kOffBar + 16 * kStages;
  static constexpr int kOffML = kOffMisc + 96;  // [kWarps][16] float2
  static constexpr int kOffSums = kOffML + kWarps * 16 * 8;
  static constexpr int kSmemBytes = kOffSums + 8 * (kWarps + 1) + 1024;
  static_assert(kSmemBytes <= kSmemMax, "shared memory budget");
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
enum FewSite : int { kFSiteFull = 41, kFSiteEmpty = 42 };

template <int D>
__global__ void __launch_bounds__(FewCfg<D>::kThreads, FewCfg<D>::kMinBlocks)
    paged_few_kernel(const __grid_constant__ PagedParams p) {
  using C = FewCfg<D>;
  constexpr int W = C::kWarps;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto full_bar = [&](int s) { return sbase + C::kOffBar + 8u * s; };
  auto empty_bar = [&](int s) { return sbase + C::kOffBar + 8u * (C::kStages + s); };
  uint8_t *misc = smem + C::kOffMisc;
  volatile int *abort_flag = reinterpret_cast<volatile int *>(misc);
  volatile int *odd = reinterpret_cast<volatile int *>(misc + 4);             // the last item with cleared V values
  PagedStart *at = reinterpret_cast<PagedStart *>(misc + 8);                  // 48 bytes
  volatile unsigned *bad = reinterpret_cast<volatile unsigned *>(misc + 56);  // [kStages] granules without a page
  static_assert(sizeof(PagedStart) <= 48 && 56 + 4 * C::kStages <= 96, "");
  float2 *s_ml = reinterpret_cast<float2 *>(smem + C::kOffML);
  const WaitCtx wctx{abort_flag, p.status};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bn = 1 << p.bn_log2;
  const int box_bytes = bn * 128, head_bytes = bn * D * 2;  // a 64-column box, a head's part of a tile
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), W);
    }
    *abort_flag = 0;
    *odd = 0;
    at->b = -1;
    fence_mbar_init();
  }
  if (warp == W && lane == 0) {
    prefetch_tmap(&p.tm_k);
    prefetch_tmap(&p.tm_v);
  }
  grid_wait();
  grid_go();  // only now: the join reads the call's inputs without a wait of its own
  if (!p.by_warp) block_stretch<C::kThreads>(p, reinterpret_cast<long long *>(smem + C::kOffSums), at);
  __syncthreads();
  PagedWalk walk;
  walk.start(p, p.by_warp ? warp_stretch(p) : *at);
  bool ok = true;

  if (warp < W) {
    const int q4 = lane >> 2, c4 = (lane & 3) * 2;
    const int sharers = W / p.HB, hb = warp / sharers, sub = warp - hb * sharers;  // warps of a kv head
    const float c2 = p.scale_log2;
    int fill = 0, item = 0;
    while (walk.next(p)) {
      ++item;
      const int nt = walk.j1 - walk.j0, rows = walk.s.n * p.G, kh = walk.kh * p.HB + hb;
      // this thread's rows: q4 and q4 + 8
      uint32_t qf[D / 16][4];
      int tok[2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int r = 8 * hf + q4;
          tok[hf] = r / p.G;
          const uint32_t *qr = reinterpret_cast<const uint32_t *>(
              p.q + ((size_t)(walk.s.start + tok[hf]) * p.H + kh * p.G + (r - tok[hf] * p.G)) * D);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            qf[k][hf] = r < rows ? qr[8 * k + (lane & 3)] : 0u;
            qf[k][hf + 2] = r < rows ? qr[8 * k + 4 + (lane & 3)] : 0u;
          }
        }
      auto words = [&](int hf) {
        return p.mask && 8 * hf + q4 < rows ? p.mask + (size_t)(walk.s.start + tok[hf]) * p.words : nullptr;
      };
      float o[D / 8][4], m_ref[2], l_sum[2];
      m_ref[0] = m_ref[1] = -INFINITY;
      l_sum[0] = l_sum[1] = 0.f;
#pragma unroll
      for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
      bool cleared = false;
      for (int j = 0; j < nt; ++j, ++fill) {
        const int slot = fill % C::kStages;
        if (ok) ok = mbar_wait_warp(full_bar(slot), (fill / C::kStages) & 1, wctx, kFSiteFull);
        const int kv0 = (walk.j0 + j) * bn + 16 * sub;
        if (ok && kv0 < walk.s.keys && !((bad[slot] >> sub) & 1)) {
          const uint32_t kt = sbase + C::kOffRing + 2 * slot * C::kTileBytes + hb * head_bytes + 16 * sub * 128;
          const uint32_t vt = kt + C::kTileBytes;
          float s[2][4] = {};
          {
            const int key = (lane & 7) + ((lane >> 4) << 3), half = (lane >> 3) & 1;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              uint32_t kf[4];
              ldsm4(kf, kt + (k >> 2) * box_bytes + key * 128 + (((2 * (k & 3) + half) ^ (key & 7)) << 4));
              mma16816(s[0], qf[k], kf[0], kf[1]);
              mma16816(s[1], qf[k], kf[2], kf[3]);
            }
          }
          const bool tail = kv0 + 16 > walk.s.len;
          if (tail) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const int pre = walk.s.len - kv0;
              const unsigned see = (pre <= 0 ? 0u : (1u << pre) - 1u) |
                                   seen_bits(words(hf), tok[hf], walk.s.keys - walk.s.len, kv0 - walk.s.len);
#pragma unroll
              for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (!((see >> (8 * n + c4 + e)) & 1)) s[n][2 * hf + e] = -INFINITY;
            }
          }
          uint32_t pf[4];
          float top[2];
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
            top[hf] = fmaxf(fmaxf(s[0][2 * hf], s[0][2 * hf + 1]), fmaxf(s[1][2 * hf], s[1][2 * hf + 1])) * c2;
          // the maximum moves only where a score is more than kRescaleTau above it (at first: above -inf);
          // the weights below go to P V in bf16 (2^-8 each), to the row sum unrounded, as in paged_fwd_kernel
          if (__any_sync(0xffffffffu, top[0] - m_ref[0] > kRescaleTau || top[1] - m_ref[1] > kRescaleTau)) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              float t = top[hf];
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
              t = fmaxf(t, m_ref[hf]);
              const float alpha = t == m_ref[hf] ? 1.f : ex2_mufu(m_ref[hf] - t);
              m_ref[hf] = t;
              l_sum[hf] *= alpha;
#pragma unroll
              for (int n = 0; n < D / 8; ++n) {
                o[n][2 * hf] *= alpha;
                o[n][2 * hf + 1] *= alpha;
              }
            }
          }
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const float neg = m_ref[hf] == -INFINITY ? 0.f : -m_ref[hf];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const float e0 = ex2_mufu(fmaf(s[n][2 * hf], c2, neg)), e1 = ex2_mufu(fmaf(s[n][2 * hf + 1], c2, neg));
              l_sum[hf] += e0 + e1;
              pf[2 * n + hf] = pack_bf16x2(e0, e1);
            }
          }
          const int key = lane & 15, part = lane >> 4;
          if (!tail) {
#pragma unroll
            for (int n = 0; n < D / 16; ++n) {
              uint32_t vf[4];
              ldsm4_t(vf, vt + (n >> 2) * box_bytes + key * 128 + (((2 * (n & 3) + part) ^ (key & 7)) << 4));
              mma16816(o[2 * n], pf, vf[0], vf[1]);
              mma16816(o[2 * n + 1], pf, vf[2], vf[3]);
            }
          } else {
            // Values that not every row sees: past the end they hold anything, and 0 * NaN is NaN; among
            // the new tokens non-finite ones are left out and added at the item's end to the rows that
            // see them.  vf[0], vf[2] hold places c4, c4 + 1; vf[1], vf[3] the ones 8 further.
            const int left = walk.s.keys - kv0 - c4, fresh = walk.s.len - kv0 - c4;
            auto cut = [&](uint32_t w, int at) {
              const uint32_t was = w;
              const uint32_t f = finite_pair(w);
              if (fresh <= at) w = (w & 0xffff0000u) | (f & 0xffffu);
              if (fresh <= at + 1) w = (w & 0x0000ffffu) | (f & 0xffff0000u);
              cleared |= w != was && left > at;
              if (left <= at) w &= 0xffff0000u;
              if (left <= at + 1) w &= 0x0000ffffu;
              return w;
            };
#pragma unroll
            for (int n = 0; n < D / 16; ++n) {
              uint32_t vf[4];
              ldsm4_t(vf, vt + (n >> 2) * box_bytes + key * 128 + (((2 * (n & 3) + part) ^ (key & 7)) << 4));
              vf[0] = cut(vf[0], 0);
              vf[1] = cut(vf[1], 8);
              vf[2] = cut(vf[2], 0);
              vf[3] = cut(vf[3], 8);
              mma16816(o[2 * n], pf, vf[0], vf[1]);
              mma16816(o[2 * n + 1], pf, vf[2], vf[3]);
            }
          }
        }
        if (!(FA_STALL(5) && fill == 0 && warp == 0)) mbar_arrive_warp(empty_bar(slot));
      }
      float row_l[2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          float l = l_sum[hf];
          l += __shfl_xor_sync(0xffffffffu, l, 1);
          l += __shfl_xor_sync(0xffffffffu, l, 2);
          row_l[hf] = l;  // m_ref is the row's already: its lanes moved it together
        }
      bool is_odd = __any_sync(0xffffffffu, cleared);
      if (sharers > 1) {
        // ----------------------------------------------------- join the warps of a kv head
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
            if ((lane & 3) == 0)
              s_ml[warp * 16 + 8 * hf + q4] = make_float2(m_ref[hf], row_l[hf]);
        if (is_odd && lane == 0) *odd = item;
        named_bar_sync(1, 32 * W);
        is_odd = *odd == item;
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const float2 *ml = s_ml + hb * sharers * 16 + 8 * hf + q4;
            float top = -INFINITY, l = 0.f;
            for (int w = 0; w < sharers; ++w) top = fmaxf(top, ml[w * 16].x);
            const float base = top == -INFINITY ? 0.f : top;
            for (int w = 0; w < sharers; ++w) {
              const float2 x = ml[w * 16];
              l += x.y * ex2_mufu(x.x - base);
            }
            const float a = ex2_mufu(m_ref[hf] - base);
            m_ref[hf] = top;
            row_l[hf] = l;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
              o[n][2 * hf] *= a;
              o[n][2 * hf + 1] *= a;
            }
          }
        float4 *join = reinterpret_cast<float4 *>(smem + C::kOffJoin);  // [W / 2][D / 8][32 lanes]
        for (int step = sharers / 2; step >= 1; step >>= 1) {
          if (sub >= step && sub < 2 * step) {
            float4 *to = join + (hb * step + sub - step) * (D / 8) * 32 + lane;
#pragma unroll
              for (int n = 0; n < D / 8; ++n)
                to[n * 32] = make_float4(o[n][0], o[n][1], o[n][2], o[n][3]);
          }
          named_bar_sync(1, 32 * W);
          if (sub < step) {
            const float4 *from = join + (hb * step + sub) * (D / 8) * 32 + lane;
#pragma unroll
              for (int n = 0; n < D / 8; ++n) {
                const float4 x = from[n * 32];
                o[n][0] += x.x;
                o[n][1] += x.y;
                o[n][2] += x.z;
                o[n][3] += x.w;
              }
          }
          named_bar_sync(1, 32 * W);
        }
      }
      if (sub == 0 && ok) {
        if (is_odd) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
              for (int n = 0; n < D / 8; ++n) {
                if (8 * hf + q4 >= rows) continue;
                float add[2];
                add_unfinite(p, walk.s, walk.b, kh, words(hf), tok[hf], walk.j0 * bn, walk.j1 * bn, D, 8 * n + c4, 2, add);
                o[n][2 * hf] += add[0];
                o[n][2 * hf + 1] += add[1];
              }
        }
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const int r = 8 * hf + q4;
            if (r >= rows) continue;
            const float l = row_l[hf];
            if (walk.whole) {
              const int h = kh * p.G + (r - tok[hf] * p.G);
              const size_t q_row = (size_t)walk.s.start + tok[hf];
              const float inv = l == 0.f ? 0.f : 1.0f / l;
              uint32_t *to = reinterpret_cast<uint32_t *>(p.o + (q_row * p.H + h) * D + c4);
#pragma unroll
              for (int n = 0; n < D / 8; ++n) to[4 * n] = pack_bf16x2(o[n][2 * hf] * inv, o[n][2 * hf + 1] * inv);
              if ((lane & 3) == 0 && p.lse) p.lse[(size_t)h * p.total + q_row] = (m_ref[hf] + __log2f(l)) * 0.69314718055994531f;
            } else {
              const int GG = p.HB * p.G, all = p.TB * GG, row = tok[hf] * GG + hb * p.G + (r - tok[hf] * p.G);
              const size_t slot = ((size_t)blockIdx.x * 2 + (walk.first ? 0 : 1)) * all;
              float *to = p.part_o + slot * D + c4 * all + row;
#pragma unroll
              for (int n = 0; n < D / 8; ++n, to += 8 * all) {
                to[0] = o[n][2 * hf];
                to[all] = o[n][2 * hf + 1];
              }
              if ((lane & 3) == 0) p.part_ml[slot + row] = make_float2(m_ref[hf], l);
            }
          }
      }
    }
  } else {
    // ===================================================== TMA producer: one lane per page, head, and K or V
    const uint64_t once = policy_evict_first();
    const int box_rows = min(p.g.page_size, bn), boxes = bn / box_rows;
    const int shift = 31 - __clz(p.g.page_size);
    // lane = (kv * HB + head) * boxes + box: at most 2 * HB * (64 / HB) / 16 = 8 lanes
    const int box = lane % boxes, head = lane / boxes % p.HB, kv = lane / (boxes * p.HB);
    int fill = 0;
    while (ok && walk.next(p)) {
      const int *row = p.g.page_table + (size_t)walk.b * p.g.max_pages;
      auto page_at = [&](int j) {  // -2 where the sequence has ended, -1 where there is no page
        const int pos = j * bn + box * box_rows;
        if (kv > 1 || pos >= walk.s.keys) return -2;
        const int page = row[pos >> shift];
        return page >= 0 && page < p.g.num_pages ? page : -1;
      };
      int page = page_at(walk.j0);
      for (int j = walk.j0; j < walk.j1 && ok; ++j, ++fill) {
        const int page_next = j + 1 < walk.j1 ? page_at(j + 1) : -2;
        const int s = fill % C::kStages;
        ok = mbar_wait_warp(empty_bar(s), ((fill / C::kStages) & 1) ^ 1, wctx, kFSiteEmpty);
        if (!ok) break;
        unsigned gone = page == -1 ? ((1u << (box_rows / 16)) - 1u) << (box * (box_rows / 16)) : 0u;
        gone = __reduce_or_sync(0xffffffffu, gone);
        if (lane == 0) {
          bad[s] = gone;
          mbar_arrive_expect_tx(full_bar(s), 2 * C::kTileBytes);
        }
        __syncwarp();
        if (kv < 2) {
          const int r0 = (j * bn + box * box_rows) & (p.g.page_size - 1);
          const uint32_t to = sbase + C::kOffRing + (2 * s + kv) * C::kTileBytes + head * head_bytes + box * box_rows * 128;
#pragma unroll
          for (int bx = 0; bx < C::kBoxes; ++bx)
            tma_load_4d_hint(to + bx * box_bytes, kv ? &p.tm_v : &p.tm_k, full_bar(s), bx * 64, walk.kh * p.HB + head, r0,
                             max(page, -1), once);
        }
        page = page_next;
      }
    }
    const uint64_t t0 = global_timer_ns();
    for (int f = max(0, fill - C::kStages); f < fill; ++f)
      while (!mbar_test(full_bar(f % C::kStages), (f / C::kStages) & 1) && global_timer_ns() - t0 < kWaitLimitNs) {}
  }
}

// Joins the parts of the items that were cut.  Blocks go by (item, chunks of it); one
// warp finds out where the item's parts are, the others take it from there: the search
// for every row by every thread was half of this kernel's time.  With up to 32 sequences
// that is before the wait for the main kernel, on lengths read from L2; with more, all is
// read after it.  A task is COLS columns
// of one row; with many parts (SHARED) p.join warps share 32 tasks and take every
// join-th part each, U of them in flight.  Parts are stored column by column, so that
// neighbouring tasks are contiguous for the kernels' stores and the loads here.  Bound
// by latency: launch, the item's place, two rounds of loads from L2; 5 us after the main
// kernel for 8 items of 256 rows in 19 parts each (21 MB, 10 us from DRAM).  At 72
// registers those 1024 blocks run at once (80: 38.0 instead of 37.4 us for the call).
constexpr int kJoinWarps = 8;  // at most; four unless all eight share their tasks
// Blocks of four warps: some 6 to 7 run at once on an SM, and many items are whole or
// short, whose blocks end at once.  (7 to an SM, each with more chunks: 48 ragged trees of
// 64 rows 59.6 instead of 54.5 us; 20: 55.4.)
constexpr int kJoinWave = 14 * 152;

template <int D, bool SHARED>
__global__ void __maxnreg__(SHARED ? 72 : 80) paged_combine_kernel(const __grid_constant__ PagedParams p, int blocks) {
  constexpr int COLS = 8, U = 4;  // one 16-byte store a task
  __shared__ float s_part[SHARED ? kJoinWarps : 1][COLS + 2][32];
  __shared__ PagedSeq s_seq;
  __shared__ unsigned s_u0, s_total;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int GG = p.HB * p.G, all = p.QT * p.TB * GG;
  const int b = (int)blockIdx.x / p.heads, kh = (int)blockIdx.x - b * p.heads;
  const int rg = min((int)blockIdx.y / p.join_y, p.groups - 1);
  const int chunk0 = (int)blockIdx.y - rg * p.join_y;
  const int chunk_step = rg < p.groups - 1 ? p.join_y : (int)gridDim.y - (p.groups - 1) * p.join_y;
  // Up to 32 sequences: one warp fetches what the call's tables say of the sequence and of the units before it,
  // before the wait, so that blocks with nothing to join can end.  More: after it, together with p.prefix.
  PagedSeq s;
  long long u0 = 0, total = 0;
  if (p.by_warp) {
    if (warp == 0) {
      const WarpUnits w = warp_units<true>(p);
      if (lane == b) {
        s_seq = w.s;
        s_u0 = w.before;
      }
      if (lane == 0) s_total = w.total;
    }
    __syncthreads();
    s = s_seq;
    u0 = s_u0;
    total = s_total;
  } else {
    grid_go();
    grid_wait();
    u0 = p.prefix[b];
    total = p.prefix[p.g.B];
    s = paged_seq(p, b);
  }
  const int tok0 = rg * p.QT * p.TB, rows = min(s.n - tok0, p.QT * p.TB) * GG;
  int tiles, groups;
  paged_units(p, s, tiles, groups);
  // the item's parts: from the block with its first tile on
  int c0 = 0, parts = 0, first = 0;
  auto find_parts = [&] {
    const long long per = stretch_units(p, total, blocks), at = u0 + (long long)(kh * groups + rg) * (tiles + p.lead);
    c0 = (int)quot(at + p.lead, per);
    parts = (int)quot(at + p.lead + tiles - 1, per) - c0 + 1;
    // only the first block can have had tiles of another item before this one's: it began before this
    // item's units (the one before them is a tile), and this is its second part
    first = 2 * c0 + (at > c0 * per ? 1 : 0);
  };
  if (rows > 0) find_parts();
  // Nothing to join: no such row group, or one block had it all and has written the result.  The first
  // block waits in any case, so that the grid does not end before the main kernel has.
  const bool idle = rows <= 0 || parts == 1;
  if (p.by_warp) {
    grid_go();
    if (idle && (blockIdx.x | blockIdx.y) != 0) return;
    grid_wait();
  }
  if (idle) return;
  const int share = warp % p.join, tasks = rows * (D / COLS), step = (int)blockDim.x / p.join;
  for (int base = chunk0 * step; base < tasks; base += chunk_step * step) {
    const int task = base + warp / p.join * 32 + lane;
    const int cg = task / rows, row = task - cg * rows;
    const bool mine = task < tasks;
    float m = -INFINITY, l = 0.f, acc[COLS] = {};
    for (int k0 = share; k0 < parts && mine; k0 += U * p.join) {
      float2 ml[U];
      float x[U][COLS];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u * p.join;
        ml[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int e = 0; e < COLS; ++e) x[u][e] = 0.f;
        if (k < parts) {
          const unsigned at = (unsigned)(k == 0 ? first : (c0 + k) * 2) * all;  // < 2^20 rows in all
          ml[u] = p.part_ml[at + row];
          const float *from = p.part_o + (at * D + COLS * cg * all + row);
#pragma unroll
          for (int e = 0; e < COLS; ++e, from += all) x[u][e] = *from;
        }
      }
      float m_new = m;
#pragma unroll
      for (int u = 0; u < U; ++u) m_new = fmaxf(m_new, ml[u].x);
      const float top = m_new == -INFINITY ? 0.f : m_new, a = ex2_mufu(m - top);
      m = m_new;
      l *= a;
#pragma unroll
      for (int e = 0; e < COLS; ++e) acc[e] *= a;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float w = ex2_mufu(ml[u].x - top);
        l += ml[u].y * w;
#pragma unroll
        for (int e = 0; e < COLS; ++e) acc[e] += x[u][e] * w;
      }
    }
    if constexpr (SHARED) {
      __syncthreads();
      s_part[warp][COLS][lane] = m;
      s_part[warp][COLS + 1][lane] = l;
#pragma unroll
      for (int e = 0; e < COLS; ++e) s_part[warp][e][lane] = acc[e];
      __syncthreads();
      if (share != 0) continue;
      for (int w = warp + 1; w < warp + p.join; ++w) {
        const float mw = s_part[w][COLS][lane], m_new = fmaxf(m, mw), top = m_new == -INFINITY ? 0.f : m_new;
        const float a = ex2_mufu(m - top), aw = ex2_mufu(mw - top);
        m = m_new;
        l = l * a + s_part[w][COLS + 1][lane] * aw;
#pragma unroll
        for (int e = 0; e < COLS; ++e) acc[e] = acc[e] * a + s_part[w][e][lane] * aw;
      }
    }
    if (!mine) continue;
    const int tok = row / GG, h = kh * GG + row - tok * GG;
    const size_t q_row = (size_t)s.start + tok0 + tok;
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    uint32_t w[COLS / 2];
#pragma unroll
    for (int e = 0; e < COLS / 2; ++e) w[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    *reinterpret_cast<uint4 *>(p.o + (q_row * p.H + h) * D + COLS * cg) = make_uint4(w[0], w[1], w[2], w[3]);
    if (cg == 0 && p.lse)
      p.lse[(size_t)h * p.total + q_row] = ((m == -INFINITY ? 0.f : m) + __log2f(l)) * 0.69314718055994531f;
  }
}

constexpr int kMaxNew = 256;

int check_paged(int B, int max_pages, int num_pages, int page_size, int max_new, int total, int H, int Hkv, int d) {
  int rc = check_page_table(B, max_pages, num_pages, page_size);
  if (rc == FA_OK) rc = check_page_rows(1, num_pages, page_size, Hkv, d);
  if (rc != FA_OK) return rc;
  if (H <= 0 || H % Hkv != 0 || max_new <= 0 || total < 0) return FA_ERR_INVALID_ARG;
  if (H > 65535 || H / Hkv > 128 || max_new > kMaxNew) return FA_ERR_UNSUPPORTED;
  if ((double)total * H * d >= (double)(1ll << 40) || (double)total * H > 2147483647.0) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// Blocks of the main kernel: as many as run at once.  (The SM count of a GB300;
// the result does not depend on it.)
constexpr int kSMs = 152;

// Places in a tile of the tcgen05 kernel: a pair of halves where a block has two row tiles.
constexpr int tile_keys(int QT) { return QT == 2 ? 128 : 64; }

struct PagedPlan {
  bool few;  // the few-rows kernel, else the tcgen05 kernel
  int QT, HB, bn, TB, blocks;
  size_t part_o, part_ml, prefix, bytes;
};

PagedPlan paged_plan(int B, int max_new, int Hkv, int G, int d) {
  PagedPlan w;
  const int rows = max_new * G;
  // One 16-row fragment.  (Two of them, at dims 64 and 128, were 40 % slower on 16 x 8000 places at 32 rows than
  // the tcgen05 kernel at dim 128, and 30 % at dim 64.)
  w.few = rows <= 16;
  w.TB = 128 / G < max_new ? 128 / G : max_new;
  w.QT = max_new > w.TB && d <= 128 ? 2 : 1;
  w.HB = !w.few ? 1 : Hkv % 4 == 0 ? 4 : Hkv % 2 == 0 ? 2 : 1;
  w.bn = w.few ? 64 / w.HB : tile_keys(w.QT);
  w.blocks = kSMs * (w.few ? (d <= 128 ? 2 : 1) : (w.QT == 1 && d <= 128 ? 2 : 1));
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  const size_t slots = (size_t)2 * w.blocks * w.HB * w.QT * w.TB * G;
  w.part_o = 0;
  w.part_ml = up(slots * d * 4);
  w.prefix = w.part_ml + up(slots * 8);
  w.bytes = w.prefix + up(((size_t)B + 1) * 8);
  return w;
}

// The main kernel, then the join.
int launch_two(PagedParams &p, int d, int blocks, int threads, int smem, void (*main)(PagedParams),
               void (*join)(PagedParams, int), cudaStream_t stream) {
  // on every launch: the attribute belongs to the function on the current device
  if (cudaFuncSetAttribute(main, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return FA_ERR_CUDA;
  const int rc = launch_after(main, blocks, 1, threads, smem, stream, p);
  if (rc != FA_OK) return rc;
  // for each (sequence, kv heads) blocks for chunks of its row groups, the last of which may be short: at most
  // kJoinWave in all, and one to a row group at least
  const long long line = (long long)p.g.B * p.heads;
  const int threads_join = 32 * (p.join > 4 ? p.join : 4), step = threads_join / p.join;
  const int full = p.QT * p.TB, last = p.max_new - (p.groups - 1) * full;
  auto chunks = [&](int tokens) { return (tokens * p.HB * p.G * (d / 8) + step - 1) / step; };
  const long long wave = kJoinWave * 128 / threads_join / line;
  long long many = wave / p.groups, end = many < chunks(last) ? many : chunks(last);
  if (end < 1) end = 1;
  if (p.groups > 1) many = (wave - end) / (p.groups - 1);
  if (many > chunks(full)) many = chunks(full);
  p.join_y = many < 1 ? 1 : (int)many;
  return launch_after(join, line, (int)((p.groups - 1) * p.join_y + end), threads_join, 0, stream, p, blocks);
}

int page_maps(PagedParams &p, const void *k_pages, const void *v_pages, int d) {
  // one head of dim 64 at a time: its neighbour's 128 bytes would be fetched and lost (measured 63 against 80 %
  // of the copy rate at 8000 places, 16 heads)
  const bool narrow = d == 64 && p.HB == 1;
  const int bn = 1 << p.bn_log2, box_rows = p.g.page_size < bn ? p.g.page_size : bn;
  return encode_page_map(&p.tm_k, k_pages, p.g.num_pages, p.g.page_size, p.Hkv, d, box_rows, narrow) ||
                 encode_page_map(&p.tm_v, v_pages, p.g.num_pages, p.g.page_size, p.Hkv, d, box_rows, narrow)
             ? FA_ERR_CUDA
             : FA_OK;
}

template <int D, int BN, int QT>
int launch_paged(PagedParams &p, int blocks, const void *q, const void *k_pages, const void *v_pages,
                 cudaStream_t stream) {
  using C = PagedCfg<D, BN, QT>;
  const uint64_t dims[4] = {(uint64_t)D, (uint64_t)p.G, (uint64_t)p.Hkv, (uint64_t)p.total};
  const uint64_t strides[3] = {(uint64_t)D * 2, (uint64_t)p.G * D * 2, (uint64_t)p.H * D * 2};
  const uint32_t box[4] = {64, (uint32_t)p.G, 1, (uint32_t)p.TB};
  if (encode_bf16_box_map(&p.tm_q, q, dims, strides, box) || page_maps(p, k_pages, v_pages, D)) return FA_ERR_CUDA;
  return launch_two(p, D, blocks, C::kThreads, C::kSmemBytes, paged_fwd_kernel<D, BN, QT>,
                    p.join > 1 ? paged_combine_kernel<D, true> : paged_combine_kernel<D, false>, stream);
}

template <int D>
int launch_few(PagedParams &p, int blocks, const void *k_pages, const void *v_pages, cudaStream_t stream) {
  using C = FewCfg<D>;
  if (page_maps(p, k_pages, v_pages, D)) return FA_ERR_CUDA;
  return launch_two(p, D, blocks, C::kThreads, C::kSmemBytes, paged_few_kernel<D>,
                    p.join > 1 ? paged_combine_kernel<D, true> : paged_combine_kernel<D, false>, stream);
}

}  // namespace

#ifdef FA_TEST_STALL
int set_test_stall_paged(int mode) {
  return cudaMemcpyToSymbol(g_test_stall, &mode, sizeof(int)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
#endif

}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_fwd_paged_workspace_bytes(int B, int max_new, int H, int Hkv, int d) {
  if (check_paged(B, 1, 1, 16, max_new, 0, H, Hkv, d) != FA_OK) return 0;
  return paged_plan(B, max_new, Hkv, H / Hkv, d).bytes;
}

int fa_fwd_paged(const void *q, const void *k_pages, const void *v_pages, const int *page_table,
                 const int *cache_lens, const int *cu_seqlens, const long long *tree_mask, int mask_words, void *o,
                 float *lse, int B, int max_pages, int num_pages, int page_size, int max_new, int total, int H,
                 int Hkv, int d, float scale, void *workspace, size_t workspace_bytes, void *stream) {
  if (!q || !k_pages || !v_pages || !page_table || !cache_lens || !cu_seqlens || !o) return FA_ERR_INVALID_ARG;
  int rc = check_paged(B, max_pages, num_pages, page_size, max_new, total, H, Hkv, d);
  if (rc != FA_OK) return rc;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (tree_mask && (long long)mask_words * 64 < max_new) return FA_ERR_INVALID_ARG;
  const PagedPlan w = paged_plan(B, max_new, Hkv, H / Hkv, d);
  // the units of one sequence are counted in 31 bits, and so are the items
  const double seq_units = ((double)max_pages * page_size / w.bn + 8) * (Hkv / w.HB) * ((max_new + w.TB - 1) / w.TB);
  const int groups = (max_new + w.TB * w.QT - 1) / (w.TB * w.QT);
  const long long items = (long long)B * (Hkv / w.HB) * groups;
  if (seq_units >= 2147483648.0 || items > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  for (const void *x : {q, k_pages, v_pages, (const void *)o})
    if (!ptr_aligned(x, 16)) return FA_ERR_ALIGNMENT;
  for (const void *x : {(const void *)page_table, (const void *)cache_lens, (const void *)cu_seqlens, (const void *)lse})
    if (!ptr_aligned(x, 4)) return FA_ERR_ALIGNMENT;
  if (!ptr_aligned(tree_mask, 8)) return FA_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < fa_fwd_paged_workspace_bytes(B, max_new, H, Hkv, d) || !ptr_aligned(workspace, 256))
    return FA_ERR_WORKSPACE;
  if ((rc = check_device()) != FA_OK) return rc;
  if (total == 0) return FA_OK;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  PagedParams p;
  p.q = static_cast<const __nv_bfloat16 *>(q);
  p.v_pages = static_cast<const __nv_bfloat16 *>(v_pages);
  p.cu = cu_seqlens;
  p.mask = reinterpret_cast<const unsigned long long *>(tree_mask);
  p.o = static_cast<__nv_bfloat16 *>(o);
  p.lse = lse;
  p.part_o = reinterpret_cast<float *>(ws + w.part_o);
  p.part_ml = reinterpret_cast<float2 *>(ws + w.part_ml);
  p.prefix = reinterpret_cast<long long *>(ws + w.prefix);
  p.status = device_status_ptr();
  if (!p.status) return FA_ERR_CUDA;
  p.g = PageGeom{page_table, cache_lens, B, max_pages, num_pages, page_size};
  p.words = mask_words;
  p.max_new = max_new;
  p.total = total;
  p.H = H;
  p.Hkv = Hkv;
  p.G = H / Hkv;
  p.TB = w.TB;
  p.bn_log2 = w.bn == 128 ? 7 : w.bn == 64 ? 6 : w.bn == 32 ? 5 : 4;
  p.heads = Hkv / w.HB;
  p.by_warp = B <= 32 && B * seq_units < 2147483648.0 - 4 * kSMs;
  p.min_units = w.few ? 2 : 1;
  // In microseconds, against none: 48 ragged sequences of drafted trees 54 (63), at head dim 64 44 (74), at
  // head dim 256 48 (56); 96 short sequences, one token each 25.7 (28.3).
  p.lead = w.few ? 2 : w.QT == 2 ? 4 : 3;
  p.groups = groups;
  // Warps to a task of the join: by the parts of an item, as long as they make one wave.
  const long long tasks = items * w.QT * w.TB * w.HB * (H / Hkv) * (d / 8);
  p.join = 1;
  while (p.join < 8 && 4 * p.join <= w.blocks / items + 1 && tasks * 2 * p.join <= 28ll * 32 * kSMs) p.join *= 2;
  p.QT = w.QT;
  p.HB = w.HB;
  p.scale_log2 = scale * 1.4426950408889634f;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (w.few) {
    if (d == 64) return launch_few<64>(p, w.blocks, k_pages, v_pages, s);
    if (d == 128) return launch_few<128>(p, w.blocks, k_pages, v_pages, s);
    return launch_few<256>(p, w.blocks, k_pages, v_pages, s);
  }
  if (d == 64)
    return w.QT == 2 ? launch_paged<64, tile_keys(2), 2>(p, w.blocks, q, k_pages, v_pages, s)
                     : launch_paged<64, tile_keys(1), 1>(p, w.blocks, q, k_pages, v_pages, s);
  if (d == 128)
    return w.QT == 2 ? launch_paged<128, tile_keys(2), 2>(p, w.blocks, q, k_pages, v_pages, s)
                     : launch_paged<128, tile_keys(1), 1>(p, w.blocks, q, k_pages, v_pages, s);
  return launch_paged<256, tile_keys(1), 1>(p, w.blocks, q, k_pages, v_pages, s);
}

}  // extern "C"
