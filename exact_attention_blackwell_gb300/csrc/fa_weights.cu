// fa_weights.cu — attention weight that the places of a paged cache get from new tokens:
// for sequence b, kv head h and place p,
//   w[b, h, p] = decay w[b, h, p] + sum over tokens i that see p and heads g of h's group
//                of exp(scale q_ig . k_p - lse_ig)
// (which places a token sees: as in fa_paged.cu).
#include <cuda_bf16.h>

#include <cmath>

#include "fa_paged.h"
#include "paged_seq.h"
#include "ptx.cuh"

namespace fa {
namespace {

// Work.  The products are taken the other way round than for attention: S^T = K Q^T with
// 128 places as the MMA's rows and the new tokens' rows (tokens x G heads of a kv head) as
// its columns.  A thread then has one place and adds up its columns: no sum crosses threads,
// nothing is joined, and each place of a kv head belongs to one block, whatever the
// division of work.  More rows than the columns of a product come in chunks, each
// multiplied with the tiles in shared memory.
//
// A unit is two neighbouring tiles of one kv head, one for each of the block's two
// warpgroups; it costs its sequence's number of chunks.  Units stand in one line (sequence,
// group of HB kv heads, pair of tiles, head), so that the rows of neighbouring heads, which
// are neighbours in memory, are fetched at about the same time, and what surrounds a place (its
// page, who sees it) is looked at once for a run of them; the line is cut by cost into equal
// stretches for the blocks, which begin with the first unit that begins in theirs.
//
// Bound by HBM with few rows: 64 users of up to 8192 places, one token, 32 on 8 heads of dim
// 128 take 78 us, 6.2 TB/s; 32 of up to 2500, trees of up to 7, 16 heads of dim 64 21.5 us,
// 3.4 TB/s, of which 7 are the way to the first product and the rest what surrounds a tile's
// (with one head to a run 29).  With many rows by that way too and by what a warpgroup does
// itself (products are there when it asks for them): 64 tokens of 32 on 8 heads of dim 128 over
// 32768 places 28.5 us, of which 4.6 to the first product, then 7 units of some 6450 cycles:
// twice 2030 for the 128 columns of a set, 630 between the sets and 1760 from unit to unit.  For
// each set the two warpgroups share 1024 cycles of the exponential unit, and shared memory
// serves 2400: 1100 of reads of the terms, 1024 of the products' operands, 256 of the tiles' way in.
struct WeightsParams {
  CUtensorMap tm_q;  // [total, Hkv, G, d]: box 64 columns x G heads x TB tokens
  CUtensorMap tm_k;  // [num_pages, page_size, Hkv, d]: box 64 columns x min(page_size, 128) rows of one head
  const int *cu;
  const unsigned long long *mask;  // [total, words] or nullptr: a chain
  const float *lse;                // [H, total]
  float *weights;                  // [B, Hkv, places]
  unsigned *status;
  PageGeom g;
  int words, max_new, total, Hkv, G, places;
  int TB, HB, RH;  // tokens of a chunk, kv heads whose rows are in shared memory together, rows from one to the next
  bool by_warp;    // few sequences, whose cost fits 31 bits
  bool stream;     // more chunks than shared memory holds: one after another for each unit, else an item's rows stay
  float scale_log2, decay;
};

// NQ: rows in shared memory.
template <int D, int NQ>
struct WeightsCfg {
  static constexpr int kBoxes = D / 64;
  static constexpr int kTileBytes = 128 * D * 2, kBoxBytes = 128 * 128;  // a tile of K, its 64-column box
  static constexpr int kQBytes = NQ * D * 2, kQBoxBytes = NQ * 128;
  static constexpr int kQBufs = NQ == 32 ? 2 : 65536 / kQBytes, kTermBufs = 8;  // sets of rows in shared memory; of their terms
  static constexpr int kWarps = 8, kMmaWarp = 8, kKeyWarp = 9, kThreads = 32 * 11;
  static constexpr int kTermBytes = kTermBufs * (3 * NQ + 4) * 4;
  static constexpr int kSmemMax = 227 * 1024;
  static constexpr int kStagesFit = (kSmemMax - 1024 - 1024 - kQBufs * kQBytes - kTermBytes) / kTileBytes;
  static constexpr int kStages = kStagesFit > 8 ? 8 : kStagesFit;
  static_assert(kStages >= 2, "a unit's two tiles");
  // S^T of warpgroup w: two buffers of NQ columns from 2 w NQ on
  static constexpr int kTmemCols = 4 * NQ;
  static_assert(NQ >= 32 && NQ % 32 == 0 && kTmemCols <= 512, "TMEM budget");
  static constexpr int kOffQ = 0, kOffRing = kQBufs * kQBytes, kOffTerms = kOffRing + kStages * kTileBytes;
  static constexpr int kOffBar = kOffTerms + kTermBytes;
  // barriers: full[S], empty[S], q_full[QB], q_free[QB], t_full[TB], t_free[TB], s_full[4], s_free[4], drain
  static constexpr int kNumBars = 2 * kStages + 2 * kQBufs + 2 * kTermBufs + 9;
  static constexpr int kOffMisc = kOffBar + 8 * kNumBars;
  static constexpr int kSmemBytes = kOffMisc + 320 + 1024;
  static_assert(kSmemBytes <= kSmemMax, "shared memory budget");
};

FA_STALL_FLAG_DECL

enum WeightsSite : int {
  kWSiteKeys = 43, kWSiteRows = 44, kWSiteTerms = 45, kWSiteEmpty = 46, kWSiteSFree = 47, kWSiteSFull = 48,
  kWSiteRowsFree = 49, kWSiteTermsFree = 50, kWSiteDrain = 51
};

// A block's units; every warp walks its own copy.
struct WeightsWalk {
  long long base, end;  // cost before the sequence, and where the block's stretch ends
  PagedSeq s;
  int b, u, units, chunks, pairs;  // the sequence's next unit, its units, their cost, pairs of tiles
  // the current run: units of neighbouring heads [hb, hb1) on the same places
  int group, pair, hb, hb1;
  bool first, entered;  // first: of its item in this block

  __device__ static PagedSeq seq(const WeightsParams &p, int b) {
    return paged_seq_of(p.cu[b], p.cu[b + 1], p.g.cache_lens[b], p.total, p.max_new, p.g.max_pages * p.g.page_size);
  }
  __device__ static int units_of(const WeightsParams &p, const PagedSeq &s) {  // fits 31 bits (checked by the host)
    return s.n == 0 ? 0 : ((s.keys + 255) >> 8) * p.Hkv;
  }
  __device__ static int chunks_of(const WeightsParams &p, const PagedSeq &s) { return s.n <= p.TB ? 1 : (s.n + p.TB - 1) / p.TB; }
  __device__ void enter(const WeightsParams &p, int u0) {  // the next unit is u0
    units = units_of(p, s);
    chunks = chunks_of(p, s);
    pairs = max((s.keys + 255) >> 8, 1);
    u = u0;
    group = pair = 0;
    hb1 = u0;  // where the next run begins
    if (u0 > 0) {
      group = u0 / (pairs * p.HB);
      hb1 = u0 - group * pairs * p.HB;
      pair = hb1 / p.HB;
      hb1 -= pair * p.HB;
    }
    entered = true;
  }
  __device__ bool next(const WeightsParams &p) {
    if (b >= p.g.B) return false;
    while (u >= units) {
      base += (long long)units * chunks;
      if (++b >= p.g.B || base >= end) {
        b = p.g.B;
        return false;
      }
      s = seq(p, b);
      enter(p, 0);
    }
    if (base + (long long)u * chunks >= end) return false;
    first = entered;
    entered = false;
    if (hb1 == p.HB) {
      hb1 = 0;
      if (++pair == pairs) {
        pair = 0;
        ++group;
        first = true;
      }
    }
    hb = hb1;
    do {  // as far as the block's stretch goes
      ++hb1;
      ++u;
    } while (hb1 < p.HB && base + (long long)u * chunks < end);
    return true;
  }
};

// a / b rounded up, a >= 0, b > 0, in 32 bits where both fit (nearly always).
__device__ __forceinline__ long long quot_up(long long a, long long b) {
  const long long c = a + b - 1;
  return ((c | b) >> 32) == 0 ? (long long)((unsigned)c / (unsigned)b) : c / b;
}

// The cost of all units and where this block begins, by the whole block together.
template <int THREADS>
__device__ __forceinline__ void weights_start(const WeightsParams &p, long long *sums, WeightsWalk *at) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  PagedSeq s;
  auto cost = [&](int b) -> long long {
    if (b >= p.g.B) return 0;
    s = WeightsWalk::seq(p, b);
    return (long long)WeightsWalk::units_of(p, s) * WeightsWalk::chunks_of(p, s);
  };
  auto scan = [&](long long x, long long &total) -> long long {  // exclusive
    long long sum = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = sum;
    __syncthreads();
    long long before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      const long long y = sums[w];
      if (w < warp) before += y;
      total += y;
    }
    return before + sum - x;
  };
  long long total = 0, done = 0;
  for (int b0 = 0; b0 < p.g.B; b0 += THREADS) {
    long long sum;
    scan(cost(b0 + (int)threadIdx.x), sum);
    total += sum;
  }
  const long long per = quot_up(total, gridDim.x), begin = min(per * blockIdx.x, total);
  for (int b0 = 0; b0 < p.g.B && done <= begin; b0 += THREADS) {
    const int b = b0 + (int)threadIdx.x;
    long long sum;
    const long long x = cost(b), before = done + scan(x, sum);
    if (b < p.g.B && begin >= before && begin < before + x) {
      at->s = s;
      at->b = b;
      at->base = before;
      at->end = min(begin + per, total);
      at->enter(p, (int)quot_up(begin - before, WeightsWalk::chunks_of(p, s)));
    }
    done += sum;
  }
}

// The same of up to 128 sequences whose cost surely fits 31 bits (p.by_warp), by every warp for
// itself: no barrier.  A call's first product is some 5 us after its launch, most of it these
// loads, the page table's, the first tiles' and the instructions' own way in: so little code.
constexpr int kByWarp = 128;
__device__ __forceinline__ WeightsWalk weights_start_by_warp(const WeightsParams &p) {
  const int lane = threadIdx.x & 31;
  PagedSeq s = {0, 0, 0, 0};
  auto cost = [&](int b) -> unsigned {
    if (b >= p.g.B) return 0u;
    s = WeightsWalk::seq(p, b);
    return (unsigned)(WeightsWalk::units_of(p, s) * WeightsWalk::chunks_of(p, s));
  };
  unsigned total = 0, done = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < p.g.B; b0 += 32) total += __reduce_add_sync(0xffffffffu, cost(b0 + lane));
  const unsigned per = (total + gridDim.x - 1) / gridDim.x, begin = min(per * blockIdx.x, total);
  WeightsWalk w;
  w.b = p.g.B;
  w.base = w.end = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < p.g.B; b0 += 32) {
    const unsigned x = cost(b0 + lane);
    unsigned after = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned y = __shfl_up_sync(0xffffffffu, after, o);
      if (lane >= o) after += y;
    }
    const unsigned before = done + after - x;
    const unsigned here = __ballot_sync(0xffffffffu, begin >= before && begin - before < x);
    if (here) {
      const int from = __ffs(here) - 1;
      w.b = b0 + from;
      const unsigned base = __shfl_sync(0xffffffffu, before, from);
      w.base = base;
      w.end = min(begin + per, total);
      w.s.start = __shfl_sync(0xffffffffu, s.start, from);
      w.s.n = __shfl_sync(0xffffffffu, s.n, from);
      w.s.len = __shfl_sync(0xffffffffu, s.len, from);
      w.s.keys = __shfl_sync(0xffffffffu, s.keys, from);
      const int chunks = WeightsWalk::chunks_of(p, w.s);
      w.enter(p, chunks == 1 ? (int)(begin - base) : (int)((begin - base + chunks - 1) / chunks));
      break;
    }
    done += __shfl_sync(0xffffffffu, after, 31);
  }
  return w;
}

// Bits [lo, hi) of a 32-bit word (both may lie outside it).
__device__ __forceinline__ unsigned bit_range(int lo, int hi) {
  lo = max(lo, 0);
  hi = min(hi, 32);
  if (lo >= hi) return 0;
  return (0xffffffffu >> (32 - (hi - lo))) << lo;
}

// Rounding.  Scores are fp32 sums.  A row's lse in log2 units is kept as a float and its
// rounding error, which as a factor 2^-error goes into the sum: as the argument's error it
// would be the same for all places of a row (up to 2^-20 of each weight).  Sums are fp32.
// Rows of a set share a base only where their lse lie within 8 (in log2 units) of one another:
// an argument c2 s - base is rounded to half a step of its size, so that a base b away from a
// row's own lse costs a weight near 1 up to b 2^-24 of it, 2^-22 with the 4 allowed here (with
// the largest lse as the base and up to 64 between them it was 2.8e-6).  Row by row the window
// above takes 38.4 us.  A weight below 2^-122 of its row's sum may become 0.
template <int D, int NQ>
__global__ void __launch_bounds__(WeightsCfg<D, NQ>::kThreads, 1) weights_kernel(const __grid_constant__ WeightsParams p) {
  using C = WeightsCfg<D, NQ>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::kOffBar;
  auto full_bar = [&](int i) { return bar0 + 8u * i; };
  auto empty_bar = [&](int i) { return bar0 + 8u * (C::kStages + i); };
  const uint32_t bar1 = bar0 + 8u * (2 * C::kStages);
  auto q_full = [&](int i) { return bar1 + 8u * i; };
  auto q_free = [&](int i) { return bar1 + 8u * (C::kQBufs + i); };
  const uint32_t bar2 = bar1 + 8u * (2 * C::kQBufs);
  auto t_full = [&](int i) { return bar2 + 8u * i; };
  auto t_free = [&](int i) { return bar2 + 8u * (C::kTermBufs + i); };
  const uint32_t bar3 = bar2 + 8u * (2 * C::kTermBufs);
  auto s_full = [&](int w, int buf) { return bar3 + 8u * (2 * w + buf); };
  auto s_free = [&](int w, int buf) { return bar3 + 8u * (4 + 2 * w + buf); };
  const uint32_t drain_bar = bar3 + 8u * 8;
  uint8_t *misc = smem + C::kOffMisc;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(misc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(misc + 4);
  WeightsWalk *at = reinterpret_cast<WeightsWalk *>(misc + 8);
  long long *sums = reinterpret_cast<long long *>(misc + 104);  // [kThreads / 32]
  static_assert(sizeof(WeightsWalk) <= 96, "");
  constexpr int kTerms = 3 * NQ + 4;  // of a set of rows: -lse2, its factor, the weight at their base; the base
  float *terms = reinterpret_cast<float *>(smem + C::kOffTerms);
  const WaitCtx wctx{abort_flag, p.status};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  static_assert(C::kNumBars <= 32 * C::kWarps, "a thread to a barrier");
  if (threadIdx.x < C::kNumBars) {
    const uint32_t bar = bar0 + 8u * threadIdx.x;
    const bool all = bar >= t_free(0) && bar < bar3, half = bar >= s_free(0, 0) && bar < drain_bar;
    mbar_init(bar, all ? C::kWarps : half ? 4 : 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    at->b = p.g.B;
    at->base = at->end = 0;
  }
  if (warp == C::kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  if (warp == C::kKeyWarp && lane == 0) {
    prefetch_tmap(&p.tm_q);
    prefetch_tmap(&p.tm_k);
  }
  // The last warp's rows (it needs them early): kv head of the item, token, query head.
  int row_hb[NQ / 32], row_tok[NQ / 32], row_head[NQ / 32];  // of this lane's rows
#pragma unroll
  for (int i = 0; i < NQ / 32; ++i) {
    const int x = lane + 32 * i, hb = x / p.RH, y = x - hb * p.RH;
    row_tok[i] = y / p.G;
    row_hb[i] = hb < p.HB && row_tok[i] < p.TB ? hb : -1;
    row_head[i] = hb * p.G + y - row_tok[i] * p.G;
  }
  tc_fence_before();
  __syncthreads();
  grid_go();  // only now: a kernel that begins early takes no tensor memory before this one has
  grid_wait();
  tc_fence_after();
  WeightsWalk walk;
  if (p.by_warp) {
    walk = weights_start_by_warp(p);
  } else {
    weights_start<C::kThreads>(p, sums, at);
    __syncthreads();
    walk = *at;
  }
  const uint32_t tmem = *tmem_slot;
  bool ok = true;

  if (warp < C::kWarps) {
    // ===================================================== two warpgroups, a thread to a place
    const int w = warp >> 2, r = threadIdx.x & 127;
    const uint32_t s_tm = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)(2 * w * NQ);
    const float c2 = p.scale_log2;
    const int shift = 31 - __clz(p.g.page_size);
    int tile_no = 0;  // products of this warpgroup so far
    // A set of rows is a step: of an item's chunk, or (p.stream) of a unit's.  Steps looked up, waited for, given back.
    int steps = 0, entered = 0, left = 0;
    // A run's place of this thread; its page and the first head's old sum are on their way while the run before is
    // worked on.
    struct Run {
      float *to;  // the first head's sum
      int pos, keys, len, n, start, chunks, hb, hb1, page, step;
      float old;
    };
    auto look_up = [&](Run &u) {
      if (!walk.next(p)) return false;
      u.keys = walk.s.keys;
      u.len = walk.s.len;
      u.n = walk.s.n;
      u.start = walk.s.start;
      u.chunks = walk.chunks;
      u.hb = walk.hb;
      u.hb1 = walk.hb1;
      if (p.stream || walk.first) steps += walk.chunks;
      u.step = steps - walk.chunks;
      u.pos = (2 * walk.pair + w) * 128 + r;
      u.to = p.weights + ((size_t)walk.b * p.Hkv + walk.group * p.HB + walk.hb) * p.places + u.pos;
      u.page = -1;
      u.old = 0.f;
      if (u.pos < min(u.keys, p.places)) {
        u.page = p.g.page_table[(size_t)walk.b * p.g.max_pages + (u.pos >> shift)];
        if (p.decay != 0.f) u.old = *u.to;
      }
      return true;
    };
    auto enter = [&](int step) {
      while (ok && entered <= step) {
        ok = mbar_wait_warp(t_full(entered % C::kTermBufs), (entered / C::kTermBufs) & 1, wctx, kWSiteTerms);
        ++entered;
      }
    };
    auto leave = [&](int step) {  // all before it (entered, as every unit goes through all its chunks)
      for (; left < step; ++left) mbar_arrive_warp(t_free(left % C::kTermBufs));
    };
    Run u;
    bool more = look_up(u);
    while (ok && more) {
      Run following;
      more = look_up(following);
      const int kv0 = u.pos - r;
      const bool mine = kv0 < u.keys;
      const bool out = u.pos < min(u.keys, p.places), held = u.page >= 0 && u.page < p.g.num_pages;
      const int j = u.pos - u.len;  // this place among the new tokens
      // every row sees all of the warp's places (what a thread without a place sums up is lost)
      const bool whole = __all_sync(0xffffffffu, !out || (held && j < 0));
      // the rows of a chunk that see this place (with several heads in a run there is one chunk)
      unsigned see[NQ / 32];
      auto look = [&](int tok0, int tokens) {
        const int rows = tokens * p.G;
#pragma unroll
        for (int i = 0; i < NQ / 32; ++i) see[i] = held ? bit_range((max(j - tok0, 0)) * p.G - 32 * i, rows - 32 * i) : 0u;
        if (held && j >= 0 && p.mask) {
#pragma unroll
          for (int i = 0; i < NQ / 32; ++i) see[i] = 0;
          const unsigned long long *word = p.mask + (size_t)(u.start + tok0) * p.words + (j >> 6);
          for (int k = 0; k < tokens; ++k, word += p.words)
            if ((*word >> (j & 63)) & 1) {
#pragma unroll
              for (int i = 0; i < NQ / 32; ++i) see[i] |= bit_range(k * p.G - 32 * i, (k + 1) * p.G - 32 * i);
            }
        }
      };
      float *to = u.to;
      float old = u.old;
      for (int h = u.hb; h < u.hb1 && ok; ++h, to += p.places) {
        const float old_next = h + 1 < u.hb1 && out && p.decay != 0.f ? to[p.places] : 0.f;
        float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
        for (int c = 0; c < u.chunks && ok; ++c) {
          const int tok0 = c * p.TB, tokens = min(p.TB, u.n - tok0), rows = tokens * p.G;
          if (!whole && h == u.hb) look(tok0, tokens);
          leave(u.step + (p.stream ? c : 0));
          enter(u.step + c);
          if (!ok) break;
          if (mine) {
            const float *set = terms + ((u.step + c) % C::kTermBufs) * kTerms;
            const float4 *neg = reinterpret_cast<const float4 *>(set + h * p.RH), *fac = neg + NQ / 4, *at_base = fac + NQ / 4;
            const float base = set[3 * NQ];  // not finite where the rows have none
            const int buf = tile_no & 1;
            ok = mbar_wait_warp(s_full(w, buf), (tile_no >> 1) & 1, wctx, kWSiteSFull);
            if (!ok) break;
            tc_fence_after();
            const uint32_t from = s_tm + (uint32_t)(buf * NQ);
            // four columns from 4 q on, whose rows all see this place: 2^(c2 s - base) 2^(base - lse2)
            auto add4 = [&](const uint32_t *s, int q) {
              const float4 f = at_base[q];
              float x[4];
              ffma2(x[0], x[1], __uint_as_float(s[0]), __uint_as_float(s[1]), c2, c2, -base, -base);
              ffma2(x[2], x[3], __uint_as_float(s[2]), __uint_as_float(s[3]), c2, c2, -base, -base);
#pragma unroll
              for (int k = 0; k < 4; ++k) x[k] = ex2_mufu(x[k]);
              ffma2(a0, a1, x[0], x[1], f.x, f.y, a0, a1);
              ffma2(a2, a3, x[2], x[3], f.z, f.w, a2, a3);
            };
            // those of them whose bits are set (rows past the last hold anything, and so do their factors)
            auto add4_seen = [&](const uint32_t *s, int q, unsigned bits) {
              const float4 n = neg[q], f = fac[q];
              const float m[4] = {n.x, n.y, n.z, n.w}, g[4] = {f.x, f.y, f.z, f.w};
              float x[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                x[k] = ex2_mufu(fmaf(__uint_as_float(s[k]), c2, m[k])) * g[k];
                x[k] = (bits >> k) & 1 ? x[k] : 0.f;
              }
              fadd2(a0, a1, a0, a1, x[0], x[1]);
              fadd2(a2, a3, a2, a3, x[2], x[3]);
            };
            auto read = [&] {  // the product is in registers
              tc_fence_before();
              if (!(FA_STALL(6) && tile_no == 0 && w == 0)) mbar_arrive_warp(s_free(w, buf));
            };
            if (NQ == 32 && rows <= 16) {  // a decoding step
              uint32_t s[16];
              tmem_ld_32x32b_x16(from, s);
              tmem_wait_ld(s);
              read();
#pragma unroll
              for (int q = 0; q < 4; ++q)
                if (4 * q < rows) add4_seen(s + 4 * q, q, (whole ? bit_range(0, rows) : see[0]) >> (4 * q));
            } else {
              const bool based = NQ > 32 && fabsf(base) < INFINITY;
#pragma unroll
              for (int i = 0; i < NQ / 32; ++i) {
                if (32 * i >= rows) break;
                uint32_t s[32];
                tmem_ld_32x32b_x32(from + (uint32_t)(32 * i), s);
                tmem_wait_ld(s);
                if (32 * i + 32 >= rows) read();
                // 32 rows that see all of the warp's places, or none
                const unsigned bits = whole ? bit_range(0, rows - 32 * i) : see[i];
                if (based && __all_sync(0xffffffffu, !out || bits == 0xffffffffu)) {
#pragma unroll
                  for (int q = 0; q < 8; ++q) add4(s + 4 * q, 8 * i + q);
                } else if (__any_sync(0xffffffffu, out && bits != 0u)) {
#pragma unroll
                  for (int q = 0; q < 8; ++q) add4_seen(s + 4 * q, 8 * i + q, bits >> (4 * q));
                }
              }
            }
            ++tile_no;
          }
        }
        const float sum = (a0 + a1) + (a2 + a3);
        if (ok && out) *to = p.decay == 0.f ? sum : fmaf(old, p.decay, sum);
        old = old_next;
      }
      u = following;
    }
  } else if (warp == C::kMmaWarp) {
    // ===================================================== MMA issue (whole warp; the elected lane issues)
    int fill = 0, step = 0, base = 0, tile_no[2] = {0, 0};  // step: sets of rows entered, base: the first one of the item or unit
    const uint64_t k_desc = make_sdesc_sw128(sbase + C::kOffRing, 0, 1024);
    const uint64_t q_desc = make_sdesc_sw128(sbase + C::kOffQ, 0, 1024);
    bool any = false;
    while (ok && walk.next(p)) {
      const int nt = (2 * walk.pair + 1) * 128 < walk.s.keys ? 2 : 1;
      if (p.stream || walk.first) {
        if (!p.stream) {
          if (elect_one())
            for (int i = base; i < step; ++i) tc_commit(q_free(i % C::kQBufs));
          __syncwarp();
        }
        base = step;
      }
      for (int h = walk.hb; h < walk.hb1 && ok; ++h) {
        for (int t = 0; t < nt && ok; ++t)
          ok = mbar_wait_warp(full_bar((fill + t) % C::kStages), ((fill + t) / C::kStages) & 1, wctx, kWSiteKeys);
        for (int c = 0; c < walk.chunks && ok; ++c) {
          const int qb = (base + c) % C::kQBufs;
          if (base + c == step) {
            ok = mbar_wait_warp(q_full(qb), (step / C::kQBufs) & 1, wctx, kWSiteRows);
            if (!ok) break;
            ++step;
          }
          tc_fence_after();
          const int rows = min(p.TB, walk.s.n - c * p.TB) * p.G;
          const uint32_t idesc = make_idesc_bf16(128, (rows + 15) & ~15, false, false);
          const uint64_t qd = q_desc + (uint64_t)((qb * C::kQBytes + h * p.RH * 128) >> 4);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (t >= nt || !ok) continue;
            const int buf = tile_no[t] & 1;
            ok = mbar_wait_warp(s_free(t, buf), ((tile_no[t] >> 1) & 1) ^ 1, wctx, kWSiteSFree);
            if (!ok) break;
            tc_fence_after();
            const uint64_t kd = k_desc + (uint64_t)((((fill + t) % C::kStages) * C::kTileBytes) >> 4);
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                mma_ss(tmem + (uint32_t)((2 * t + buf) * NQ), kd + (uint32_t)(((kk >> 2) * C::kBoxBytes + (kk & 3) * 32) >> 4),
                       qd + (uint32_t)(((kk >> 2) * C::kQBoxBytes + (kk & 3) * 32) >> 4), idesc, kk > 0);
              tc_commit(s_full(t, buf));
            }
            __syncwarp();
            any = true;
            ++tile_no[t];
          }
          if (p.stream && ok) {
            if (elect_one()) tc_commit(q_free(qb));
            __syncwarp();
          }
        }
        if (!ok) break;
        if (elect_one())
          for (int t = 0; t < nt; ++t) tc_commit(empty_bar((fill + t) % C::kStages));
        __syncwarp();
        fill += nt;
      }
    }
    // Drain: every MMA this warp issued completes before TMEM is released.
    if (any) {
      if (elect_one()) tc_commit(drain_bar);
      __syncwarp();
      if (!mbar_wait_warp(drain_bar, 0, wctx, kWSiteDrain) && *abort_flag) {
        const uint64_t t0 = global_timer_ns();
        while (!mbar_test(drain_bar, 0) && global_timer_ns() - t0 < kWaitLimitNs) {}
      }
    }
  } else if (warp == C::kKeyWarp) {
    // ===================================================== K tiles (one lane per page of a tile)
    const uint64_t once = policy_evict_first();
    const int box_rows = min(p.g.page_size, 128), boxes = 128 / box_rows;
    const int shift = 31 - __clz(p.g.page_size);
    int fill = 0;
    while (ok && walk.next(p)) {
      const int *row = p.g.page_table + (size_t)walk.b * p.g.max_pages;
      int pages[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int pos = (2 * walk.pair + t) * 128 + lane * box_rows;
        pages[t] = lane < boxes && pos < walk.s.keys ? row[pos >> shift] : -1;
        if (pages[t] < 0 || pages[t] >= p.g.num_pages) pages[t] = -1;  // zeros
      }
      for (int h = walk.hb; h < walk.hb1 && ok; ++h) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int kv0 = (2 * walk.pair + t) * 128, pos = kv0 + lane * box_rows;
          if (kv0 >= walk.s.keys || !ok) break;
          const int slot = fill % C::kStages;
          ok = mbar_wait_warp(empty_bar(slot), ((fill / C::kStages) & 1) ^ 1, wctx, kWSiteEmpty);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(full_bar(slot), C::kTileBytes);
          __syncwarp();
          if (lane < boxes) {
            const int r0 = pos & (p.g.page_size - 1);
#pragma unroll
            for (int bx = 0; bx < C::kBoxes; ++bx)
              tma_load_4d_hint(sbase + C::kOffRing + slot * C::kTileBytes + bx * C::kBoxBytes + lane * box_rows * 128, &p.tm_k,
                               full_bar(slot), bx * 64, walk.group * p.HB + h, r0, pages[t], once);
          }
          // The old sums come with the tile: in a stream of tiles that fills the memory's queues a load takes
          // longer than a unit.
          if (p.decay != 0.f && lane < 4 && kv0 + 32 * lane < min(walk.s.keys, p.places))
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p.weights + ((size_t)walk.b * p.Hkv + walk.group * p.HB + h) * p.places +
                                                         kv0 + 32 * lane));
          ++fill;
        }
      }
    }
    // Every copy issued lands before the block exits (normally they already have).
    const uint64_t t0 = global_timer_ns();
    for (int f = max(0, fill - C::kStages); f < fill; ++f)
      while (!mbar_test(full_bar(f % C::kStages), (f / C::kStages) & 1) && global_timer_ns() - t0 < kWaitLimitNs) {}
  } else {
    // ===================================================== the tokens' rows and what their lse puts into the sums
    int step = 0;
    float lse[NQ / 32];  // of the next chunk: on their way during the waits of the one before
    auto look_up = [&](int c) {
      const int tok0 = c * p.TB, tokens = min(p.TB, walk.s.n - tok0);
#pragma unroll
      for (int i = 0; i < NQ / 32; ++i) {
        lse[i] = 0.f;
        if (row_hb[i] >= 0 && row_tok[i] < tokens)
          lse[i] = p.lse[(size_t)(walk.group * p.HB * p.G + row_head[i]) * p.total + walk.s.start + tok0 + row_tok[i]];
      }
    };
    while (ok && walk.next(p)) {
      if (!(p.stream || walk.first)) continue;
      look_up(0);
      for (int c = 0; c < walk.chunks && ok; ++c) {
        const int qb = step % C::kQBufs, tb = step % C::kTermBufs;
        const int tokens = min(p.TB, walk.s.n - c * p.TB);
        ok = mbar_wait_warp(q_free(qb), ((step / C::kQBufs) & 1) ^ 1, wctx, kWSiteRowsFree);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(q_full(qb), p.HB * C::kBoxes * p.TB * p.G * 128);
          for (int hb = 0; hb < p.HB; ++hb)
            for (int bx = 0; bx < C::kBoxes; ++bx)
              tma_load_4d(sbase + C::kOffQ + qb * C::kQBytes + bx * C::kQBoxBytes + hb * p.RH * 128, &p.tm_q, q_full(qb), bx * 64, 0,
                          walk.group * p.HB + hb, walk.s.start + c * p.TB);
        }
        ++step;
        __syncwarp();
        ok = mbar_wait_warp(t_free(tb), (((step - 1) / C::kTermBufs) & 1) ^ 1, wctx, kWSiteTermsFree);
        if (!ok) break;
        float *t = terms + tb * kTerms;
        float here[NQ / 32];
#pragma unroll
        for (int i = 0; i < NQ / 32; ++i) here[i] = lse[i];
        if (c + 1 < walk.chunks) look_up(c + 1);
        float hi[NQ / 32], lo[NQ / 32], top = -INFINITY, low = INFINITY;
        bool finite = true;  // the lse of all rows
#pragma unroll
        for (int i = 0; i < NQ / 32; ++i) {
          constexpr float kLog2e = 1.44269502162933349609375f, kLog2eLow = 1.925963033500920e-8f;  // log2(e) is their sum
          hi[i] = here[i] * kLog2e;
          lo[i] = fmaf(here[i], kLog2e, -hi[i]) + here[i] * kLog2eLow;
          if (!(fabsf(hi[i]) < INFINITY)) lo[i] = 0.f;
          // a token that saw nothing has lse = -inf and gives nothing
          t[lane + 32 * i] = here[i] == -INFINITY ? -INFINITY : -hi[i];
          t[NQ + lane + 32 * i] = fmaf(lo[i], -0.693147180559945309f, 1.f);
          if (NQ > 32 && row_hb[i] >= 0 && row_tok[i] < tokens) {
            finite &= fabsf(hi[i]) < INFINITY;
            top = fmaxf(top, hi[i]);
            low = fminf(low, hi[i]);
          }
        }
        if (NQ > 32) {  // with few rows the base is not used
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
          }
          // One base for all, at most 4 from each: the largest, or 4 above the smallest.  A row that its lse leaves out
          // may have any score: beside the others' base 2^score may be infinite, which times a factor of 0 is not 0, so
          // such a set goes row by row.
          const float base = __all_sync(0xffffffffu, finite) && top - low <= 8.f ? fminf(top, low + 4.f) : INFINITY;
#pragma unroll
          for (int i = 0; i < NQ / 32; ++i) {
            const float d = base - hi[i], back = base - d, rest = (base - (d + back)) + (back - hi[i]);  // base - hi = d + rest
            t[2 * NQ + lane + 32 * i] = exp2f(d) * fmaf(rest - lo[i], 0.693147180559945309f, 1.f);
          }
          if (lane == 0) t[3 * NQ] = base;
        }
        mbar_arrive_warp(t_full(tb));
      }
    }
    const uint64_t t0 = global_timer_ns();
    for (int f = max(0, step - C::kQBufs); f < step; ++f)
      while (!mbar_test(q_full(f % C::kQBufs), (f / C::kQBufs) & 1) && global_timer_ns() - t0 < kWaitLimitNs) {}
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

constexpr int kSMs = 152;

template <int D, int NQ>
int launch_weights(WeightsParams &p, const void *q, const void *k_pages, cudaStream_t stream) {
  using C = WeightsCfg<D, NQ>;
  p.stream = (p.max_new + p.TB - 1) / p.TB > C::kQBufs;
  const uint64_t dims[4] = {(uint64_t)D, (uint64_t)p.G, (uint64_t)p.Hkv, (uint64_t)p.total};
  const uint64_t strides[3] = {(uint64_t)D * 2, (uint64_t)p.G * D * 2, (uint64_t)p.Hkv * p.G * D * 2};
  const uint32_t box[4] = {64, (uint32_t)p.G, 1, (uint32_t)p.TB};
  // head dim 64, one head at a time: its neighbour's 128 bytes are not fetched with it (as in fa_paged.cu)
  if (encode_bf16_box_map(&p.tm_q, q, dims, strides, box) ||
      encode_page_map(&p.tm_k, k_pages, p.g.num_pages, p.g.page_size, p.Hkv, D, p.g.page_size < 128 ? p.g.page_size : 128,
                      D == 64 && p.HB == 1))
    return FA_ERR_CUDA;
  // on every launch: the attribute belongs to the function on the current device
  if (cudaFuncSetAttribute(weights_kernel<D, NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes) != cudaSuccess)
    return FA_ERR_CUDA;
  return launch_after(weights_kernel<D, NQ>, kSMs, 1, C::kThreads, C::kSmemBytes, stream, p);
}

}  // namespace

#ifdef FA_TEST_STALL
int set_test_stall_weights(int mode) {
  return cudaMemcpyToSymbol(g_test_stall, &mode, sizeof(int)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
#endif

}  // namespace fa

using namespace fa;

extern "C" {

int fa_attention_weights_paged(const void *q, const void *k_pages, const int *page_table, const int *cache_lens,
                               const int *cu_seqlens, const long long *tree_mask, int mask_words, const float *lse,
                               float *weights, int places, float decay, int B, int max_pages, int num_pages,
                               int page_size, int max_new, int total, int H, int Hkv, int d, float scale,
                               void *stream) {
  if (!q || !k_pages || !page_table || !cache_lens || !cu_seqlens || !lse || !weights) return FA_ERR_INVALID_ARG;
  int rc = check_paged(B, max_pages, num_pages, page_size, max_new, total, H, Hkv, d);
  if (rc != FA_OK) return rc;
  if (!std::isfinite(scale) || !(scale > 0.f) || !std::isfinite(decay) || decay < 0.f) return FA_ERR_INVALID_ARG;
  if (tree_mask && (long long)mask_words * 64 < max_new) return FA_ERR_INVALID_ARG;
  if (places <= 0) return FA_ERR_INVALID_ARG;
  if ((double)B * Hkv * places >= (double)(1ll << 40)) return FA_ERR_UNSUPPORTED;
  // the units of one sequence are counted in 31 bits
  const double seq_units = ((double)max_pages * page_size / 256 + 1) * Hkv;
  if (seq_units >= 2147483648.0) return FA_ERR_UNSUPPORTED;
  if (!ptr_aligned(q, 16) || !ptr_aligned(k_pages, 16)) return FA_ERR_ALIGNMENT;
  for (const void *x : {(const void *)page_table, (const void *)cache_lens, (const void *)cu_seqlens, (const void *)lse,
                        (const void *)weights})
    if (!ptr_aligned(x, 4)) return FA_ERR_ALIGNMENT;
  if (!ptr_aligned(tree_mask, 8)) return FA_ERR_ALIGNMENT;
  if ((rc = check_device()) != FA_OK) return rc;
  if (total == 0) return FA_OK;
  WeightsParams p = {};
  p.cu = cu_seqlens;
  p.mask = reinterpret_cast<const unsigned long long *>(tree_mask);
  p.lse = lse;
  p.weights = weights;
  p.status = device_status_ptr();
  if (!p.status) return FA_ERR_CUDA;
  p.g = PageGeom{page_table, cache_lens, B, max_pages, num_pages, page_size};
  p.words = mask_words;
  p.max_new = max_new;
  p.total = total;
  p.Hkv = Hkv;
  p.G = H / Hkv;
  p.places = places;
  p.scale_log2 = (float)((double)scale * 1.4426950408889634);
  p.decay = decay;
  // Rows of up to 32 in all (a decoding step, a short chain): a longer ring of K tiles, 16 columns at a time (trees
  // of up to 7 of 16 heads of dim 64 21.4 us instead of 24.5 with room for 128 rows; one token of 64 users the same).
  const bool few = max_new * p.G <= 32;
  const int room = few ? 32 : 128;
  p.TB = room / p.G < max_new ? room / p.G : max_new;
  p.RH = (p.TB * p.G + 7) & ~7;
  p.HB = 1;
  while (max_new == p.TB && p.HB < 4 && Hkv % (2 * p.HB) == 0 && 2 * p.HB * p.RH <= room) p.HB *= 2;
  p.by_warp = B <= kByWarp && B * seq_units * ((max_new + p.TB - 1) / p.TB) < 2147483648.0 - 4 * kSMs;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (few)
    return d == 64 ? launch_weights<64, 32>(p, q, k_pages, s)
                   : d == 128 ? launch_weights<128, 32>(p, q, k_pages, s) : launch_weights<256, 32>(p, q, k_pages, s);
  return d == 64 ? launch_weights<64, 128>(p, q, k_pages, s)
                 : d == 128 ? launch_weights<128, 128>(p, q, k_pages, s) : launch_weights<256, 128>(p, q, k_pages, s);
}

}  // extern "C"
