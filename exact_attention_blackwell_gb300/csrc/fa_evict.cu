// fa_evict.cu — a paged cache cut down to a budget: of each (layer, sequence, kv head)
// the places with the largest sums of attention weight and the most recent ones stay and
// move together, in their order, with their sums.
//
// For a sequence of a > keep places: its last `recent` places stay, and of the a - recent
// before them the keep - recent with the largest sums; equal sums, the lower place first;
// a NaN counts as lower than everything.  One kernel finds the places, the next moves the
// rows: place i of the result was place kept[i], and kept ascends, so kept[i] >= i.
#include <cuda_bf16.h>

#include <climits>

#include "fa_paged.h"
#include "ptx.cuh"

namespace fa {
namespace {

// These kernels begin while the kernel before them may still be writing what they read
// (launch_after), so no pointer here is __restrict__ (see fa_cache.cu).

struct EvictParams {
  uint4 *k_pages, *v_pages;
  float *weights;   // [layers, B, Hkv, places]
  const int *refs;  // [num_pages]
  int *lens_out, *kept;  // [B], [layers, B, Hkv, keep]
  PageGeom g;
  int layers, Hkv, places, keep, recent, chunks;  // chunks: 16-byte pieces of a head's row
};

// Larger sums give larger numbers; -0 is 0, NaN is 0 and all else above it.
__device__ __forceinline__ unsigned rank_of(float x) {
  if (x != x) return 0u;
  const unsigned u = __float_as_uint(x + 0.f);
  return u >> 31 ? ~u : u | 0x80000000u;
}

// ------------------------------------------------------------------ which places stay
// Does the row hold more than the budget, fit the sums, have a page for every place and own
// those that are written?
__device__ __forceinline__ bool goes(const EvictParams &p, int b, int len) {
  bool bad = false;
  const bool longer = len > p.keep && len <= p.places && len <= (long long)p.g.max_pages * p.g.page_size;
  if (longer)
    for (int c = threadIdx.x; c < (len + p.g.page_size - 1) / p.g.page_size; c += blockDim.x) {
      const int page = p.g.page_table[(size_t)b * p.g.max_pages + c];
      if (page < 0 || page >= p.g.num_pages) bad = true;
      else if ((long long)c * p.g.page_size < p.keep && p.refs[page] > 1) bad = true;
    }
  return !__syncthreads_or(bad) && longer;
}

// Exclusive sum over the block (of two 16-bit counts at once); *total gets the whole sum.
template <int THREADS>
__device__ __forceinline__ unsigned scan(unsigned x, unsigned *warp_sums, unsigned *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned s = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  unsigned w = lane < THREADS / 32 ? warp_sums[lane] : 0u;
#pragma unroll
  for (int o = 1; o < THREADS / 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  *total = __shfl_sync(0xffffffffu, w, THREADS / 32 - 1);
  const unsigned before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  return s - x + (warp > 0 ? before : 0u);
}

template <int CS>
__device__ __forceinline__ void cluster_barrier() {
  if (CS == 1) {
    __syncthreads();
  } else {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
}
// A cluster of CS blocks to a row of sums, each with a stretch of it, which it keeps in shared
// memory (up to `cap` of them; longer rows are read again from L2, by one block).  The smallest
// rank that stays is found from the top, 8 bits at a time: a histogram of the ranks that agree
// with what is known so far, and the bin in which the count from above reaches what is needed;
// ranks of a bin that all stay need no more bits.  Every block stores its histogram into all of
// them, so that a round costs one barrier of the cluster and no read of another block's memory
// (reading them cost 1.3 us a round); beside the sums over all blocks it adds up those of the
// blocks before its own, which say where its places will go.  Bound by latency: 8 rows of 32768
// sums take 11 us, of which 2 are the table's and the sums' way in, 1.2 to 1.9 each of four
// rounds, and 1.4 the places' way out.
template <int THREADS, int CS>
__global__ void __launch_bounds__(THREADS) evict_select_kernel(const __grid_constant__ EvictParams p, int cap) {
  constexpr int kBins = 256, kOwn = kBins / 32, kEarly = 8;
  extern __shared__ float keys[];
  __shared__ __align__(16) unsigned hist[kBins], hists[CS == 1 ? 1 : 2][CS == 1 ? 1 : CS][kBins];  // of all blocks
  __shared__ unsigned warp_sums[32];
  __shared__ unsigned s_prefix, s_need, s_count, s_above, s_equal;
  grid_go();
  grid_wait();
  const int tid = threadIdx.x;
  const unsigned item = blockIdx.x / CS;
  const int rank = CS == 1 ? 0 : (int)(blockIdx.x % CS);
  const int b = (int)(item / p.Hkv) % p.g.B;
  const int len = p.g.cache_lens[b];
  float *w = p.weights + (size_t)item * p.places;
  int *kept = p.kept + (size_t)item * p.keep;
  // this block's stretch [lo, hi), x[i - lo]
  const int n = min(max(len, 0), p.places);
  const int part = CS == 1 ? n : ((n + CS - 1) / CS + 3) & ~3;
  const int lo = min(rank * part, n), hi = min(lo + part, n);
  const bool held = hi - lo <= cap;
  float early[kEarly];  // on their way while the table is looked at
#pragma unroll
  for (int e = 0; e < kEarly; ++e) {
    const int i = tid + e * THREADS;
    early[e] = held && i < hi - lo ? w[lo + i] : 0.f;
  }
  // every block of the cluster has begun before another one stores into its shared memory
  if (CS > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const bool go = goes(p, b, len);
  if (CS > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (rank == 0 && item < (unsigned)(p.Hkv * p.g.B) && item % p.Hkv == 0 && tid == 0) p.lens_out[b] = go ? p.keep : len;
  if (!go) {  // the whole cluster; the budget may be any number, and a step past it pass 31 bits
    for (long long i = rank * THREADS + tid; i < p.keep; i += CS * THREADS) kept[i] = i < len ? (int)i : -1;
    return;
  }
  const float *x = w + lo;
  if (held) {
#pragma unroll
    for (int e = 0; e < kEarly; ++e)
      if (const int i = tid + e * THREADS; i < hi - lo) keys[i] = early[e];
#pragma unroll 8
    for (int i = tid + kEarly * THREADS; i < hi - lo; i += THREADS) keys[i] = w[lo + i];
    x = keys;
  }
  const int older = len - p.recent, stay = p.keep - p.recent;
  unsigned prefix = 0, need = stay;
  // what stays before this block's stretch: recent places, and by rank above the last one; equal to it
  unsigned above = (unsigned)max(lo - older, 0), equal = 0;
  int shift = 32, round = 0;
  while (shift > 0 && stay > 0) {
    const int known = shift;
    shift -= 8;
    if (tid < kBins) hist[tid] = 0;
    __syncthreads();  // and x is there
#pragma unroll 4
    for (int i = tid; i < min(hi, older) - lo; i += THREADS) {
      const unsigned r = rank_of(x[i]);
      if (known == 32 || r >> known == prefix) atomicAdd(&hist[(r >> shift) & 255u], 1u);
    }
    if (CS > 1) {
      __syncthreads();
      for (int i = tid; i < CS * kBins / 4; i += THREADS) {  // what these arrays held two rounds ago has been read
        const uint4 v = reinterpret_cast<const uint4 *>(hist)[i % (kBins / 4)];
        const uint32_t to = smem_u32(&hists[round & 1][rank][4 * (i % (kBins / 4))]);
        st_cluster_v4(mapa_shared(to, i / (kBins / 4)), v.x, v.y, v.z, v.w);
      }
    }
    cluster_barrier<CS>();
    if (tid < 32) {
      // eight bins to a lane, the highest first; low word: all blocks, high word: those before this one
      unsigned long long own[kOwn] = {};
#pragma unroll
      for (int o = 0; o < CS; ++o)
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const unsigned *from = CS == 1 ? hist : hists[round & 1][o];
          const uint4 v = *reinterpret_cast<const uint4 *>(from + kBins - kOwn * (tid + 1) + 4 * (1 - g));
          const unsigned bin[4] = {v.w, v.z, v.y, v.x};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            own[4 * g + e] += bin[e];
            if (CS > 1 && o < rank) own[4 * g + e] += (unsigned long long)bin[e] << 32;
          }
        }
      unsigned long long count = 0;
#pragma unroll
      for (int e = 0; e < kOwn; ++e) count += own[e];
      unsigned long long over = count;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, over, o);
        if (tid >= o) over += y;
      }
      over -= count;
      if ((unsigned)over < need && (unsigned)over + (unsigned)count >= need) {
#pragma unroll
        for (int e = 0; e < kOwn; ++e) {
          if ((unsigned)over < need && (unsigned)over + (unsigned)own[e] >= need) {
            s_prefix = prefix << 8 | (kBins - 1 - (kOwn * tid + e));
            s_need = need - (unsigned)over;
            s_count = (unsigned)own[e];
            s_above = (unsigned)(over >> 32);
            s_equal = (unsigned)(own[e] >> 32);
          }
          over += own[e];
        }
      }
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
    above += s_above;
    equal = s_equal;
    ++round;
    if (s_count == need) break;
  }
  if (CS == 1) __syncthreads();
  else if (stay == 0) cluster_barrier<CS>();  // every block holds its stretch, so that sums may be written
  // In order: all above it, and the first `need` that equal it; four places to a thread.
  for (int i0 = lo; i0 < hi; i0 += 4 * THREADS) {
    float y[4];
    unsigned f[4], sum4 = 0;  // 1: stays, 0x10000: equal to the last that stays
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = i0 + 4 * tid + e;
      y[e] = i < hi ? x[i - lo] : 0.f;
      f[e] = i < hi && i >= older ? 1u : 0u;
      if (i < min(hi, older) && stay > 0) {
        const unsigned r = rank_of(y[e]) >> shift;
        f[e] = r > prefix ? 1u : r == prefix ? 0x10000u : 0u;
      }
      sum4 += f[e];
    }
    unsigned sum;
    const unsigned at = scan<THREADS>(sum4, warp_sums, &sum);
    unsigned a = above + (at & 0xffffu), q = equal + (at >> 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (f[e] == 1u || (f[e] && q < need)) {
        const unsigned to = a + min(q, need);
        kept[to] = i0 + 4 * tid + e;
        w[to] = y[e];  // to <= its place: read already
      }
      a += f[e] & 0xffffu;
      q += f[e] >> 16;
    }
    above += sum & 0xffffu;
    equal += sum >> 16;
  }
  __syncthreads();
  for (int i = max(p.keep, lo) + tid; i < hi; i += THREADS) w[i] = 0.f;
}

// ------------------------------------------------------------------ their rows
// A cluster of CS blocks moves the k or the v rows of one (layer, sequence, kv head), a round
// of CS * kRoundPieces 16-byte pieces at a time in ascending order.  A round is read whole
// before any of it is written (a barrier of the cluster), and what later rounds read lies
// behind what earlier ones wrote.  Where the rows are is looked up, a row to a thread, a round
// ahead, while the data is on its way.  Bound by HBM: 4096 streams of 1024 rows of dim 128 take
// 286 us, 6.9 TB/s (every thread looking up its own rows, without a round's lead, 620); 16
// streams of 2048 rows 9 us in clusters of 8, 27 in blocks of their own.
constexpr int kMoveThreads = 256, kInFlight = 8;
constexpr int kMaxRoundRows = kMoveThreads * kInFlight / 8;  // head dim 64

template <int CS>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictParams p) {
  __shared__ long long s_from[3][kMaxRoundRows], s_to[3][kMaxRoundRows];  // in pieces; -1: nothing to move
  grid_go();
  grid_wait();
  const unsigned stream = blockIdx.x / CS, item = stream >> 1;
  const int rank = blockIdx.x % CS;
  const int b = (int)(item / p.Hkv) % p.g.B, h = item % p.Hkv, layer = item / p.Hkv / p.g.B;
  if (p.g.cache_lens[b] <= p.keep || p.lens_out[b] != p.keep) return;  // the whole cluster
  const int *kept = p.kept + (size_t)item * p.keep, *table = p.g.page_table + (size_t)b * p.g.max_pages;
  uint4 *pages = ((stream & 1) ? p.v_pages : p.k_pages) + (size_t)layer * p.g.num_pages * p.g.page_size * p.Hkv * p.chunks;
  const int shift = 31 - __clz(p.g.page_size), mask = p.g.page_size - 1;
  const int step = kMoveThreads / p.chunks, rows = step * kInFlight;  // of a block's round
  const int c = threadIdx.x % p.chunks, row = threadIdx.x / p.chunks;
  const int rounds = (p.keep + CS * rows - 1) / (CS * rows);
  auto look_up = [&](int n) {  // the rows of round n
    const int i = (n * CS + rank) * rows + (int)threadIdx.x;
    if ((int)threadIdx.x >= rows) return;
    long long from = -1, to = -1;
    if (i < p.keep) {
      const int f = kept[i];
      if (f != i) {
        from = ((((long long)table[f >> shift] << shift) + (f & mask)) * p.Hkv + h) * p.chunks;
        to = ((((long long)table[i >> shift] << shift) + (i & mask)) * p.Hkv + h) * p.chunks;
      }
    }
    s_from[n % 3][threadIdx.x] = from;
    s_to[n % 3][threadIdx.x] = to;
  };
  look_up(0);
  __syncthreads();
  for (int n = 0; n < rounds; ++n) {
    uint4 x[kInFlight];
    long long from[kInFlight];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) from[u] = s_from[n % 3][u * step + row];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u)
      if (from[u] >= 0) x[u] = pages[from[u] + c];
    if (n + 1 < rounds) look_up(n + 1);
    cluster_barrier<CS>();
#pragma unroll
    for (int u = 0; u < kInFlight; ++u)
      if (from[u] >= 0) pages[s_to[n % 3][u * step + row] + c] = x[u];
  }
}

// launch_after for clusters of CS blocks.
template <int CS, typename... P, typename... A>
int launch_clusters(void (*kernel)(P...), long long clusters, int threads, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(clusters * CS));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = CS;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = CS > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <int THREADS, int CS>
int launch_select(const EvictParams &p, long long items, int most, cudaStream_t stream) {
  const long long part = ((long long)p.places + CS - 1) / CS + 3;  // a block's stretch
  const int cap = part < most ? (int)part : most;
  if (cap * 4 > 30 * 1024 && cudaFuncSetAttribute(evict_select_kernel<THREADS, CS>,
                                                  cudaFuncAttributeMaxDynamicSharedMemorySize, most * 4) != cudaSuccess)
    return FA_ERR_CUDA;
  return launch_clusters<CS>(evict_select_kernel<THREADS, CS>, items, THREADS, (size_t)cap * 4, stream, p, cap);
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

int fa_cache_evict(const int *page_refs, void *k_pages, void *v_pages, const int *page_table, const int *cache_lens,
                   float *weights, int places, int keep, int recent, int *lens_out, int *kept, int B, int max_pages,
                   int num_pages, int page_size, int layers, int Hkv, int d, void *stream) {
  if (!page_refs || !k_pages || !v_pages || !page_table || !cache_lens || !weights || !lens_out || (keep > 0 && !kept))
    return FA_ERR_INVALID_ARG;
  int rc = check_page_table(B, max_pages, num_pages, page_size);
  if (rc == FA_OK) rc = check_page_rows(layers, num_pages, page_size, Hkv, d);
  if (rc != FA_OK) return rc;
  if (places <= 0 || keep < 0 || recent < 0 || recent > keep || lens_out == cache_lens || k_pages == v_pages)
    return FA_ERR_INVALID_ARG;
  const double items = (double)layers * B * Hkv;
  if (items > 1073741823.0 || items * places >= (double)(1ll << 40) || items * keep >= (double)(1ll << 40))
    return FA_ERR_UNSUPPORTED;
  if (!ptr_aligned(k_pages, 16) || !ptr_aligned(v_pages, 16)) return FA_ERR_ALIGNMENT;
  for (const void *x : {(const void *)page_refs, (const void *)page_table, (const void *)cache_lens, (const void *)weights,
                        (const void *)lens_out, (const void *)kept})
    if (!ptr_aligned(x, 4)) return FA_ERR_ALIGNMENT;
  if ((rc = check_device()) != FA_OK) return rc;
  EvictParams p = {};
  p.k_pages = static_cast<uint4 *>(k_pages);
  p.v_pages = static_cast<uint4 *>(v_pages);
  p.weights = weights;
  p.refs = page_refs;
  p.lens_out = lens_out;
  p.kept = kept;
  p.g = PageGeom{page_table, cache_lens, B, max_pages, num_pages, page_size};
  p.layers = layers;
  p.Hkv = Hkv;
  p.places = places;
  p.keep = keep;
  p.recent = recent;
  p.chunks = d / 8;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const long long rows = (long long)items;
  // Short rows, many of them: small blocks, several to an SM (2048 rows of 1100 sums with their moves 323 us, with
  // large blocks 362).  Few long rows: clusters, one block to an SM.  8 rows of 8192, 32768, 100000 sums with their
  // moves in clusters of 8: 13.9, 17.8, 34 us (of 4: 19.9 for 32768), one block to a row: 14.9, 36, 143; 32 rows of
  // 32768 in clusters of 4: 34.5, one block to a row: 48.5.
  constexpr int kMost = 48 * 1024;
  if (places <= 8192 && rows > 152) rc = launch_select<256, 1>(p, rows, 8192, s);
  else if (places >= 4096 && rows * 8 <= 152 && places <= 8 * kMost) rc = launch_select<1024, 8>(p, rows, kMost, s);
  else if (places >= 4096 && rows * 4 <= 152 && places <= 4 * kMost) rc = launch_select<1024, 4>(p, rows, kMost, s);
  else rc = launch_select<1024, 1>(p, rows, kMost, s);
  if (rc != FA_OK || keep == 0) return rc;
  // few streams of rows: clusters, as long as one wave holds them and there are rows for all their blocks
  const long long streams = 2 * rows, round = kMoveThreads * kInFlight / p.chunks, full = (keep + round - 1) / round;
  auto fits = [&](int cs) { return streams * cs <= 2 * 152 && full >= cs; };
  if (fits(8)) return launch_clusters<8>(evict_move_kernel<8>, streams, kMoveThreads, 0, s, p);
  if (fits(4)) return launch_clusters<4>(evict_move_kernel<4>, streams, kMoveThreads, 0, s, p);
  if (fits(2)) return launch_clusters<2>(evict_move_kernel<2>, streams, kMoveThreads, 0, s, p);
  return launch_clusters<1>(evict_move_kernel<1>, streams, kMoveThreads, 0, s, p);
}

}  // extern "C"
