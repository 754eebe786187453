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
constexpr int kSelThreads = 1024;

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
  unsigned w = warp_sums[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const unsigned before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  return s - x + (warp > 0 ? before : 0u);
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const __grid_constant__ EvictParams p) {
  __shared__ unsigned hist[256], warp_sums[32];
  __shared__ unsigned s_prefix, s_need;
  grid_go();
  grid_wait();
  const int tid = threadIdx.x;
  const int b = (int)(blockIdx.x / p.Hkv) % p.g.B;
  const int len = p.g.cache_lens[b];
  float *w = p.weights + (size_t)blockIdx.x * p.places;
  int *kept = p.kept + (size_t)blockIdx.x * p.keep;
  const bool go = goes(p, b, len);
  if (blockIdx.x < p.Hkv * p.g.B && blockIdx.x % p.Hkv == 0 && tid == 0) p.lens_out[b] = go ? p.keep : len;
  if (!go) {
    for (int i = tid; i < p.keep; i += kSelThreads) kept[i] = i < len ? i : -1;
    return;
  }
  // the rank of the last one that stays, eight bits at a time from the top
  const int older = len - p.recent, stay = p.keep - p.recent;
  unsigned prefix = 0, need = stay;
  for (int shift = 24; shift >= 0 && stay > 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int i = tid; i < older; i += kSelThreads) {
      const unsigned r = rank_of(w[i]);
      if (shift == 24 || r >> (shift + 8) == prefix) atomicAdd(&hist[(r >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      unsigned above = 0;
      int digit = 255;
      while (digit > 0 && above + hist[digit] < need) above += hist[digit--];
      s_prefix = prefix << 8 | digit;
      s_need = need - above;
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
  }
  // in order: all above it, and the first `need` that equal it
  unsigned above = 0, equal = 0;
  for (int i0 = 0; i0 < len; i0 += kSelThreads) {
    const int i = i0 + tid;
    const float x = i < len ? w[i] : 0.f;
    const unsigned r = rank_of(x);
    const bool gt = i < len && (i >= older || (stay > 0 && r > prefix));
    const bool eq = i < older && stay > 0 && r == prefix;
    unsigned sum;
    const unsigned at = scan((gt ? 1u : 0u) | (eq ? 0x10000u : 0u), warp_sums, &sum);
    const unsigned a = above + (at & 0xffffu), e = equal + (at >> 16);
    if (gt || (eq && e < need)) {
      const unsigned to = a + min(e, need);
      kept[to] = i;
      w[to] = x;  // to <= i: read already
    }
    above += sum & 0xffffu;
    equal += sum >> 16;
  }
  __syncthreads();
  for (int i = p.keep + tid; i < len; i += kSelThreads) w[i] = 0.f;
}

// ------------------------------------------------------------------ their rows
// A block moves the k or the v rows of one (layer, sequence, kv head), a stretch of rows at
// a time in ascending order: a stretch is read whole before it is written, and what later
// stretches read lies behind what earlier ones wrote.
constexpr int kMoveThreads = 256, kInFlight = 8;

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictParams p) {
  grid_go();
  grid_wait();
  const unsigned item = blockIdx.x >> 1;
  const int b = (int)(item / p.Hkv) % p.g.B, h = item % p.Hkv, layer = item / p.Hkv / p.g.B;
  if (p.g.cache_lens[b] <= p.keep || p.lens_out[b] != p.keep) return;
  const int *kept = p.kept + (size_t)item * p.keep;
  uint4 *pages = ((blockIdx.x & 1) ? p.v_pages : p.k_pages) + (size_t)layer * p.g.num_pages * p.g.page_size * p.Hkv * p.chunks;
  const int c = threadIdx.x % p.chunks, rows = kMoveThreads / p.chunks;
  for (int i0 = 0; i0 < p.keep; i0 += rows * kInFlight) {
    uint4 x[kInFlight];
    uint4 *to[kInFlight];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      const int i = i0 + u * rows + (int)threadIdx.x / p.chunks;
      to[u] = nullptr;
      if (i >= p.keep) continue;
      const int from = kept[i];
      const int fp = page_of(p.g, b, from), tp = page_of(p.g, b, i);
      if (from == i || fp < 0 || tp < 0) continue;
      x[u] = pages[(((size_t)fp * p.g.page_size + from % p.g.page_size) * p.Hkv + h) * p.chunks + c];
      to[u] = pages + (((size_t)tp * p.g.page_size + i % p.g.page_size) * p.Hkv + h) * p.chunks + c;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kInFlight; ++u)
      if (to[u]) *to[u] = x[u];
  }
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
  if (places <= 0 || keep < 0 || recent < 0 || recent > keep || lens_out == cache_lens) return FA_ERR_INVALID_ARG;
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
  rc = launch_after(evict_select_kernel, (long long)items, 1, kSelThreads, 0, s, p);
  if (rc != FA_OK || keep == 0) return rc;
  return launch_after(evict_move_kernel, 2 * (long long)items, 1, kMoveThreads, 0, s, p);
}

}  // extern "C"
