// fa_cache.cu — operators of a paged key/value cache: writing new rows into the
// pages, moving an accepted path together, sharing rows of the page table by
// counting, taking pages and giving them back.
//
// All state lives on the device (page table, lengths, one count per page), so a
// serving step needs no host synchronisation and can be captured in a graph.
// There is no free list: a page is free iff its count is zero and pages are
// taken lowest number first, so the outcome never depends on the order in which
// atomics land.
#include <cuda_bf16.h>

#include <climits>

#include "fa_paged.h"

namespace fa {
namespace {

// These kernels begin while the kernel before them may still be writing what they read
// (launch_after): so no pointer here is __restrict__.  That would promise that its contents
// hold for the whole kernel, and a load through it could come before grid_wait or from a
// cache that is not kept in step.

// ------------------------------------------------------------------ append
// One warp per token: rows of Hkv * d bf16 of k and v, 16 bytes a lane and step.
// Bound by HBM: 131 thousand tokens of 16 heads of dim 128 take 309 us, 6.95 TB/s; a decoding
// step of 64 tokens 2.6 us, which is launching and a chain of three loads.
constexpr int kAppendSteps = 4;  // 16-byte pieces of k and of v that a lane has in flight

__global__ void __launch_bounds__(128)
    cache_append_kernel(const uint4 *k, const uint4 *v, uint4 *k_pages, uint4 *v_pages,
                        const __grid_constant__ PageGeom g, const int *cu, int total, int chunks) {
  grid_go();
  grid_wait();
  const int lane = threadIdx.x & 31;
  const int t = (int)(blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5));
  if (t >= total) return;
  const int b = seq_of_token(cu, g.B, t);
  const long long i = (long long)t - cu[b];
  const int len = g.cache_lens[b];
  if (i < 0 || t >= cu[b + 1] || len < 0) return;
  const int page = page_of(g, b, len + i);
  if (page < 0) return;
  const size_t row = (size_t)page * g.page_size + (size_t)((len + i) % g.page_size);
  const uint4 *ks = k + (size_t)t * chunks, *vs = v + (size_t)t * chunks;
  uint4 *kd = k_pages + row * chunks, *vd = v_pages + row * chunks;
  for (int c0 = lane; c0 < chunks; c0 += 32 * kAppendSteps) {
    uint4 x[kAppendSteps], y[kAppendSteps];
#pragma unroll
    for (int u = 0; u < kAppendSteps; ++u)
      if (const int c = c0 + 32 * u; c < chunks) {
        x[u] = ks[c];
        y[u] = vs[c];
      }
#pragma unroll
    for (int u = 0; u < kAppendSteps; ++u)
      if (const int c = c0 + 32 * u; c < chunks) {
        kd[c] = x[u];
        vd[c] = y[u];
      }
  }
}

// ------------------------------------------------------------------ compact
// One block per (sequence, layer, k or v); each thread carries its 16-byte
// columns of the rows along the path in ascending order.  A path ascends, so
// row i is never the source of a later move (source of move j > i is >= j), and
// a thread touches its own columns only: no barrier is needed between moves, and
// six of them are in flight (32 sequences x 32 layers, 8 heads of dim 128, paths of up to
// 17, replayed in a graph: 17.2 us; one at a time 21, eight with fewer blocks on an SM 17.7,
// k and v by one block 17.4; a call among others 16.0, the kernel alone under ncu 15.5).  Bound by the lookups along the path and then by HBM.
constexpr int kPathChunk = 128, kMoves = 6;

__global__ void __launch_bounds__(128, 11)
    cache_compact_kernel(uint4 *k_pages, uint4 *v_pages, const __grid_constant__ PageGeom g, const int *accepted,
                         const int *n_accepted, int *lens_out, int max_accepted, int layers, int chunks) {
  __shared__ long long s_src[kPathChunk], s_dst[kPathChunk];
  __shared__ int s_bad;
  grid_go();
  grid_wait();
  const int per_seq = 2 * layers;
  const int b = blockIdx.x / per_seq, part = blockIdx.x % per_seq;
  const int layer = part >> 1;
  uint4 *pages = ((part & 1) ? v_pages : k_pages) + (size_t)layer * g.num_pages * g.page_size * chunks;
  const int len = g.cache_lens[b];
  const int n = len < 0 ? 0 : max(0, min(n_accepted[b], max_accepted));
  const int *path = accepted + (size_t)b * max_accepted;
  const long long cap = (long long)g.max_pages * g.page_size;
  int moved = 0;
  for (int i0 = 0; i0 < n; i0 += kPathChunk) {
    const int i = i0 + (int)threadIdx.x;
    if (threadIdx.x == 0) s_bad = INT_MAX;
    __syncthreads();
    if (i < n) {
      const int e = path[i], before = i > 0 ? path[i - 1] : -1;
      // the path ends where it stops ascending or leaves the table
      if (e <= before || (long long)len + e >= cap) atomicMin(&s_bad, i);
      const long long ps = (long long)len + e, pd = (long long)len + i;
      const int fs = page_of(g, b, ps), fd = page_of(g, b, pd);
      const bool move = e != i && fs >= 0 && fd >= 0;
      s_src[threadIdx.x] = move ? (long long)fs * g.page_size + ps % g.page_size : -1;
      s_dst[threadIdx.x] = move ? (long long)fd * g.page_size + pd % g.page_size : -1;
    }
    __syncthreads();
    const int stop = min(min(n - i0, kPathChunk), s_bad == INT_MAX ? INT_MAX : s_bad - i0);
    for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
      for (int m0 = 0; m0 < stop; m0 += kMoves) {
        uint4 x[kMoves];
#pragma unroll
        for (int u = 0; u < kMoves; ++u)
          if (m0 + u < stop && s_src[m0 + u] >= 0) x[u] = pages[(size_t)s_src[m0 + u] * chunks + c];
#pragma unroll
        for (int u = 0; u < kMoves; ++u)
          if (m0 + u < stop && s_src[m0 + u] >= 0) pages[(size_t)s_dst[m0 + u] * chunks + c] = x[u];
      }
    }
    moved += max(stop, 0);
    const bool ended = s_bad != INT_MAX;
    __syncthreads();
    if (ended) break;
  }
  if (part == 0 && threadIdx.x == 0) lens_out[b] = len + moved;
}

// ------------------------------------------------------------------ fork
__device__ __forceinline__ int pages_held(int len, int page_size, int max_pages) {
  if (len <= 0) return 0;
  return min((int)(((long long)len + page_size - 1) / page_size), max_pages);
}

// A block owns `cols` columns of every row, so it can read all parents' entries
// (kept in shared memory) before it writes any.  Bound by latency: 128 rows of 2048
// entries take 5 us.
__global__ void __launch_bounds__(1024)
    cache_fork_kernel(int *refs, int *table, const int *lens, const int *parents, int *lens_out, int B, int max_pages,
                      int num_pages, int page_size, int cols) {
  extern __shared__ int fresh[];  // [B, cols]
  grid_go();
  grid_wait();
  const int c0 = blockIdx.x * cols;
  for (int e = threadIdx.x; e < B * cols; e += blockDim.x) {
    const int b = e / cols, c = c0 + e % cols;
    int par = parents[b];
    if (par < -1 || par >= B) par = b;
    if (c0 == 0 && e % cols == 0) lens_out[b] = par < 0 ? 0 : lens[par];
    if (par == b || c >= max_pages) continue;
    const int now =
        par >= 0 && c < pages_held(lens[par], page_size, max_pages) ? table[(size_t)par * max_pages + c] : -1;
    const int old = c < pages_held(lens[b], page_size, max_pages) ? table[(size_t)b * max_pages + c] : -1;
    if (now != old) {  // counts of a page kept in place do not change
      if (now >= 0 && now < num_pages) atomicAdd(refs + now, 1);
      if (old >= 0 && old < num_pages) atomicSub(refs + old, 1);
    }
    fresh[e] = now;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < B * cols; e += blockDim.x) {
    const int b = e / cols, c = c0 + e % cols;
    int par = parents[b];
    if (par < -1 || par >= B) par = b;
    if (par != b && c < max_pages) table[(size_t)b * max_pages + c] = fresh[e];
  }
}

// ------------------------------------------------------------------ resize
// One block keeps the books: shrinking rows give their pages back, then the
// growing rows' needs are summed, then free pages are handed out lowest first.
// The block's time is a chain of loads, each about 0.6 us; so lengths are kept in
// shared memory, and the counts of the first pages are fetched with them and used
// where no row shrinks.  48 rows growing by up to 40 places and shrinking again take 17.6 us
// in two calls in a graph; 64 rows taking 640 pages and giving them back 12.5 us with the free
// pages in front and 55 where they follow 198000 held ones (13 stretches, read one after
// another).
constexpr int kBookThreads = 1024;
constexpr int kPagesPerThread = 16, kStretch = kBookThreads * kPagesPerThread;

// Exclusive sum over the block; *total gets the whole sum.
__device__ int block_scan(int x, int *warp_sums, int *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned s = x;  // sums may wrap (see s_need)
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  unsigned w = lane < kBookThreads / 32 ? (unsigned)warp_sums[lane] : 0u;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  *total = (int)__shfl_sync(0xffffffffu, w, 31);
  const unsigned base = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  return (int)(s - (unsigned)x + (warp > 0 ? base : 0u));
}

// copies: [0] their number, then (from, to, rows) for each
__global__ void __launch_bounds__(kBookThreads)
    cache_resize_kernel(int *refs, int *table, const int *lens, const int *new_lens, int *lens_out, int *status,
                        int *copies, int B, int max_pages, int num_pages, int page_size) {
  extern __shared__ int sm[];
  int *had = sm, *want = sm + B;              // lengths; -1 in both where the row is refused
  int *last = sm + 2 * B;   // a growing row's shared partial page (or -1)
  int *first = sm + 3 * B;  // its first rank among the taken pages, doubled; + 1 where it copies
  unsigned short *list = reinterpret_cast<unsigned short *>(sm + 4 * B);  // [kStretch]
  __shared__ int warp_sums[32];
  __shared__ int s_refused, s_copies;
  __shared__ unsigned long long s_need;  // the ranks below are 32 bits: they are used only where this fits the pool
  const int tid = threadIdx.x;
  const long long cap = (long long)max_pages * page_size;
  if (tid == 0) {
    s_refused = s_copies = 0;
    s_need = 0;
  }
  __syncthreads();
  grid_go();
  grid_wait();
  auto held = [&](int len) { return (int)(((long long)len + page_size - 1) / page_size); };
  // free pages of this thread's 16 from start + 16 tid on, as bits
  auto free_pages = [&](int start) {
    const int p = start + tid * kPagesPerThread;
    unsigned mask = 0;
    if (p + kPagesPerThread <= num_pages && (reinterpret_cast<uintptr_t>(refs) & 15u) == 0) {
#pragma unroll
      for (int i = 0; i < kPagesPerThread / 4; ++i) {
        const int4 x = __ldcg(reinterpret_cast<const int4 *>(refs + p) + i);
        mask |= ((x.x == 0) | (x.y == 0) << 1 | (x.z == 0) << 2 | (x.w == 0) << 3) << (4 * i);
      }
    } else {
      for (int i = 0; i < kPagesPerThread; ++i)
        if (p + i < num_pages && __ldcg(refs + p + i) == 0) mask |= 1u << i;
    }
    return mask;
  };
  unsigned mask = free_pages(0);
  bool shrinks = false;
  for (int b = tid; b < B; b += kBookThreads) {
    int a = lens[b], n = new_lens[b];
    if (a < 0 || n < 0 || a > cap || n > cap) {
      atomicAdd(&s_refused, 1);
      lens_out[b] = a;
      a = n = -1;
    }
    had[b] = a;
    want[b] = n;
    shrinks |= n < a;
  }
  if (__syncthreads_or(shrinks)) {
    for (int b = tid >> 5; b < B; b += kBookThreads / 32) {  // one warp a row
      if (want[b] >= had[b]) continue;
      for (int c = held(want[b]) + (tid & 31); c < held(had[b]); c += 32) {
        const int page = table[(size_t)b * max_pages + c];
        if (page >= 0 && page < num_pages) atomicSub(refs + page, 1);
        table[(size_t)b * max_pages + c] = -1;
      }
    }
    __threadfence();
    __syncthreads();
    mask = free_pages(0);
  }

  // growing rows whose last page is shared and only partly filled
  bool grows = false, any_shared = false;
  for (int b = tid; b < B; b += kBookThreads) {
    const int a = had[b];
    int page = -1;
    grows |= want[b] > a;
    if (want[b] > a && a % page_size != 0) {
      page = table[(size_t)b * max_pages + a / page_size];
      const int count = page >= 0 && page < num_pages ? __ldcg(refs + page) : 0;
      if (count <= 1) page = -1;
      first[b] = count;  // until the row's rank takes its place
    }
    last[b] = page;
    any_shared |= page >= 0;
  }
  const bool sharing = __syncthreads_or(any_shared);
  // in row order, each of them takes a copy while another row still holds the page
  int total = 0;
  if (__syncthreads_or(grows)) {
    for (int b0 = 0; b0 < B; b0 += kBookThreads) {
      const int b = b0 + tid;
      int need = 0, copy = 0;
      if (b < B && want[b] > had[b]) {
        if (sharing && last[b] >= 0) {
          int rank = 0;  // rows before this one that have to copy the same page
#pragma unroll 8
          for (int o = 0; o < b; ++o) rank += last[o] == last[b];
          copy = first[b] - rank > 1;
        }
        need = held(want[b]) - held(had[b]) + copy;
      }
      // a row needs at most 2^26 pages + 1: 32 of them stay below 2^32
      const unsigned warp_need = __reduce_add_sync(0xffffffffu, (unsigned)need);
      if ((tid & 31) == 0 && warp_need) atomicAdd(&s_need, (unsigned long long)warp_need);
      int sum;
      const int at = block_scan(need, warp_sums, &sum);
      if (b < B) first[b] = (int)(((unsigned)total + (unsigned)at) * 2u) + copy;
      total = (int)((unsigned)total + (unsigned)sum);
    }
    __syncthreads();
  }
  const bool fits = s_need <= (unsigned long long)num_pages;
  if (!fits) total = INT_MAX;  // more than there can be: count the free pages, all of them
  // enough free pages?  Those of the last stretch looked at stay in `mask`
  int found = 0, p0 = 0, at = 0;
  for (; p0 < num_pages && found < total; p0 += kStretch) {
    if (p0 > 0) mask = free_pages(p0);
    int sum;
    at = block_scan(__popc(mask), warp_sums, &sum);
    found += sum;
  }
  const bool can = fits && found >= total;
  if (tid == 0) {
    status[0] = can ? 0 : (int)min(s_need - (unsigned long long)found, (unsigned long long)INT_MAX);
    status[1] = s_refused;
  }
  for (int b = tid; b < B; b += kBookThreads)
    if (had[b] >= 0) lens_out[b] = want[b] > had[b] && !can ? had[b] : want[b];
  if (!can || total == 0) {
    if (tid == 0) copies[0] = 0;
    return;
  }
  int done = 0;
  const bool once = p0 <= kStretch;  // one stretch held them all: it is still in registers
  for (int s0 = 0; done < total; s0 += kStretch) {
    int sum = found;
    if (!once) {
      mask = free_pages(s0);
      at = block_scan(__popc(mask), warp_sums, &sum);
    }
    // the stretch's free pages in order, then one thread for each of them
    const int take = min(sum, total - done);
    int k = at;
    for (unsigned m = mask; m && k < take; m &= m - 1)
      list[k++] = (unsigned short)(tid * kPagesPerThread + __ffs(m) - 1);
    __syncthreads();
    for (int i = tid; i < take; i += kBookThreads) {
      const int page = s0 + list[i];
      k = done + i;
      int lo = 0, hi = B;  // the last row whose first rank is <= k
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((first[mid] >> 1) <= k) lo = mid;
        else hi = mid;
      }
      const int a = had[lo];
      int *row = table + (size_t)lo * max_pages;
      const int copy = first[lo] & 1, nth = k - (first[lo] >> 1);
      if (copy && nth == 0) {
        const int c = atomicAdd(&s_copies, 1);
        copies[1 + 3 * c] = last[lo];
        copies[2 + 3 * c] = page;
        copies[3 + 3 * c] = a % page_size;
        atomicSub(refs + last[lo], 1);
        row[a / page_size] = page;
      } else {
        row[held(a) + nth - copy] = page;
      }
      refs[page] = 1;
    }
    done += sum;
    __syncthreads();
  }
  __syncthreads();
  if (tid == 0) copies[0] = s_copies;
}

// The filled rows of shared pages, in every layer, k and v: contiguous runs of
// rows * chunks 16-byte pieces, cut into pieces of kCopyChunk.  Bound by HBM: about
// 24 us for 64 rows' part-filled pages in 24 layers of 8 heads of dim 128.
constexpr int kCopyChunk = 2048;

__global__ void __launch_bounds__(256)
    cache_copy_kernel(uint4 *k_pages, uint4 *v_pages, const int *copies, int num_pages, int page_size, int layers,
                      int chunks) {
  grid_go();
  grid_wait();
  const int page_chunks = page_size * chunks;
  const int pieces = (page_chunks + kCopyChunk - 1) / kCopyChunk;
  const long long work = (long long)copies[0] * layers * 2 * pieces;
  for (long long w = blockIdx.x; w < work; w += gridDim.x) {
    const int piece = (int)(w % pieces);
    const long long r = w / pieces;
    const int part = (int)(r % (2 * layers)), c = (int)(r / (2 * layers));
    const int from = copies[1 + 3 * c], to = copies[2 + 3 * c];
    const int end = min(copies[3 + 3 * c] * chunks, (piece + 1) * kCopyChunk);
    uint4 *pages = ((part & 1) ? v_pages : k_pages) + (size_t)(part >> 1) * num_pages * page_chunks;
    const uint4 *src = pages + (size_t)from * page_chunks;
    uint4 *dst = pages + (size_t)to * page_chunks;
    uint4 x[kCopyChunk / 256];
#pragma unroll
    for (int u = 0; u < kCopyChunk / 256; ++u)
      if (const int i = piece * kCopyChunk + u * 256 + (int)threadIdx.x; i < end) x[u] = src[i];
#pragma unroll
    for (int u = 0; u < kCopyChunk / 256; ++u)
      if (const int i = piece * kCopyChunk + u * 256 + (int)threadIdx.x; i < end) dst[i] = x[u];
  }
}

constexpr int kMaxBookRows = 4096;  // rows whose books fit the shared memory of one block
constexpr int kPlainSmem = 47 * 1024;  // with what is static, a launch has this much without asking

size_t resize_bytes(int B) { return ((size_t)(1 + 3 * (size_t)B) * 4 + 255) & ~size_t(255); }

}  // namespace

int check_page_table(int B, int max_pages, int num_pages, int page_size) {
  if (B <= 0 || max_pages <= 0 || num_pages <= 0 || page_size <= 0) return FA_ERR_INVALID_ARG;
  if (B > 65535) return FA_ERR_UNSUPPORTED;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128 && page_size != 256)
    return FA_ERR_UNSUPPORTED;
  if ((long long)max_pages * page_size > (1ll << 30)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

int check_page_rows(int layers, int num_pages, int page_size, int Hkv, int d) {
  if (layers <= 0 || Hkv <= 0 || d <= 0) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128 && d != 256) return FA_ERR_UNSUPPORTED;
  if (Hkv > 65535 || layers > 65535) return FA_ERR_UNSUPPORTED;
  if ((double)layers * num_pages * page_size * Hkv * d >= (double)(1ll << 40)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

}  // namespace fa

using namespace fa;

extern "C" {

int fa_cache_append(const void *k, const void *v, void *k_pages, void *v_pages, const int *page_table,
                    const int *cache_lens, const int *cu_seqlens, int B, int max_pages, int num_pages, int page_size,
                    int total, int Hkv, int d, void *stream) {
  if (!k_pages || !v_pages || !page_table || !cache_lens || !cu_seqlens) return FA_ERR_INVALID_ARG;
  if (total != 0 && (!k || !v)) return FA_ERR_INVALID_ARG;
  int rc = check_page_table(B, max_pages, num_pages, page_size);
  if (rc == FA_OK) rc = check_page_rows(1, num_pages, page_size, Hkv, d);
  if (rc != FA_OK) return rc;
  if (total < 0) return FA_ERR_INVALID_ARG;
  if ((double)total * Hkv * d >= (double)(1ll << 40)) return FA_ERR_UNSUPPORTED;
  for (const void *x : {k, v, (const void *)k_pages, (const void *)v_pages})
    if (!ptr_aligned(x, 16)) return FA_ERR_ALIGNMENT;
  for (const void *x : {(const void *)page_table, (const void *)cache_lens, (const void *)cu_seqlens})
    if (!ptr_aligned(x, 4)) return FA_ERR_ALIGNMENT;
  if ((rc = check_device()) != FA_OK) return rc;
  if (total == 0) return FA_OK;
  const PageGeom g{page_table, cache_lens, B, max_pages, num_pages, page_size};
  const unsigned grid = (unsigned)(((long long)total + 3) / 4);
  return launch_after(cache_append_kernel, grid, 1, 128, 0, static_cast<cudaStream_t>(stream),
                      static_cast<const uint4 *>(k), static_cast<const uint4 *>(v), static_cast<uint4 *>(k_pages),
                      static_cast<uint4 *>(v_pages), g, cu_seqlens, total, Hkv * d / 8);
}

int fa_cache_compact(void *k_pages, void *v_pages, const int *page_table, const int *cache_lens, const int *accepted,
                     const int *n_accepted, int *lens_out, int B, int max_accepted, int max_pages, int num_pages,
                     int page_size, int layers, int Hkv, int d, void *stream) {
  if (!k_pages || !v_pages || !page_table || !cache_lens || !accepted || !n_accepted || !lens_out)
    return FA_ERR_INVALID_ARG;
  int rc = check_page_table(B, max_pages, num_pages, page_size);
  if (rc == FA_OK) rc = check_page_rows(layers, num_pages, page_size, Hkv, d);
  if (rc != FA_OK) return rc;
  if (max_accepted <= 0 || lens_out == cache_lens) return FA_ERR_INVALID_ARG;
  if ((long long)B * layers * 2 > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  if (!ptr_aligned(k_pages, 16) || !ptr_aligned(v_pages, 16)) return FA_ERR_ALIGNMENT;
  for (const void *x : {(const void *)page_table, (const void *)cache_lens, (const void *)accepted,
                        (const void *)n_accepted, (const void *)lens_out})
    if (!ptr_aligned(x, 4)) return FA_ERR_ALIGNMENT;
  if ((rc = check_device()) != FA_OK) return rc;
  const PageGeom g{page_table, cache_lens, B, max_pages, num_pages, page_size};
  return launch_after(cache_compact_kernel, (long long)B * layers * 2, 1, 128, 0, static_cast<cudaStream_t>(stream),
                      static_cast<uint4 *>(k_pages), static_cast<uint4 *>(v_pages), g, accepted, n_accepted, lens_out,
                      max_accepted, layers, Hkv * d / 8);
}

int fa_cache_fork(int *page_refs, int *page_table, const int *cache_lens, const int *parents, int *lens_out, int B,
                  int max_pages, int num_pages, int page_size, void *stream) {
  if (!page_refs || !page_table || !cache_lens || !parents || !lens_out) return FA_ERR_INVALID_ARG;
  int rc = check_page_table(B, max_pages, num_pages, page_size);
  if (rc != FA_OK) return rc;
  if (lens_out == cache_lens) return FA_ERR_INVALID_ARG;
  if (B > kMaxBookRows) return FA_ERR_UNSUPPORTED;
  for (const void *x : {(const void *)page_refs, (const void *)page_table, (const void *)cache_lens,
                        (const void *)parents, (const void *)lens_out})
    if (!ptr_aligned(x, 4)) return FA_ERR_ALIGNMENT;
  if ((rc = check_device()) != FA_OK) return rc;
  int cols = 8;  // one 32-byte sector of each row at least
  while (cols < 1024 && cols < max_pages && B * cols * 2 <= 1024) cols *= 2;
  const int smem = B * cols * 4;
  if (smem > kPlainSmem && cudaFuncSetAttribute(cache_fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                kMaxBookRows * 8 * 4) != cudaSuccess)
    return FA_ERR_CUDA;
  const unsigned grid = (unsigned)((max_pages + cols - 1) / cols);
  const int threads = B * cols >= 1024 ? 1024 : (B * cols + 31) / 32 * 32;
  return launch_after(cache_fork_kernel, grid, 1, threads, smem, static_cast<cudaStream_t>(stream), page_refs,
                      page_table, cache_lens, parents, lens_out, B, max_pages, num_pages, page_size, cols);
}

size_t fa_cache_resize_workspace_bytes(int B) { return B > 0 && B <= kMaxBookRows ? resize_bytes(B) : 0; }

int fa_cache_resize(int *page_refs, void *k_pages, void *v_pages, int *page_table, const int *cache_lens,
                    const int *new_lens, int *lens_out, int *status, int B, int max_pages, int num_pages,
                    int page_size, int layers, int Hkv, int d, void *workspace, size_t workspace_bytes,
                    void *stream) {
  if (!page_refs || !k_pages || !v_pages || !page_table || !cache_lens || !new_lens || !lens_out || !status)
    return FA_ERR_INVALID_ARG;
  int rc = check_page_table(B, max_pages, num_pages, page_size);
  if (rc == FA_OK) rc = check_page_rows(layers, num_pages, page_size, Hkv, d);
  if (rc != FA_OK) return rc;
  if (lens_out == cache_lens || lens_out == new_lens) return FA_ERR_INVALID_ARG;
  if (B > kMaxBookRows || num_pages > (1 << 30)) return FA_ERR_UNSUPPORTED;
  if (!ptr_aligned(k_pages, 16) || !ptr_aligned(v_pages, 16)) return FA_ERR_ALIGNMENT;
  for (const void *x : {(const void *)page_refs, (const void *)page_table, (const void *)cache_lens,
                        (const void *)new_lens, (const void *)lens_out, (const void *)status})
    if (!ptr_aligned(x, 4)) return FA_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < resize_bytes(B) || !ptr_aligned(workspace, 256)) return FA_ERR_WORKSPACE;
  if ((rc = check_device()) != FA_OK) return rc;
  int *copies = static_cast<int *>(workspace);
  const int smem = B * 16 + kStretch * 2;
  if (smem > kPlainSmem && cudaFuncSetAttribute(cache_resize_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                kMaxBookRows * 16 + kStretch * 2) != cudaSuccess)
    return FA_ERR_CUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  rc = launch_after(cache_resize_kernel, 1, 1, kBookThreads, smem, s, page_refs, page_table, cache_lens, new_lens,
                    lens_out, status, copies, B, max_pages, num_pages, page_size);
  if (rc != FA_OK) return rc;
  return launch_after(cache_copy_kernel, 152 * 2, 1, 256, 0, s, static_cast<uint4 *>(k_pages),
                      static_cast<uint4 *>(v_pages), (const int *)copies, num_pages, page_size, layers, Hkv * d / 8);
}

}  // extern "C"
