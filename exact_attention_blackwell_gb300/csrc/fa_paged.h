// fa_paged.h — what the paged key/value cache's kernels (fa_cache.cu, fa_paged.cu)
// share, beside fa_internal.h.
#pragma once

#include "fa_internal.h"

namespace fa {

#ifdef __CUDACC__
// The kernels of a decoding step follow one another and are short, so each may be
// launched while the one before it drains: it sets itself up, and before its first
// access to global memory waits until everything launched before has completed
// (launch_after; grid_wait).  grid_go lets the next such kernel begin early.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_go() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
int launch_after(void (*kernel)(P...), long long blocks, int blocks_y, int threads, size_t smem, cudaStream_t stream,
                 A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks, (unsigned)blocks_y);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
#endif

// A paged key/value cache (fa_cache.cu, fa_paged.cu): pages [num_pages,
// page_size, Hkv, d] bf16, place p of sequence b in row p % page_size of page
// page_table[b][p / page_size].
struct PageGeom {
  const int *page_table;  // [B, max_pages]
  const int *cache_lens;  // [B]
  int B, max_pages, num_pages, page_size;
};

inline bool ptr_aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
// Argument checks of the page table's and the pages' sizes (FA_OK or the error).
int check_page_table(int B, int max_pages, int num_pages, int page_size);
int check_page_rows(int layers, int num_pages, int page_size, int Hkv, int d);
// The same of attention over the cache, with its new tokens (fa_paged.cu).
int check_paged(int B, int max_pages, int num_pages, int page_size, int max_new, int total, int H, int Hkv, int d);

#ifdef __CUDACC__
// Page of place `pos` of sequence b, or -1 where there is none: outside the
// table, or an entry that names no page.
__device__ __forceinline__ int page_of(const PageGeom &g, int b, long long pos) {
  if (pos < 0 || pos >= (long long)g.max_pages * g.page_size) return -1;
  const int page = g.page_table[(size_t)b * g.max_pages + (int)(pos / g.page_size)];
  return page >= 0 && page < g.num_pages ? page : -1;
}

// Sequence of packed token t: the last b with cu[b] <= t, found by a whole warp
// 32 offsets at a time (two dependent loads for up to 1024 sequences).  Always
// in [0, B); a table that does not ascend gives some such value.
__device__ __forceinline__ int seq_of_token(const int *cu, int B, int t) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + (int)(threadIdx.x & 31) * step;
    const unsigned seen = __ballot_sync(0xffffffffu, at < hi && (at == lo || cu[at] <= t));
    lo += (31 - __clz(seen)) * step;
    hi = min(lo + step, hi);
  }
  return lo;
}
#endif

// FA_OK on a GB300 (compute capability 10.3), else FA_ERR_UNSUPPORTED or FA_ERR_CUDA.
int check_device();

// Encodes a 4-D bf16 tensor map, box[0] = 64 columns, 128-byte swizzle; strides in bytes
// for dims 1..3.
int encode_bf16_box_map(CUtensorMap *map, const void *base, const uint64_t dims[4], const uint64_t strides[3],
                        const uint32_t box[4]);

// Map of k or v pages [num_pages, page_size, Hkv, d]: box = 64 columns x `box_rows`
// rows of one head, 128-byte swizzle.  `narrow`: fetch 128 instead of 256 bytes into L2
// around each box row (for boxes whose 128-byte rows are all that is read of a row).
int encode_page_map(CUtensorMap *map, const void *pages, int num_pages, int page_size, int Hkv, int d, int box_rows,
                    bool narrow);

// Test builds only (-DFA_TEST_STALL), as in fa_internal.h: 4: the paged kernel's first P,
// 5: the few-rows paged kernel's first tile read, 6: the weight sums' first product read.
#ifdef FA_TEST_STALL
int set_test_stall_paged(int mode);
int set_test_stall_weights(int mode);
#endif

}  // namespace fa
