// paged_seq.h — what a call's tables say of one sequence of the paged attention, held
// inside the call's arrays whatever the tables contain.  Free of CUDA headers, so that
// the arithmetic also compiles for the host.
#pragma once

#ifdef __CUDACC__
#define FA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define FA_HOST_DEVICE inline
#endif

namespace fa {

// Sequence b: its first new token, their number, places cached, places in all.
struct PagedSeq {
  int start, n, len, keys;
};

// From its offsets c0, c1 and its length.  Both ends are brought into [0, total] before they
// are subtracted (c1 may be anything, and c1 - c0 may pass 32 bits), so 0 <= start and
// start + n <= total.  places: what a row of the page table has room for, at most 2^30.
FA_HOST_DEVICE PagedSeq paged_seq_of(int c0, int c1, int cache_len, int total, int max_new, int places) {
  PagedSeq s;
  s.start = c0 < 0 ? 0 : c0 < total ? c0 : total;
  const int end = c1 < s.start ? s.start : c1 < total ? c1 : total;
  s.n = end - s.start < max_new ? end - s.start : max_new;
  s.len = cache_len < 0 ? 0 : cache_len < places ? cache_len : places;
  s.keys = s.len + s.n < places ? s.len + s.n : places;
  return s;
}

}  // namespace fa
