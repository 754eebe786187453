// fa_paged.cu — attention of a few new tokens over a paged key/value cache:
// one token, a chain, or a tree of drafted tokens for each sequence.
//
// New token i of sequence b (c_b places cached before, n_b new) sees place p iff
// p < c_b, or p = c_b + j with j < n_b and, in a chain, j <= i, in a tree, bit j
// of the token's mask set.  What a token does not see contributes nothing,
// whatever it holds; a token that sees nothing gets O = 0 and LSE = -inf.
#include <cuda_bf16.h>

#include <cmath>

#include "fa_internal.h"

namespace fa {
namespace {

struct PagedParams {
  const __nv_bfloat16 *q, *k_pages, *v_pages;
  const int *cu;
  const long long *mask;  // [total, words] or nullptr: a chain
  __nv_bfloat16 *o;
  float *lse;
  PageGeom g;
  int words, max_new, total, H, Hkv;
  float scale;
};

// One block per (token, head); each warp takes every fourth visible key, the
// lanes share the head dimension.
template <int D>
__global__ void __launch_bounds__(128) paged_simple_kernel(const __grid_constant__ PagedParams p) {
  constexpr int E = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x / p.H, h = blockIdx.x % p.H, kh = h / (p.H / p.Hkv);
  const int b = seq_of_token(p.cu, p.g.B, t);
  const int start = p.cu[b], n = min(min(p.cu[b + 1], p.total) - start, p.max_new), i = t - start;
  const int len = max(p.g.cache_lens[b], 0);
  if (i < 0 || i >= n) return;
  float q[E], acc[E] = {}, m = -INFINITY, l = 0.f;
  for (int e = 0; e < E; ++e) q[e] = __bfloat162float(p.q[((size_t)t * p.H + h) * D + lane + 32 * e]) * p.scale;
  for (int pos = warp; pos < len + n; pos += 4) {
    if (pos >= len) {
      const int j = pos - len;
      const bool sees = p.mask ? (p.mask[(size_t)t * p.words + j / 64] >> (j % 64)) & 1 : j <= i;
      if (!sees) continue;
    }
    const int page = page_of(p.g, b, pos);
    if (page < 0) continue;
    const size_t row = ((size_t)page * p.g.page_size + pos % p.g.page_size) * p.Hkv + kh;
    float s = 0.f;
    for (int e = 0; e < E; ++e) s += q[e] * __bfloat162float(p.k_pages[row * D + lane + 32 * e]);
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float m_new = fmaxf(m, s);
    const float a = __expf(m - m_new), w = __expf(s - m_new);
    l = l * a + w;
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * a + w * __bfloat162float(p.v_pages[row * D + lane + 32 * e]);
    m = m_new;
  }
  __shared__ float s_m[4], s_l[4], s_acc[4][D];
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  for (int e = 0; e < E; ++e) s_acc[warp][lane + 32 * e] = acc[e];
  __syncthreads();
  const float top = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
  float sum = 0.f;
  for (int w = 0; w < 4; ++w)
    if (s_l[w] > 0.f) sum += s_l[w] * __expf(s_m[w] - top);
  for (int c = threadIdx.x; c < D; c += 128) {
    float x = 0.f;
    for (int w = 0; w < 4; ++w)
      if (s_l[w] > 0.f) x += s_acc[w][c] * __expf(s_m[w] - top);
    p.o[((size_t)t * p.H + h) * D + c] = __float2bfloat16(sum > 0.f ? x / sum : 0.f);
  }
  if (threadIdx.x == 0 && p.lse) p.lse[(size_t)h * p.total + t] = sum > 0.f ? top + logf(sum) : -INFINITY;
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

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_fwd_paged_workspace_bytes(int B, int max_new, int H, int Hkv, int d) {
  if (check_paged(B, 1, 1, 16, max_new, 0, H, Hkv, d) != FA_OK) return 0;
  return 256;
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
  for (const void *x : {q, k_pages, v_pages, (const void *)o})
    if (!ptr_aligned(x, 16)) return FA_ERR_ALIGNMENT;
  for (const void *x : {(const void *)page_table, (const void *)cache_lens, (const void *)cu_seqlens, (const void *)lse})
    if (!ptr_aligned(x, 4)) return FA_ERR_ALIGNMENT;
  if (!ptr_aligned(tree_mask, 8)) return FA_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < fa_fwd_paged_workspace_bytes(B, max_new, H, Hkv, d) || !ptr_aligned(workspace, 256))
    return FA_ERR_WORKSPACE;
  if ((rc = check_device()) != FA_OK) return rc;
  if (total == 0) return FA_OK;
  PagedParams p;
  p.q = static_cast<const __nv_bfloat16 *>(q);
  p.k_pages = static_cast<const __nv_bfloat16 *>(k_pages);
  p.v_pages = static_cast<const __nv_bfloat16 *>(v_pages);
  p.cu = cu_seqlens;
  p.mask = tree_mask;
  p.o = static_cast<__nv_bfloat16 *>(o);
  p.lse = lse;
  p.g = PageGeom{page_table, cache_lens, B, max_pages, num_pages, page_size};
  p.words = mask_words;
  p.max_new = max_new;
  p.total = total;
  p.H = H;
  p.Hkv = Hkv;
  p.scale = scale;
  const unsigned grid = (unsigned)total * (unsigned)H;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d == 64) paged_simple_kernel<64><<<grid, 128, 0, s>>>(p);
  else if (d == 128) paged_simple_kernel<128><<<grid, 128, 0, s>>>(p);
  else paged_simple_kernel<256><<<grid, 128, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
