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

struct WeightsParams {
  const __nv_bfloat16 *q, *k_pages;
  const int *cu;
  const unsigned long long *mask;  // [total, words] or nullptr: a chain
  const float *lse;                // [H, total]
  float *weights;                  // [B, Hkv, places]
  PageGeom g;
  int words, max_new, total, H, Hkv, G, places;
  float scale_log2, decay;
};

// A warp takes one place of one kv head at a time.
template <int D>
__global__ void __launch_bounds__(256) weights_kernel(const __grid_constant__ WeightsParams p) {
  grid_go();
  grid_wait();
  const int b = blockIdx.y / p.Hkv, kh = blockIdx.y - b * p.Hkv, lane = threadIdx.x & 31;
  const PagedSeq s = paged_seq_of(p.cu[b], p.cu[b + 1], p.g.cache_lens[b], p.total, p.max_new, p.g.max_pages * p.g.page_size);
  if (s.n == 0) return;
  for (int at = blockIdx.x * 8 + (threadIdx.x >> 5); at < min(s.keys, p.places); at += gridDim.x * 8) {
    const int page = page_of(p.g, b, at);
    float sum = 0.f;
    if (page >= 0) {
      const __nv_bfloat16 *k = p.k_pages + (((size_t)page * p.g.page_size + at % p.g.page_size) * p.Hkv + kh) * D;
      float kx[D / 32];
#pragma unroll
      for (int e = 0; e < D / 32; ++e) kx[e] = __bfloat162float(k[32 * e + lane]);
      for (int i = 0; i < s.n; ++i) {
        const int j = at - s.len;
        if (j >= 0 && (p.mask ? !((p.mask[(size_t)(s.start + i) * p.words + (j >> 6)] >> (j & 63)) & 1) : j > i)) continue;
        for (int h = kh * p.G; h < (kh + 1) * p.G; ++h) {
          const __nv_bfloat16 *q = p.q + ((size_t)(s.start + i) * p.H + h) * D;
          float dot = 0.f;
#pragma unroll
          for (int e = 0; e < D / 32; ++e) dot = fmaf(kx[e], __bfloat162float(q[32 * e + lane]), dot);
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
          const float lse = p.lse[(size_t)h * p.total + s.start + i];
          if (lse != -INFINITY) sum += ex2_mufu(fmaf(dot, p.scale_log2, -lse * 1.4426950408889634f));
        }
      }
    }
    if (lane == 0) {
      float *w = p.weights + (size_t)blockIdx.y * p.places + at;
      *w = p.decay == 0.f ? sum : fmaf(*w, p.decay, sum);
    }
  }
}

}  // namespace
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
  if (!ptr_aligned(q, 16) || !ptr_aligned(k_pages, 16)) return FA_ERR_ALIGNMENT;
  for (const void *x : {(const void *)page_table, (const void *)cache_lens, (const void *)cu_seqlens, (const void *)lse,
                        (const void *)weights})
    if (!ptr_aligned(x, 4)) return FA_ERR_ALIGNMENT;
  if (!ptr_aligned(tree_mask, 8)) return FA_ERR_ALIGNMENT;
  if ((long long)B * Hkv > 65535) return FA_ERR_UNSUPPORTED;
  if ((rc = check_device()) != FA_OK) return rc;
  if (total == 0) return FA_OK;
  WeightsParams p = {};
  p.q = static_cast<const __nv_bfloat16 *>(q);
  p.k_pages = static_cast<const __nv_bfloat16 *>(k_pages);
  p.cu = cu_seqlens;
  p.mask = reinterpret_cast<const unsigned long long *>(tree_mask);
  p.lse = lse;
  p.weights = weights;
  p.g = PageGeom{page_table, cache_lens, B, max_pages, num_pages, page_size};
  p.words = mask_words;
  p.max_new = max_new;
  p.total = total;
  p.H = H;
  p.Hkv = Hkv;
  p.G = H / Hkv;
  p.places = places;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.decay = decay;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  void (*kernel)(WeightsParams) = d == 64 ? weights_kernel<64> : d == 128 ? weights_kernel<128> : weights_kernel<256>;
  return launch_after(kernel, 256, B * Hkv, 256, 0, s, p);
}

}  // extern "C"
