// fa_rope.cu — queries and keys made ready for attention: each head's row normalised
// (or not) and its leading columns rotated by the token's positions, in one pass; the
// same with keys and values going into the pages of a cache; and the backward pass.
//
// For a row x of d values, weights w and eps, r = (mean(x^2) + eps)^(-1/2):
//   y = x r w                                   (y = x without weights)
//   (y_a, y_b) -> (y_a c - y_b s, y_b c + y_a s),  c = cos(p f_i), s = sin(p f_i)
// for pair i of the rot / 2 pairs of columns, with the position p on the pair's axis.
// Backward, from g = the gradient rotated back (s -> -s):
//   dw = sum over tokens and heads of g x r,   dx = r (w g - x r^2 mean(x w g)).
#include <cuda_bf16.h>

#include <cmath>

#include "fa_paged.h"
#include "ptx.cuh"

namespace fa {
namespace {

// These kernels begin while the kernel before them may still be writing what they read
// (launch_after), so no pointer here is __restrict__ (see fa_cache.cu).

constexpr int kMaxHalf = 128;  // pairs of columns
constexpr int kMaxAxes = 4;

// Rows of `heads` heads for each token; strides in 16-byte pieces.
struct Rows {
  const uint4 *x;
  long long token, head;
  int heads;
};

struct RopeParams {
  Rows q, k, v;         // forward: inputs; v: cache only
  Rows gq, gk;          // backward: gradients of the rotated rows
  uint4 *q_out, *k_out;  // dense [total, heads, d]; backward: dq, dk
  const void *wq, *wk;   // [d] or nullptr: no norm
  const float *inv_freq;  // [half]
  const int *positions;   // [axes, total] or nullptr (cache only): the place in the cache
  int total, half, bf16_weights;
  float eps;
  unsigned axis[kMaxHalf / 16];  // two bits for each pair
  // cache
  uint4 *k_pages, *v_pages;
  const int *cu;
  PageGeom g;
  // backward: [blocks][2][d] sums of the blocks
  float *part;
};

// A head's row is shared by kLanes lanes, each with two 16-byte pieces, A and B.
template <int D>
struct RowCfg {
  static constexpr int kLanes = D / 16, kHeads = 32 / kLanes;  // heads of a warp's step
};

// Angles.  f turns a position into radians; the kernels count in turns, where whole ones
// can be dropped exactly: step = f / (2 pi) in units of 2^-64 turns, wrapped, and position
// * step in wrapping 64-bit integers is the angle whatever the position's size (off by
// |position| * 2^-63 turns: 1e-9 radians at the far end of 32 bits; fp32 products lose
// whole turns past 2^24).  f = m 2^e with a 24-bit m; m * 2^64 / (2 pi) is 88 bits.
__device__ __forceinline__ unsigned long long turns_per_step(float f) {
  constexpr unsigned long long kInvTwoPi = 0x28BE60DB9391054Aull;  // 2^64 / (2 pi)
  const unsigned bits = __float_as_uint(f);
  const int e = (bits >> 23) & 0xff;
  const unsigned long long m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u);
  const unsigned long long lo = m * kInvTwoPi, hi = __umul64hi(m, kInvTwoPi);
  const int s = 150 - (e ? e : 1);  // f = m 2^-s
  unsigned long long g;
  if (s >= 128) g = 0;
  else if (s >= 64) g = hi >> (s - 64);
  else if (s > 0) g = (lo >> s) | (hi << (64 - s));
  else g = -s < 64 ? lo << -s : 0;
  return bits >> 31 ? 0ull - g : g;
}

// A warp's cosines and sines of one token, into its own shared memory.
__device__ __forceinline__ void turn(const RopeParams &p, const unsigned long long *step, float *cs, float *sn, int t,
                                     int place) {
  __syncwarp();
  for (int f = threadIdx.x & 31; f < p.half; f += 32) {
    int at = place;
    if (p.positions) at = p.positions[(size_t)((p.axis[f >> 4] >> (2 * (f & 15))) & 3u) * p.total + t];
    const int part = (int)(((unsigned long long)(long long)at * step[f]) >> 32);  // of a turn, in 2^-32
    sincospif((float)part * 0x1p-31f, sn + f, cs + f);
  }
  __syncwarp();
}

// Where lane `sub` of a head has its pieces, which of them are rotated and by which pairs.
//   halves: pairs (i, half + i): A and B are partners; columns past rot are split alike
//   neighbours: pairs (2 i, 2 i + 1) inside each piece
template <int D, bool NEXT>
struct Lane {
  int a, b;  // pieces of the row
  bool turn_a, turn_b;
  int fa, fb;  // first pair of each piece (NEXT), or of both
  __device__ explicit Lane(int sub, int half) {
    if (NEXT) {
      a = sub;
      b = D / 16 + sub;
      turn_a = 8 * a < 2 * half;
      turn_b = 8 * b < 2 * half;
      fa = 4 * a;
      fb = 4 * b;
    } else {
      const int n = half / 8;  // lanes with pairs
      turn_a = turn_b = sub < n;
      a = sub < n ? sub : 2 * n + (sub - n);
      b = sub < n ? n + sub : D / 16 + sub;
      fa = fb = 8 * sub;
    }
  }
  // cosines and sines of the 8 pairs: 4 of A then 4 of B (NEXT)
  __device__ void load(const float *cs, const float *sn, float (&c)[8], float (&s)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = 1.f, s[e] = 0.f;
    if (turn_a) {
#pragma unroll
      for (int e = 0; e < (NEXT ? 4 : 8); ++e) c[e] = cs[fa + e], s[e] = sn[fa + e];
    }
    if (NEXT && turn_b) {
#pragma unroll
      for (int e = 4; e < 8; ++e) c[e] = cs[fb + e - 4], s[e] = sn[fb + e - 4];
    }
  }
  // x[0..7] = A, x[8..15] = B, turned by the angle (BACK: by its negative).  Columns that
  // are not rotated are left as they are, infinities among them.
  template <bool BACK>
  __device__ void rotate(float (&x)[16], const float (&c)[8], const float (&s)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = NEXT ? 2 * e : e, j = NEXT ? 2 * e + 1 : e + 8;
      if (NEXT ? (e < 4 ? turn_a : turn_b) : turn_a) {
        const float u = x[i], w = x[j], sine = BACK ? -s[e] : s[e];
        x[i] = u * c[e] - w * sine;
        x[j] = w * c[e] + u * sine;
      }
    }
  }
};

__device__ __forceinline__ void unpack(const uint4 &v, float *x) {
  const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(w[e] << 16);
    x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack(const float *x) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

// Sum over the lanes that share a head.
template <int D>
__device__ __forceinline__ float head_sum(float x) {
#pragma unroll
  for (int o = 1; o < RowCfg<D>::kLanes; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// What a block keeps: the pairs' steps, the weights as fp32 (q, k), each warp's angles.
template <int D, int WARPS>
struct RopeSmem {
  unsigned long long step[kMaxHalf];
  float w[2][D];
  float cs[WARPS][D / 2], sn[WARPS][D / 2];
};
template <int D, int WARPS>
__device__ __forceinline__ void set_up(const RopeParams &p, RopeSmem<D, WARPS> &sm) {
  for (int f = threadIdx.x; f < p.half; f += 32 * WARPS) sm.step[f] = turns_per_step(p.inv_freq[f]);
  for (int e = threadIdx.x; e < 2 * D; e += 32 * WARPS) {
    const void *w = e < D ? p.wq : p.wk;
    const int c = e < D ? e : e - D;
    float x = 1.f;
    if (w) x = p.bf16_weights ? __bfloat162float(static_cast<const __nv_bfloat16 *>(w)[c]) : static_cast<const float *>(w)[c];
    sm.w[e < D ? 0 : 1][c] = x;
  }
  __syncthreads();
}

// ------------------------------------------------------------------ forward
// A warp's task is one token and up to kSteps steps of heads of q, k or v: all its rows are
// in flight at once, and the angles are computed while they arrive.  Sums and products are
// fp32; the one rounding is the result's, to bf16 (2^-8 of it).  Bound by HBM.
constexpr int kSteps = 4, kFwdWarps = 8;

template <int D, bool NEXT, bool CACHE>
__global__ void __launch_bounds__(32 * kFwdWarps) rope_kernel(const __grid_constant__ RopeParams p) {
  using C = RowCfg<D>;
  constexpr int kTaskHeads = kSteps * C::kHeads;
  __shared__ RopeSmem<D, kFwdWarps> sm;
  grid_go();
  grid_wait();
  set_up(p, sm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % C::kLanes;
  const Lane<D, NEXT> at(sub, p.half);
  const int tq = (p.q.heads + kTaskHeads - 1) / kTaskHeads, tk = (p.k.heads + kTaskHeads - 1) / kTaskHeads;
  const int tasks = tq + (CACHE ? 2 : 1) * tk;  // of a token
  const long long warps = (long long)gridDim.x * kFwdWarps, first = (long long)blockIdx.x * kFwdWarps + warp;
  const long long hop_t = warps / tasks;
  const int hop = (int)(warps % tasks);
  long long t = first / tasks;
  int task = (int)(first % tasks);
  for (; t < p.total; t += hop_t, task += hop, t += task >= tasks, task -= task >= tasks ? tasks : 0) {
    const int kind = task < tq ? 0 : task < tq + tk ? 1 : 2;  // q, k, v
    const Rows &x = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
    const int h0 = (task - (kind == 0 ? 0 : kind == 1 ? tq : tq + tk)) * kTaskHeads + lane / C::kLanes;
    const uint4 *from = x.x + t * x.token + h0 * x.head;
    uint4 A[kSteps], B[kSteps];
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      A[u] = B[u] = make_uint4(0, 0, 0, 0);
      if (h0 + u * C::kHeads < x.heads) {
        A[u] = from[u * C::kHeads * x.head + at.a];
        B[u] = from[u * C::kHeads * x.head + at.b];
      }
    }
    uint4 *to;
    int place = 0;
    if (CACHE) {
      const int b = seq_of_token(p.cu, p.g.B, (int)t);
      const long long i = t - p.cu[b];
      const int len = p.g.cache_lens[b];
      if (i < 0 || t >= p.cu[b + 1]) continue;  // behind the last sequence
      place = (int)(max(len, 0) + i);
      if (kind > 0) {
        const int page = len < 0 ? -1 : page_of(p.g, b, len + i);
        if (page < 0) continue;
        const size_t row = (size_t)page * p.g.page_size + (size_t)((len + i) % p.g.page_size);
        to = (kind == 1 ? p.k_pages : p.v_pages) + (row * x.heads + h0) * (D / 8);
      } else {
        to = p.q_out + ((size_t)t * x.heads + h0) * (D / 8);
      }
    } else {
      to = (kind == 0 ? p.q_out : p.k_out) + ((size_t)t * x.heads + h0) * (D / 8);
    }
    if (kind < 2) {
      turn(p, sm.step, sm.cs[warp], sm.sn[warp], (int)t, place);
      float c[8], s[8], w[16];
      at.load(sm.cs[warp], sm.sn[warp], c, s);
      const bool norm = (kind == 0 ? p.wq : p.wk) != nullptr;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        w[e] = sm.w[kind][8 * at.a + e];
        w[8 + e] = sm.w[kind][8 * at.b + e];
      }
#pragma unroll
      for (int u = 0; u < kSteps; ++u) {
        float y[16];
        unpack(A[u], y);
        unpack(B[u], y + 8);
        if (norm) {
          float sum = 0.f;
#pragma unroll
          for (int e = 0; e < 16; ++e) sum = fmaf(y[e], y[e], sum);
          const float r = rsqrtf(head_sum<D>(sum) * (1.0f / D) + p.eps);
#pragma unroll
          for (int e = 0; e < 16; ++e) y[e] = y[e] * r * w[e];
        }
        at.template rotate<false>(y, c, s);
        A[u] = pack(y);
        B[u] = pack(y + 8);
      }
    }
#pragma unroll
    for (int u = 0; u < kSteps; ++u)
      if (h0 + u * C::kHeads < x.heads) {
        to[u * C::kHeads * (D / 8) + at.a] = A[u];
        to[u * C::kHeads * (D / 8) + at.b] = B[u];
      }
  }
}

// ------------------------------------------------------------------ backward
// As the forward, with the inputs read beside the gradients where there are norms.  A
// thread adds up dw for its 16 columns over all its tasks, first of q, then of k; a block
// adds its warps' sums in shared memory and leaves them in p.part, which rope_dw_kernel
// adds up.  The division into tasks does not depend on the device, so results are bitwise
// reproducible.  Bound by HBM.
constexpr int kBwdSteps = 2, kBwdWarps = 8, kBwdBlocks = 2 * 152;

template <int D, bool NEXT>
__global__ void __launch_bounds__(32 * kBwdWarps) rope_bwd_kernel(const __grid_constant__ RopeParams p) {
  using C = RowCfg<D>;
  constexpr int kTaskHeads = kBwdSteps * C::kHeads;
  __shared__ RopeSmem<D, kBwdWarps> sm;
  __shared__ float sums[kBwdWarps][D];
  grid_go();
  grid_wait();
  set_up(p, sm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % C::kLanes;
  const Lane<D, NEXT> at(sub, p.half);
  const long long warps = (long long)gridDim.x * kBwdWarps, first = (long long)blockIdx.x * kBwdWarps + warp;
#pragma unroll 1
  for (int kind = 0; kind < 2; ++kind) {
    const Rows &gy = kind ? p.gk : p.gq, &x = kind ? p.k : p.q;
    uint4 *out = kind ? p.k_out : p.q_out;
    const bool norm = (kind ? p.wk : p.wq) != nullptr;
    const int heads = gy.heads, tasks = (heads + kTaskHeads - 1) / kTaskHeads;
    const long long hop_t = warps / tasks;
    const int hop = (int)(warps % tasks);
    long long t = first / tasks;
    int task = (int)(first % tasks);
    float dw[16] = {}, w[16];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[e] = sm.w[kind][8 * at.a + e];
      w[8 + e] = sm.w[kind][8 * at.b + e];
    }
    for (; t < p.total; t += hop_t, task += hop, t += task >= tasks, task -= task >= tasks ? tasks : 0) {
      const int h0 = task * kTaskHeads + lane / C::kLanes;
      uint4 A[kBwdSteps], B[kBwdSteps], X[kBwdSteps], Y[kBwdSteps];
#pragma unroll
      for (int u = 0; u < kBwdSteps; ++u) {
        const int h = h0 + u * C::kHeads;
        A[u] = B[u] = X[u] = Y[u] = make_uint4(0, 0, 0, 0);
        if (h < heads) {
          const uint4 *from = gy.x + t * gy.token + h * gy.head;
          A[u] = from[at.a];
          B[u] = from[at.b];
          if (norm) {
            from = x.x + t * x.token + h * x.head;
            X[u] = from[at.a];
            Y[u] = from[at.b];
          }
        }
      }
      turn(p, sm.step, sm.cs[warp], sm.sn[warp], (int)t, 0);
      float c[8], s[8];
      at.load(sm.cs[warp], sm.sn[warp], c, s);
#pragma unroll
      for (int u = 0; u < kBwdSteps; ++u) {
        float g[16];
        unpack(A[u], g);
        unpack(B[u], g + 8);
        at.template rotate<true>(g, c, s);
        if (norm) {
          float y[16], sum = 0.f, dot = 0.f;
          unpack(X[u], y);
          unpack(Y[u], y + 8);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            sum = fmaf(y[e], y[e], sum);
            dot = fmaf(y[e], w[e] * g[e], dot);
          }
          const float r = rsqrtf(head_sum<D>(sum) * (1.0f / D) + p.eps);
          const float k = head_sum<D>(dot) * (1.0f / D) * r * r;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            if (h0 + u * C::kHeads < heads) dw[e] = fmaf(g[e], y[e] * r, dw[e]);
            g[e] = r * (w[e] * g[e] - y[e] * k);
          }
        }
        if (h0 + u * C::kHeads < heads) {
          uint4 *to = out + ((size_t)t * heads + h0 + u * C::kHeads) * (D / 8);
          to[at.a] = pack(g);
          to[at.b] = pack(g + 8);
        }
      }
    }
    if (p.part == nullptr) continue;
    // over the heads of the warp's steps, then over the warps
#pragma unroll
    for (int e = 0; e < 16; ++e) {
#pragma unroll
      for (int o = C::kLanes; o < 32; o <<= 1) dw[e] += __shfl_xor_sync(0xffffffffu, dw[e], o);
      if (lane < C::kLanes) sums[warp][8 * (e < 8 ? at.a : at.b) + (e & 7)] = dw[e];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < D; e += 32 * kBwdWarps) {
      float x_sum = 0.f;
#pragma unroll
      for (int v = 0; v < kBwdWarps; ++v) x_sum += sums[v][e];
      p.part[((size_t)blockIdx.x * 2 + kind) * D + e] = x_sum;
    }
    __syncthreads();
  }
}

// Sums of `blocks` rows of 2 d columns, 32 columns to a block.  Bound by latency.
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float *part, int blocks, int d, float *dwq, float *dwk) {
  __shared__ float s[32][33];
  grid_go();
  grid_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  float x = 0.f;
#pragma unroll 4
  for (int b = warp; b < blocks; b += 32) x += part[(size_t)b * 2 * d + col];
  s[warp][lane] = x;
  __syncthreads();
  if (warp == 0) {
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < 32; ++v) sum += s[v][lane];
    float *to = col < d ? dwq : dwk;
    if (to) to[col < d ? col : col - d] = sum;
  }
}

constexpr int kMaxHeads = 65535;

// Sizes and angles, common to the three entry points.
int check_rope(int total, int H, int Hkv, int d, int rot, int n_axes, const int *axes, float eps, const float *inv_freq,
               const int *positions) {
  if (total < 0 || H <= 0 || Hkv <= 0 || d <= 0 || rot <= 0 || n_axes <= 0 || !inv_freq) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || eps < 0.f || rot > d) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128 && d != 256) return FA_ERR_UNSUPPORTED;
  if (rot % 16 != 0 || n_axes > kMaxAxes || H > kMaxHeads || Hkv > kMaxHeads) return FA_ERR_UNSUPPORTED;
  if ((double)total * H * d >= (double)(1ll << 40) || (double)total * Hkv * d >= (double)(1ll << 40))
    return FA_ERR_UNSUPPORTED;
  if (!axes && n_axes != 1) return FA_ERR_INVALID_ARG;
  if (axes)
    for (int i = 0; i < rot / 2; ++i)
      if (axes[i] < 0 || axes[i] >= n_axes) return FA_ERR_INVALID_ARG;
  if (!ptr_aligned(inv_freq, 4) || !ptr_aligned(positions, 4)) return FA_ERR_ALIGNMENT;
  return FA_OK;
}

// Pointers and strides (in elements) of rows: 16-byte pieces.
int check_rows(const void *x, long long token, long long head) {
  return ptr_aligned(x, 16) && token % 8 == 0 && head % 8 == 0 ? FA_OK : FA_ERR_ALIGNMENT;
}
Rows rows_of(const void *x, long long token, long long head, int heads) {
  return Rows{static_cast<const uint4 *>(x), token / 8, head / 8, heads};
}

int check_weights(const void *wq, const void *wk, int bf16) {
  return ptr_aligned(wq, bf16 ? 2 : 4) && ptr_aligned(wk, bf16 ? 2 : 4) ? FA_OK : FA_ERR_ALIGNMENT;
}

void set_angles(RopeParams &p, const int *positions, const float *inv_freq, int rot, const int *axes) {
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.half = rot / 2;
  for (unsigned &w : p.axis) w = 0;
  if (axes)
    for (int i = 0; i < p.half; ++i) p.axis[i >> 4] |= (unsigned)axes[i] << (2 * (i & 15));
}

template <int D, bool CACHE>
int launch_rope(const RopeParams &p, bool next, cudaStream_t stream) {
  constexpr int kTaskHeads = kSteps * RowCfg<D>::kHeads;
  const long long tasks = (p.q.heads + kTaskHeads - 1) / kTaskHeads +
                          (long long)(CACHE ? 2 : 1) * ((p.k.heads + kTaskHeads - 1) / kTaskHeads);
  const long long blocks = (p.total * tasks + kFwdWarps - 1) / kFwdWarps, most = 152 * 3;
  return launch_after(next ? rope_kernel<D, true, CACHE> : rope_kernel<D, false, CACHE>, blocks < most ? blocks : most, 1,
                      32 * kFwdWarps, 0, stream, p);
}
template <bool CACHE>
int launch_rope(const RopeParams &p, int d, bool next, cudaStream_t stream) {
  return d == 64 ? launch_rope<64, CACHE>(p, next, stream)
                 : d == 128 ? launch_rope<128, CACHE>(p, next, stream) : launch_rope<256, CACHE>(p, next, stream);
}

template <int D>
int launch_bwd(const RopeParams &p, bool next, int blocks, cudaStream_t stream) {
  return launch_after(next ? rope_bwd_kernel<D, true> : rope_bwd_kernel<D, false>, blocks, 1, 32 * kBwdWarps, 0, stream, p);
}

size_t bwd_bytes(int d) { return (size_t)kBwdBlocks * 2 * d * 4; }

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

int fa_qk_norm_rope(const void *q, long long q_token, long long q_head, const void *k, long long k_token,
                    long long k_head, const int *positions, int n_axes, const float *inv_freq, int rot,
                    const int *axes, const void *q_weight, const void *k_weight, int bf16_weights, float eps,
                    int interleaved, void *q_out, void *k_out, int total, int H, int Hkv, int d, void *stream) {
  int rc = check_rope(total, H, Hkv, d, rot, n_axes, axes, eps, inv_freq, positions);
  if (rc != FA_OK) return rc;
  if (total > 0 && (!q || !k || !positions || !q_out || !k_out)) return FA_ERR_INVALID_ARG;
  if (check_rows(q, q_token, q_head) || check_rows(k, k_token, k_head) || check_rows(q_out, 0, 0) || check_rows(k_out, 0, 0) ||
      check_weights(q_weight, k_weight, bf16_weights))
    return FA_ERR_ALIGNMENT;
  if ((rc = check_device()) != FA_OK) return rc;
  if (total == 0) return FA_OK;
  RopeParams p = {};
  p.q = rows_of(q, q_token, q_head, H);
  p.k = rows_of(k, k_token, k_head, Hkv);
  p.q_out = static_cast<uint4 *>(q_out);
  p.k_out = static_cast<uint4 *>(k_out);
  p.wq = q_weight;
  p.wk = k_weight;
  p.bf16_weights = bf16_weights;
  p.eps = eps;
  p.total = total;
  set_angles(p, positions, inv_freq, rot, axes);
  return launch_rope<false>(p, d, interleaved != 0, static_cast<cudaStream_t>(stream));
}

size_t fa_qk_norm_rope_bwd_workspace_bytes(int d) { return d == 64 || d == 128 || d == 256 ? bwd_bytes(d) : 0; }

int fa_qk_norm_rope_bwd(const void *dq_out, long long dq_token, long long dq_head, const void *dk_out,
                        long long dk_token, long long dk_head, const void *q, long long q_token, long long q_head,
                        const void *k, long long k_token, long long k_head, const int *positions, int n_axes,
                        const float *inv_freq, int rot, const int *axes, const void *q_weight, const void *k_weight,
                        int bf16_weights, float eps, int interleaved, void *dq, void *dk, float *dq_weight,
                        float *dk_weight, int total, int H, int Hkv, int d, void *workspace, size_t workspace_bytes,
                        void *stream) {
  int rc = check_rope(total, H, Hkv, d, rot, n_axes, axes, eps, inv_freq, positions);
  if (rc != FA_OK) return rc;
  if (total > 0 && (!dq_out || !dk_out || !positions || !dq || !dk)) return FA_ERR_INVALID_ARG;
  if ((q_weight && (!dq_weight || (total > 0 && !q))) || (k_weight && (!dk_weight || (total > 0 && !k))))
    return FA_ERR_INVALID_ARG;
  if (check_rows(dq_out, dq_token, dq_head) || check_rows(dk_out, dk_token, dk_head) || check_rows(q, q_token, q_head) ||
      check_rows(k, k_token, k_head) || check_rows(dq, 0, 0) || check_rows(dk, 0, 0) ||
      check_weights(q_weight, k_weight, bf16_weights) || !ptr_aligned(dq_weight, 4) || !ptr_aligned(dk_weight, 4))
    return FA_ERR_ALIGNMENT;
  const bool norm = q_weight || k_weight;
  if (norm && (!workspace || workspace_bytes < bwd_bytes(d) || !ptr_aligned(workspace, 256))) return FA_ERR_WORKSPACE;
  if ((rc = check_device()) != FA_OK) return rc;
  if (total == 0 && !norm) return FA_OK;
  RopeParams p = {};
  p.gq = rows_of(dq_out, dq_token, dq_head, H);
  p.gk = rows_of(dk_out, dk_token, dk_head, Hkv);
  p.q = rows_of(q, q_token, q_head, H);
  p.k = rows_of(k, k_token, k_head, Hkv);
  p.q_out = static_cast<uint4 *>(dq);
  p.k_out = static_cast<uint4 *>(dk);
  p.wq = q_weight;
  p.wk = k_weight;
  p.bf16_weights = bf16_weights;
  p.eps = eps;
  p.total = total;
  p.part = norm ? static_cast<float *>(workspace) : nullptr;
  set_angles(p, positions, inv_freq, rot, axes);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const long long rows = (long long)total * (H > Hkv ? H : Hkv);  // a warp takes 4 of them or more
  const int blocks = rows < 32ll * kBwdBlocks ? (int)((rows + 31) / 32) + (rows == 0) : kBwdBlocks;
  const bool next = interleaved != 0;
  rc = d == 64 ? launch_bwd<64>(p, next, blocks, s) : d == 128 ? launch_bwd<128>(p, next, blocks, s) : launch_bwd<256>(p, next, blocks, s);
  if (rc != FA_OK || !norm) return rc;
  return launch_after(rope_dw_kernel, 2 * d / 32, 1, 1024, 0, s, (const float *)p.part, blocks, d,
                      q_weight ? dq_weight : nullptr, k_weight ? dk_weight : nullptr);
}

int fa_cache_append_rope(const void *q, long long q_token, long long q_head, const void *k, long long k_token,
                         long long k_head, const void *v, long long v_token, long long v_head, void *k_pages,
                         void *v_pages, const int *page_table, const int *cache_lens, const int *cu_seqlens,
                         const int *positions, int n_axes, const float *inv_freq, int rot, const int *axes,
                         const void *q_weight, const void *k_weight, int bf16_weights, float eps, int interleaved,
                         void *q_out, int B, int max_pages, int num_pages, int page_size, int total, int H, int Hkv,
                         int d, void *stream) {
  if (!k_pages || !v_pages || !page_table || !cache_lens || !cu_seqlens) return FA_ERR_INVALID_ARG;
  int rc = check_page_table(B, max_pages, num_pages, page_size);
  if (rc == FA_OK) rc = check_page_rows(1, num_pages, page_size, Hkv, d);
  if (rc == FA_OK) rc = check_rope(total, H, Hkv, d, rot, n_axes, axes, eps, inv_freq, positions);
  if (rc != FA_OK) return rc;
  if (total > 0 && (!q || !k || !v || !q_out)) return FA_ERR_INVALID_ARG;
  if (check_rows(q, q_token, q_head) || check_rows(k, k_token, k_head) || check_rows(v, v_token, v_head) ||
      check_rows(q_out, 0, 0) || check_rows(k_pages, 0, 0) || check_rows(v_pages, 0, 0) ||
      check_weights(q_weight, k_weight, bf16_weights))
    return FA_ERR_ALIGNMENT;
  for (const void *x : {(const void *)page_table, (const void *)cache_lens, (const void *)cu_seqlens})
    if (!ptr_aligned(x, 4)) return FA_ERR_ALIGNMENT;
  if ((rc = check_device()) != FA_OK) return rc;
  if (total == 0) return FA_OK;
  RopeParams p = {};
  p.q = rows_of(q, q_token, q_head, H);
  p.k = rows_of(k, k_token, k_head, Hkv);
  p.v = rows_of(v, v_token, v_head, Hkv);
  p.q_out = static_cast<uint4 *>(q_out);
  p.wq = q_weight;
  p.wk = k_weight;
  p.bf16_weights = bf16_weights;
  p.eps = eps;
  p.total = total;
  p.k_pages = static_cast<uint4 *>(k_pages);
  p.v_pages = static_cast<uint4 *>(v_pages);
  p.cu = cu_seqlens;
  p.g = PageGeom{page_table, cache_lens, B, max_pages, num_pages, page_size};
  set_angles(p, positions, inv_freq, rot, axes);
  return launch_rope<true>(p, d, interleaved != 0, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
