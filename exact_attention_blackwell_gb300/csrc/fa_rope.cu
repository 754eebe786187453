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
  int parts;  // pieces that a token's rows are cut into (backward: of q)
  int k_parts, q_blocks;  // backward: of k, and the blocks that work on q
  float eps;
  unsigned axis[kMaxHalf / 16];  // two bits for each pair
  // cache
  uint4 *k_pages, *v_pages;
  const int *cu;
  PageGeom g;
  // backward: [blocks][d] sums of the blocks
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
// whole turns past 2^24).  f = m 2^-s with a 24-bit m.  f may be as large as 2^128, so that
// 1 / (2 pi) has to be known to 64 + 128 bits: m * 2^192 / (2 pi) is 216 bits, of which the
// step is the 64 from 128 + s on.  (With the first 64 bits of 1 / (2 pi) alone the step was
// off by f / 2 units: 4e-6 radians at the far end for f = 1e4.)
__device__ __forceinline__ unsigned long long turns_per_step(float f) {
  // the lowest word first
  constexpr unsigned kInvTwoPi[6] = {0x4F10E410u, 0x36D8A566u, 0x7D4D3770u, 0x7F09D5F4u, 0x9391054Au, 0x28BE60DBu};
  const unsigned bits = __float_as_uint(f);
  const int e = (bits >> 23) & 0xff;
  const unsigned m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u);
  const int from = 278 - (e ? e : 1), word = from >> 5;  // 128 + s, 23 to 277
  unsigned long long sum = 0;
  unsigned a = 0, b = 0, c = 0;  // the product's words from there on
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    sum = (i < 6 ? (unsigned long long)m * kInvTwoPi[i < 6 ? i : 0] : 0ull) + (sum >> 32);
    if (i == word) a = (unsigned)sum;
    if (i == word + 1) b = (unsigned)sum;
    if (i == word + 2) c = (unsigned)sum;
  }
  const unsigned lo = __funnelshift_r(a, b, from), hi = __funnelshift_r(b, c, from);  // by from % 32
  const unsigned long long g = (unsigned long long)hi << 32 | lo;
  return bits >> 31 ? 0ull - g : g;
}

// A lane's share of a token's angles: pairs lane, lane + 32, ...
template <int D>
struct Share {
  static constexpr int kN = (D / 2 + 31) / 32;
  int at[kN];  // positions
  __device__ void load(const RopeParams &p, long long t) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int f = (threadIdx.x & 31) + 32 * i;
      at[i] = f < p.half ? p.positions[(size_t)((p.axis[f >> 4] >> (2 * (f & 15))) & 3u) * p.total + t] : 0;
    }
  }
  __device__ void place(int x) {
#pragma unroll
    for (int i = 0; i < kN; ++i) at[i] = x;
  }
  // cosines and sines into the warp's own shared memory
  __device__ void turn(const RopeParams &p, const unsigned long long *step, float *cs, float *sn) const {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int f = (threadIdx.x & 31) + 32 * i;
      if (f < p.half) {
        const int part = (int)(((unsigned long long)(long long)at[i] * step[f]) >> 32);  // of a turn, in 2^-32
        sincospif((float)part * 0x1p-31f, sn + f, cs + f);
      }
    }
    __syncwarp();
  }
};

// Where lane `sub` of a head has its pieces A and B, and which of its eight pairs of columns
// are rotated, by which angles.
//   halves: pairs (i, half + i), one column in A and one in B; columns past rot are split alike
//   neighbours (NEXT): pairs (2 i, 2 i + 1), four in each piece
// A lane's values are held as xa[8], xb[8]: the first and the second columns of its pairs.
template <int D, bool NEXT>
struct Lane {
  int a, b;  // pieces of the row
  bool turn_a, turn_b;  // its first and its last four pairs
  int fa, fb;           // their angles
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
      fa = 8 * sub;
      fb = 8 * sub + 4;
    }
  }
  __device__ void unpack(const uint4 &A, const uint4 &B, float (&xa)[8], float (&xb)[8]) const {
    const unsigned v[8] = {A.x, A.y, A.z, A.w, B.x, B.y, B.z, B.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float lo = __uint_as_float(v[e] << 16), hi = __uint_as_float(v[e] & 0xffff0000u);
      if (NEXT) xa[e] = lo, xb[e] = hi;
      else if (e < 4) xa[2 * e] = lo, xa[2 * e + 1] = hi;
      else xb[2 * e - 8] = lo, xb[2 * e - 7] = hi;
    }
  }
  __device__ void pack(const float (&xa)[8], const float (&xb)[8], uint4 &A, uint4 &B) const {
    unsigned v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[e] = NEXT ? pack_bf16x2(xa[e], xb[e])
                  : e < 4 ? pack_bf16x2(xa[2 * e], xa[2 * e + 1]) : pack_bf16x2(xb[2 * e - 8], xb[2 * e - 7]);
    A = make_uint4(v[0], v[1], v[2], v[3]);
    B = make_uint4(v[4], v[5], v[6], v[7]);
  }
  // per pair, from an array over the row's columns
  __device__ void columns(const float *row, float (&ya)[8], float (&yb)[8]) const {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const float4 v = *reinterpret_cast<const float4 *>(row + 8 * (g < 2 ? a : b) + 4 * (g & 1));
      if (NEXT) {
        ya[2 * g] = v.x, yb[2 * g] = v.y, ya[2 * g + 1] = v.z, yb[2 * g + 1] = v.w;
      } else {
        float *y = g < 2 ? ya + 4 * g : yb + 4 * (g - 2);
        y[0] = v.x, y[1] = v.y, y[2] = v.z, y[3] = v.w;
      }
    }
  }
  __device__ void angles(const float *cs, const float *sn, float (&c)[8], float (&s)[8]) const {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      float4 x = make_float4(1.f, 1.f, 1.f, 1.f), y = make_float4(0.f, 0.f, 0.f, 0.f);
      if (g ? turn_b : turn_a) {
        x = *reinterpret_cast<const float4 *>(cs + (g ? fb : fa));
        y = *reinterpret_cast<const float4 *>(sn + (g ? fb : fa));
      }
      c[4 * g] = x.x, c[4 * g + 1] = x.y, c[4 * g + 2] = x.z, c[4 * g + 3] = x.w;
      s[4 * g] = y.x, s[4 * g + 1] = y.y, s[4 * g + 2] = y.z, s[4 * g + 3] = y.w;
    }
  }
  __device__ bool turned(int e) const { return e < 4 ? turn_a : turn_b; }
};

// Sum over the lanes that share a head.
template <int D>
__device__ __forceinline__ float head_sum(float x) {
#pragma unroll
  for (int o = 1; o < RowCfg<D>::kLanes; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ float square_sum(const float (&xa)[8], const float (&xb)[8]) {
  float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    ffma2(s0, s1, xa[e], xa[e + 1], xa[e], xa[e + 1], s0, s1);
    ffma2(s2, s3, xb[e], xb[e + 1], xb[e], xb[e + 1], s2, s3);
  }
  return (s0 + s1) + (s2 + s3);
}

// What a block keeps: the pairs' steps, the weights as fp32 (q, k), each warp's angles.
template <int D, int WARPS>
struct RopeSmem {
  unsigned long long step[kMaxHalf];
  __align__(16) float w[2][D];
  __align__(16) float cs[WARPS][D / 2];
  __align__(16) float sn[WARPS][D / 2];
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
// A step is kHeads heads of one token's q, k or v: a row to kLanes lanes.  A token's steps are
// cut into p.parts equal pieces, and a warp goes through its pieces kSteps steps at a time,
// the next ones' rows on their way while these are worked on.  The weights go into the
// rotation's factors, once for a token, and r is multiplied last.  Sums and products are fp32;
// the one rounding is the result's, to bf16 (2^-8 of it).  Bound by HBM: 32768 tokens of 16 + 16
// heads of dim 128 take 86 us, 6.3 TB/s (a task at a time, without the steps ahead, 104); 20011
// tokens of 32 + 8 heads from views, pairs of neighbours on three axes, 69 us, 6.0 TB/s; 65536
// into the pages with their values 242 us, 6.7 TB/s.  64 tokens into the cache 4.5 us: launch,
// the token's way to its page, the rows.
constexpr int kSteps = 3, kFwdWarps = 8, kFwdBlocks = 2;

template <int D, bool NEXT, bool CACHE>
__global__ void __launch_bounds__(32 * kFwdWarps, kFwdBlocks) rope_kernel(const __grid_constant__ RopeParams p) {
  using C = RowCfg<D>;
  __shared__ RopeSmem<D, kFwdWarps> sm;
  grid_go();
  grid_wait();
  set_up(p, sm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Lane<D, NEXT> at(lane % C::kLanes, p.half);
  const int nq = (p.q.heads + C::kHeads - 1) / C::kHeads, nk = (p.k.heads + C::kHeads - 1) / C::kHeads;
  const int steps = nq + (CACHE ? 2 : 1) * nk, each = (steps + p.parts - 1) / p.parts;
  const int warps = gridDim.x * kFwdWarps, first = blockIdx.x * kFwdWarps + warp;
  // where the warp is: a token, its piece, and of that the steps from s on
  struct Here {
    unsigned t;
    int piece, s;
  };
  auto begin = [&](Here &h) { h.s = h.piece * each; };
  auto ahead = [&](Here &h) {  // the next steps
    h.s += kSteps;
    if (h.s < min((h.piece + 1) * each, steps)) return;
    h.t += warps / p.parts;
    h.piece += warps % p.parts;
    if (h.piece >= p.parts) h.piece -= p.parts, ++h.t;
    begin(h);
  };
  auto kind_of = [&](int s) { return s < nq ? 0 : s < nq + nk ? 1 : 2; };
  auto head_of = [&](int s, int kind) { return (s - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk)) * C::kHeads + lane / C::kLanes; };
  auto live = [&](const Here &h, int u) { return h.t < (unsigned)p.total && h.s + u < min((h.piece + 1) * each, steps); };
  uint4 A[kSteps], B[kSteps];
  Share<D> share, share_next;
  int place = 0, page = -1, row = 0, place_next = 0, page_next = -1, row_next = 0;  // of the token in its sequence's cache
  bool mine = true, mine_next = true;
  auto fetch = [&](const Here &h, uint4 (&X)[kSteps], uint4 (&Y)[kSteps]) {
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      X[u] = Y[u] = make_uint4(0, 0, 0, 0);
      if (!live(h, u)) continue;
      const int kind = kind_of(h.s + u), head = head_of(h.s + u, kind);
      const Rows &r = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
      if (head >= r.heads) continue;
      const uint4 *from = r.x + (long long)h.t * r.token + head * r.head;
      X[u] = from[at.a];
      Y[u] = from[at.b];
    }
  };
  auto look_up = [&](unsigned t) {  // of the token that comes next
    if (t >= (unsigned)p.total) return;
    if (CACHE) {
      const int b = seq_of_token(p.cu, p.g.B, (int)t);
      const long long i = (long long)t - p.cu[b];
      const int len = p.g.cache_lens[b];
      mine_next = i >= 0 && (int)t < p.cu[b + 1];  // else behind the last sequence
      place_next = (int)(max(len, 0) + i);
      page_next = mine_next && len >= 0 ? page_of(p.g, b, len + i) : -1;
      row_next = (int)((len + i) & (p.g.page_size - 1));
    }
    if (!CACHE || p.positions) share_next.load(p, t);
    else share_next.place(place_next);
  };
  Here here;
  here.t = first / p.parts;
  here.piece = first % p.parts;
  begin(here);
  fetch(here, A, B);
  look_up(here.t);
  unsigned t_now = 0xffffffffu;
  int kind_now = -1;
  float ca[8], sa[8], cb[8], nsb[8];
  while (here.t < (unsigned)p.total) {
    if (here.t != t_now) {
      share = share_next;
      place = place_next, page = page_next, row = row_next, mine = mine_next;
      share.turn(p, sm.step, sm.cs[warp], sm.sn[warp]);
      kind_now = -1;
      t_now = here.t;
    }
    Here next = here;
    ahead(next);
    uint4 X[kSteps], Y[kSteps];
    fetch(next, X, Y);
    if (next.t != here.t) look_up(next.t);
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      if (!live(here, u)) continue;
      const int kind = kind_of(here.s + u), head = head_of(here.s + u, kind);
      const Rows &r = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
      if (kind < 2) {
        if (kind != kind_now) {
          float c[8], s[8], wa[8], wb[8];
          at.angles(sm.cs[warp], sm.sn[warp], c, s);
          at.columns(sm.w[kind], wa, wb);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            ca[e] = c[e] * wa[e];
            sa[e] = s[e] * wa[e];
            cb[e] = c[e] * wb[e];
            nsb[e] = -s[e] * wb[e];
          }
          kind_now = kind;
        }
        float xa[8], xb[8], ya[8], yb[8], k = 1.f;
        at.unpack(A[u], B[u], xa, xb);
        if ((kind == 0 ? p.wq : p.wk) != nullptr) k = rsqrtf(head_sum<D>(square_sum(xa, xb)) * (1.0f / D) + p.eps);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          fmul2(ya[e], ya[e + 1], xa[e], xa[e + 1], ca[e], ca[e + 1]);
          fmul2(yb[e], yb[e + 1], xb[e], xb[e + 1], cb[e], cb[e + 1]);
          if (2 * p.half == D || at.turned(e)) {  // the others are left as they are, infinities among them
            ffma2(ya[e], ya[e + 1], xb[e], xb[e + 1], nsb[e], nsb[e + 1], ya[e], ya[e + 1]);
            ffma2(yb[e], yb[e + 1], xa[e], xa[e + 1], sa[e], sa[e + 1], yb[e], yb[e + 1]);
          }
          fmul2(ya[e], ya[e + 1], ya[e], ya[e + 1], k, k);
          fmul2(yb[e], yb[e + 1], yb[e], yb[e + 1], k, k);
        }
        at.pack(ya, yb, A[u], B[u]);
      }
      if (head >= r.heads || (CACHE && (!mine || (kind > 0 && page < 0)))) continue;
      uint4 *to = kind == 0 ? p.q_out : p.k_out;
      size_t line = here.t;
      if (CACHE && kind > 0) {
        to = kind == 1 ? p.k_pages : p.v_pages;
        line = (size_t)page * p.g.page_size + row;
      }
      to += (line * r.heads + head) * (D / 8);
      to[at.a] = A[u];
      to[at.b] = B[u];
    }
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      A[u] = X[u];
      B[u] = Y[u];
    }
    here = next;
  }
}

// ------------------------------------------------------------------ backward
// As the forward, a step at a time, with the inputs read beside the gradients where there are
// norms.  A lane's pieces come by asynchronous copies into places of its own in shared memory,
// kRing - 1 steps ahead.  The first blocks work on q and the others on k, in proportion to
// their heads, so that a thread adds up dw for 16 columns of one weight in registers; a block
// adds its warps' sums and leaves them in p.part, which rope_dw_kernel adds up.  The division
// into steps does not depend on the device, so results are bitwise reproducible.  Bound by
// HBM: the forward's 32768 tokens take 125 us with rope_dw_kernel, 6.4 TB/s (205 with each step's
// loads in registers and q and k one after the other, whose 350 instructions a step were the
// bound); 6009 tokens of 16 + 4 heads of dim 256 38 us, 4.9 TB/s, of which some 9 are set-up,
// the last steps and the second kernel.
constexpr int kBwdWarps = 8, kBwdBlocks = 2 * 152, kRing = 3;

__device__ __forceinline__ void copy16(uint32_t to, const void *from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const void *from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// One step of one warp: pieces of the gradient (A, B) and of the input; a lane's positions, with
// the first step of a token's piece.
template <int D>
struct BwdStage {
  uint4 x[4][32];
  int at[Share<D>::kN][32];
};

template <int D, bool NEXT>
__global__ void __launch_bounds__(32 * kBwdWarps, 2) rope_bwd_kernel(const __grid_constant__ RopeParams p) {
  using C = RowCfg<D>;
  __shared__ RopeSmem<D, kBwdWarps> sm;
  __shared__ float sums[kBwdWarps][D];
  extern __shared__ __align__(16) uint8_t stages[];
  grid_go();
  grid_wait();
  set_up(p, sm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  BwdStage<D> *ring = reinterpret_cast<BwdStage<D> *>(stages) + warp * kRing;
  const Lane<D, NEXT> at(lane % C::kLanes, p.half);
  const int kind = (int)blockIdx.x < p.q_blocks ? 0 : 1;
  const Rows gy = kind ? p.gk : p.gq, in = kind ? p.k : p.q;
  const bool norm = (kind ? p.wk : p.wq) != nullptr;
  const int heads = gy.heads, steps = (heads + C::kHeads - 1) / C::kHeads;
  const int parts = kind ? p.k_parts : p.parts, each = (steps + parts - 1) / parts;
  const int warps = (kind ? (int)gridDim.x - p.q_blocks : p.q_blocks) * kBwdWarps;
  const int first = ((int)blockIdx.x - (kind ? p.q_blocks : 0)) * kBwdWarps + warp;
  const unsigned hop_t = warps / parts, hop = warps % parts;
  // where the warp is: a token, its piece, and of that step s; and the lane's head there
  struct Here {
    unsigned t;
    int piece, s;
  };
  auto ahead = [&](Here &h) {
    if (++h.s < min((h.piece + 1) * each, steps)) return;
    h.t += hop_t;
    h.piece += hop;
    if (h.piece >= parts) h.piece -= parts, ++h.t;
    h.s = h.piece * each;
  };
  auto head_of = [&](const Here &h) { return h.s * C::kHeads + lane / C::kLanes; };
  auto fetch = [&](const Here &h, int slot) {  // a lane reads back only what it has copied itself
    if (h.t < (unsigned)p.total) {
      BwdStage<D> &to = ring[slot];
      const int head = head_of(h);
      if (head < heads) {
        const uint4 *from = gy.x + ((long long)h.t * gy.token + head * gy.head);
        copy16(smem_u32(&to.x[0][lane]), from + at.a);
        copy16(smem_u32(&to.x[1][lane]), from + at.b);
        if (norm) {
          from = in.x + ((long long)h.t * in.token + head * in.head);
          copy16(smem_u32(&to.x[2][lane]), from + at.a);
          copy16(smem_u32(&to.x[3][lane]), from + at.b);
        }
      }
      if (h.s == h.piece * each) {
#pragma unroll
        for (int i = 0; i < Share<D>::kN; ++i)
          if (const int f = lane + 32 * i; f < p.half)
            copy4(smem_u32(&to.at[i][lane]), p.positions + (size_t)((p.axis[f >> 4] >> (2 * (f & 15))) & 3u) * p.total + h.t);
      }
    }
    copies_end();
  };
  uint4 *out = kind ? p.k_out : p.q_out;
  float dwa[8] = {}, dwb[8] = {}, c[8], s[8], ns[8];
  Here here, next;
  here.t = first / parts;
  here.piece = first % parts;
  here.s = here.piece * each;
  next = here;
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) {
    fetch(next, i);
    ahead(next);
  }
  int slot = 0;
  for (; here.t < (unsigned)p.total; ahead(here)) {
    fetch(next, slot == 0 ? kRing - 1 : slot - 1);
    ahead(next);
    copies_wait<kRing - 1>();
    const BwdStage<D> &stage = ring[slot];
    if (here.s == here.piece * each) {
      Share<D> share;
#pragma unroll
      for (int i = 0; i < Share<D>::kN; ++i) share.at[i] = stage.at[i][lane];
      share.turn(p, sm.step, sm.cs[warp], sm.sn[warp]);
      at.angles(sm.cs[warp], sm.sn[warp], c, s);
#pragma unroll
      for (int e = 0; e < 8; ++e) ns[e] = -s[e];
    }
    // A lane without a row has old pieces, which stay in its own values: its head's lanes have none either.
    const int head = head_of(here);
    float ga[8], gb[8];
    {
      float da[8], db[8];
      at.unpack(stage.x[0][lane], stage.x[1][lane], da, db);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        fmul2(ga[e], ga[e + 1], da[e], da[e + 1], c[e], c[e + 1]);
        fmul2(gb[e], gb[e + 1], db[e], db[e + 1], c[e], c[e + 1]);
        if (2 * p.half == D || at.turned(e)) {
          ffma2(ga[e], ga[e + 1], db[e], db[e + 1], s[e], s[e + 1], ga[e], ga[e + 1]);
          ffma2(gb[e], gb[e + 1], da[e], da[e + 1], ns[e], ns[e + 1], gb[e], gb[e + 1]);
        }
      }
    }
    if (norm) {
      float xa[8], xb[8], ha[8], hb[8], d0 = 0.f, d1 = 0.f, d2 = 0.f, d3 = 0.f;
      at.unpack(stage.x[2][lane], stage.x[3][lane], xa, xb);
      at.columns(sm.w[kind], ha, hb);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {  // h = w g
        fmul2(ha[e], ha[e + 1], ha[e], ha[e + 1], ga[e], ga[e + 1]);
        fmul2(hb[e], hb[e + 1], hb[e], hb[e + 1], gb[e], gb[e + 1]);
        ffma2(d0, d1, xa[e], xa[e + 1], ha[e], ha[e + 1], d0, d1);
        ffma2(d2, d3, xb[e], xb[e + 1], hb[e], hb[e + 1], d2, d3);
      }
      float sum = square_sum(xa, xb), dot = (d0 + d1) + (d2 + d3);
#pragma unroll
      for (int o = 1; o < C::kLanes; o <<= 1)
        fadd2(sum, dot, sum, dot, __shfl_xor_sync(0xffffffffu, sum, o), __shfl_xor_sync(0xffffffffu, dot, o));
      const float r = rsqrtf(sum * (1.0f / D) + p.eps), k = -dot * (1.0f / D) * r * r * r;
      if (head < heads) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          fmul2(ga[e], ga[e + 1], ga[e], ga[e + 1], xa[e], xa[e + 1]);
          fmul2(gb[e], gb[e + 1], gb[e], gb[e + 1], xb[e], xb[e + 1]);
          ffma2(dwa[e], dwa[e + 1], ga[e], ga[e + 1], r, r, dwa[e], dwa[e + 1]);
          ffma2(dwb[e], dwb[e + 1], gb[e], gb[e + 1], r, r, dwb[e], dwb[e + 1]);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        fmul2(xa[e], xa[e + 1], xa[e], xa[e + 1], k, k);
        fmul2(xb[e], xb[e + 1], xb[e], xb[e + 1], k, k);
        ffma2(ga[e], ga[e + 1], ha[e], ha[e + 1], r, r, xa[e], xa[e + 1]);
        ffma2(gb[e], gb[e + 1], hb[e], hb[e + 1], r, r, xb[e], xb[e + 1]);
      }
    }
    if (head < heads) {
      uint4 A, B, *to = out + ((size_t)here.t * heads + head) * (D / 8);
      at.pack(ga, gb, A, B);
      to[at.a] = A;
      to[at.b] = B;
    }
    slot = slot + 1 == kRing ? 0 : slot + 1;
  }
  copies_wait<0>();
  if (p.part == nullptr) return;
  // over the heads of the warp's steps, then over the warps
#pragma unroll
  for (int e = 0; e < 8; ++e) {
#pragma unroll
    for (int o = C::kLanes; o < 32; o <<= 1) {
      dwa[e] += __shfl_xor_sync(0xffffffffu, dwa[e], o);
      dwb[e] += __shfl_xor_sync(0xffffffffu, dwb[e], o);
    }
    if (lane < C::kLanes) {
      sums[warp][NEXT ? 8 * (e < 4 ? at.a : at.b) + 2 * (e & 3) : 8 * at.a + e] = dwa[e];
      sums[warp][NEXT ? 8 * (e < 4 ? at.a : at.b) + 2 * (e & 3) + 1 : 8 * at.b + e] = dwb[e];
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < D; e += 32 * kBwdWarps) {
    float x_sum = 0.f;
#pragma unroll
    for (int v = 0; v < kBwdWarps; ++v) x_sum += sums[v][e];
    p.part[(size_t)blockIdx.x * D + e] = x_sum;
  }
}

// Sums of q's and of k's blocks' rows of d columns, 32 columns of one of them to a block, in
// the order of the blocks' numbers.  Bound by latency: some 3 us behind the main kernel.
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float *part, int q_blocks, int blocks, int d, float *dwq,
                                                       float *dwk) {
  __shared__ float s[32][33];
  grid_go();
  grid_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, groups = d / 32, kind = blockIdx.x / groups;
  const int col = blockIdx.x % groups * 32 + lane;
  float *to = kind ? dwk : dwq;
  if (to == nullptr) return;
  float x = 0.f;
  const int end = kind ? blocks : q_blocks;
#pragma unroll 8
  for (int b = (kind ? q_blocks : 0) + warp; b < end; b += 32) x += part[(size_t)b * d + col];
  s[warp][lane] = x;
  __syncthreads();
  if (warp == 0) {
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < 32; ++v) sum += s[v][lane];
    to[col] = sum;
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

// Pieces of a token's steps, so that there are `pieces` at least in all, one for each warp: 64
// tokens of 32 + 8 + 8 heads of dim 128 into the cache 4.5 us instead of 9.9 with a warp to a
// token.  (Four pieces for each warp of the backward pass changed nothing.)
int parts_for(int total, int steps, int pieces) {
  const long long want = ((long long)pieces + total - 1) / (total > 0 ? total : 1), parts = want < 1 ? 1 : want > steps ? steps : want;
  const int each = (int)((steps + parts - 1) / parts);
  return (steps + each - 1) / each;  // none of them empty
}

template <int D, bool CACHE>
int launch_rope(RopeParams &p, bool next, cudaStream_t stream) {
  constexpr int kHeads = RowCfg<D>::kHeads, kBlocks = 152 * kFwdBlocks;
  const int steps = (p.q.heads + kHeads - 1) / kHeads + (CACHE ? 2 : 1) * ((p.k.heads + kHeads - 1) / kHeads);
  p.parts = parts_for(p.total, steps, kBlocks * kFwdWarps);
  const long long blocks = ((long long)p.total * p.parts + kFwdWarps - 1) / kFwdWarps;
  return launch_after(next ? rope_kernel<D, true, CACHE> : rope_kernel<D, false, CACHE>, blocks < kBlocks ? blocks : kBlocks, 1,
                      32 * kFwdWarps, 0, stream, p);
}
template <bool CACHE>
int launch_rope(RopeParams &p, int d, bool next, cudaStream_t stream) {
  return d == 64 ? launch_rope<64, CACHE>(p, next, stream)
                 : d == 128 ? launch_rope<128, CACHE>(p, next, stream) : launch_rope<256, CACHE>(p, next, stream);
}

template <int D>
int launch_bwd(RopeParams &p, bool next, int *blocks, cudaStream_t stream) {
  constexpr int kHeads = RowCfg<D>::kHeads, kSmem = kBwdWarps * kRing * sizeof(BwdStage<D>);
  auto steps = [](int heads) { return (heads + kHeads - 1) / kHeads; };
  const long long sq = steps(p.gq.heads), sk = steps(p.gk.heads), all = (sq + sk) * p.total;
  // as many blocks as run at once, or one for every kBwdWarps * 2 steps
  const long long want = all / (2 * kBwdWarps) + 2;
  *blocks = want < kBwdBlocks ? (int)want : kBwdBlocks;
  p.q_blocks = (int)((*blocks * sq + (sq + sk) / 2) / (sq + sk));
  p.q_blocks = p.q_blocks < 1 ? 1 : p.q_blocks < *blocks ? p.q_blocks : *blocks - 1;
  p.parts = parts_for(p.total, (int)sq, p.q_blocks * kBwdWarps);
  p.k_parts = parts_for(p.total, (int)sk, (*blocks - p.q_blocks) * kBwdWarps);
  void (*kernel)(RopeParams) = next ? rope_bwd_kernel<D, true> : rope_bwd_kernel<D, false>;
  // on every launch: the attribute belongs to the function on the current device
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess) return FA_ERR_CUDA;
  return launch_after(kernel, *blocks, 1, 32 * kBwdWarps, kSmem, stream, p);
}

size_t bwd_bytes(int d) { return (size_t)kBwdBlocks * d * 4; }

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
  int blocks = 1;
  const bool next = interleaved != 0;
  rc = d == 64 ? launch_bwd<64>(p, next, &blocks, s) : d == 128 ? launch_bwd<128>(p, next, &blocks, s) : launch_bwd<256>(p, next, &blocks, s);
  if (rc != FA_OK || !norm) return rc;
  return launch_after(rope_dw_kernel, 2 * d / 32, 1, 1024, 0, s, (const float *)p.part, p.q_blocks, blocks, d,
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
  if ((total > 0 && (!q || !k || !v || !q_out)) || k_pages == v_pages) return FA_ERR_INVALID_ARG;
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
