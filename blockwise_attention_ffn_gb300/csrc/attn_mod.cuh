// attn_mod.cuh -- what the modified attention's kernels share: the key window
// of a query row, the capped score and the distance bias.
//
//   score of query i and key j:  y = C tanh(x / C) - a |i - j|,  x = q.k / sqrt(d)
//   (C the cap, or y = x - a |i - j| without one), visible iff
//   lo_i <= j < hi_i; everything below is in units of log 2: y log2(e).
//
// The cap's cost.  tanh through an exponential and a reciprocal takes two more
// special-function operations per score beside the softmax's own, and those
// units already bound the softmax.  Trained scores sit well inside the cap, so
// wherever every score of a warp's tile has |x| <= 0.6 C an odd polynomial of
// degree 9 in x / C is taken instead (error 2.8e-8, below fp32's own at the
// scores' size), at half the arithmetic rate of fp32 pairs and no special
// function; the exact form serves every other tile.
#pragma once

#include "attn_common.cuh"

namespace bpt {

// Window of query row q (index in its sequence) of sequence bi: the given
// begin and end, clamped to the sequence, and the causal limit; empty (0, 0)
// where nothing is visible and for rows past the sequence.
__device__ __forceinline__ int2 key_window(const int32_t* row_begin, const int32_t* row_end, int causal, int s, int bi,
                                           int q) {
  if (q >= s) return make_int2(0, 0);
  const long long at = (long long)bi * s + q;
  int lo = row_begin ? max(row_begin[at], 0) : 0;
  int hi = row_end ? min(row_end[at], s) : s;
  if (causal) hi = min(hi, q + 1);
  return lo < hi ? make_int2(lo, hi) : make_int2(0, 0);
}

// tanh for |y| <= 0.6, two at a time: y (1 + u (c1 + u (c2 + u (c3 + u c4)))),
// u = y^2, a least-maximum fit of the odd polynomial of degree 9
__device__ __forceinline__ uint64_t tanh2_small(uint64_t y) {
  const uint64_t u = mul2(y, y);
  uint64_t q = fma2(u, f2(0.01531921f, 0.01531921f), f2(-0.05199434f, -0.05199434f));
  q = fma2(u, q, f2(0.13308098f, 0.13308098f));
  q = fma2(u, q, f2(-0.33332248f, -0.33332248f));
  return fma2(mul2(u, q), y, y);
}
constexpr float TANH_SMALL = 0.6f;

// tanh(y) = 1 - 2 / (1 + e^(2y)): absolute error about 2^-23, saturating
// exactly; y2 = 2 log2(e) y
__device__ __forceinline__ float tanh_any(float y2) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2(y2)));
  return fmaf(-2.f, r, 1.f);
}

// largest |v| of N values (NaN ignored)
template <int N>
__device__ __forceinline__ float amax_of(const uint32_t (&v)[N]) {
  float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < N; i += 2)
    m[(i >> 1) & 3] = max3f(m[(i >> 1) & 3], fabsf(__uint_as_float(v[i])), fabsf(__uint_as_float(v[i + 1])));
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// The bias -a |i - j| along a run of 64 consecutive indices from `first`
// against the fixed index `self`, as base + k * step for k = 0..63, unless
// the run passes `self` strictly inside (mixed).  below_only: indices above
// `self` are masked anyway; above_only: those below.
struct BiasLine {
  float base, step;
  bool mixed;
};
__device__ __forceinline__ BiasLine bias_line(float slope2, int self, int first, bool below_only, bool above_only) {
  BiasLine b;
  const int dist = self - first;  // > 0: the run starts below self
  const bool below = !above_only && dist >= (below_only ? 1 : 63);
  b.mixed = dist > 0 && !below && !above_only;
  b.base = below ? -slope2 * (float)dist : slope2 * (float)dist;
  b.step = below ? slope2 : -slope2;
  return b;
}

}  // namespace bpt
