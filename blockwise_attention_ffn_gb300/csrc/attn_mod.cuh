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
// a warp whose 64 columns all have |x| <= C/4 takes an odd polynomial of
// degree 5 in x (error 8e-8 C, below an fp32 step of the largest of them),
// within 0.6 C one of degree 9 (3e-8 C), both in packed fp32 arithmetic.  Only
// beyond that the exponential is taken, with an error of 2^-23 C.  Up to C = 64 that
// is 2^-17, below what a probability's rounding to bf16 leaves of it by far; under a
// larger cap it would swamp the warp's small scores, which then keep the first
// polynomial, element by element (at C = 50 that would cost rows of saturated scores,
// 8192 x (32 + 8 + 8) heads of 128, causal, 900 us against 790 forward and 2,260
// against 1,850 backward).
#pragma once

#include <float.h>
#include <math.h>
#include <string.h>

#include <algorithm>

#include "attn_common.cuh"

namespace bpt {

// Window of query row q (index in its sequence) of sequence bi: the given
// begin and end, clamped to the sequence, and the causal limit; empty (0, 0)
// where nothing is visible and for rows past the sequence.  In two steps, so
// that a kernel can read a window long before it needs it.
__device__ __forceinline__ int2 raw_window(const int32_t* row_begin, const int32_t* row_end, int s, int bi, int q) {
  const long long at = (long long)bi * s + q;
  return make_int2(row_begin && q < s ? row_begin[at] : 0, row_end && q < s ? row_end[at] : s);
}
__device__ __forceinline__ int2 clamped_window(int2 raw, int causal, int s, int q) {
  const int lo = max(raw.x, 0), hi = causal ? min(min(raw.y, s), q + 1) : min(raw.y, s);
  return q < s && lo < hi ? make_int2(lo, hi) : make_int2(0, 0);
}
__device__ __forceinline__ int2 key_window(const int32_t* row_begin, const int32_t* row_end, int causal, int s, int bi,
                                           int q) {
  return clamped_window(raw_window(row_begin, row_end, s, bi, q), causal, s, q);
}

// The cap as the kernels take it: with z a raw score (q.k), x = z / sqrt(d)
// and k = 1 / (C sqrt(d)), the polynomials of tanh(k z), least-maximum fits,
// in powers of z: z (c[0] + w (c[1] + w c[2])) for |k z| <= 0.25 and
// z (e[0] + w (e[1] + ... )) for |k z| <= 0.6, w = z^2, each times `out`.
struct CapCoef {
  float near1, near2;  // largest |z| of the two (near2 = near1: the second is not taken)
  uint64_t c[3], e[5];  // the coefficients, twice each: operands of packed arithmetic
  float k2, out;        // 2 log2(e) k, and what tanh is multiplied with
  int large;            // cap above 64
};
inline uint64_t twice(float v) {
  uint32_t u;
  memcpy(&u, &v, 4);
  return (uint64_t)u << 32 | u;
}
inline CapCoef cap_coef(double cap, double k, double out) {
  const double n5[3] = {1.0, -0.33322915, 0.128460431};
  const double n9[5] = {1.0, -0.33332248, 0.133080983, -0.0519943379, 0.0153192074};
  CapCoef f;
  f.near1 = (float)(0.25 / k);
  f.near2 = (float)(0.6 / k);
  double kk = k * out, least = INFINITY;
  for (int i = 0; i < 5; ++i, kk *= k * k) {
    if (i < 3) f.c[i] = twice((float)(n5[i] * kk));
    f.e[i] = twice((float)(n9[i] * kk));
    least = std::min(least, fabs(n9[i] * kk));
  }
  f.k2 = (float)(2.8853900817779268 * k);
  f.out = (float)out;
  f.large = cap > 64.0;
  // Under a large cap the powers of k leave fp32 (from C = 917 at d = 128 where
  // out = 1; caps of up to 2^20 leave the first polynomial's within it): lost terms
  // would be wrong scores, so the exact form takes the second one's range.
  if (least < FLT_MIN) f.near2 = f.near1;
  return f;
}
__device__ __forceinline__ uint64_t both(float v) { return f2(v, v); }
__device__ __forceinline__ uint64_t near1_factor(const CapCoef& f, uint64_t z) {
  const uint64_t w = mul2(z, z);
  return fma2(w, fma2(w, f.c[2], f.c[1]), f.c[0]);
}
__device__ __forceinline__ uint64_t near2_factor(const CapCoef& f, uint64_t z) {
  const uint64_t w = mul2(z, z);
  uint64_t q = fma2(w, f.e[4], f.e[3]);
  q = fma2(w, q, f.e[2]);
  q = fma2(w, q, f.e[1]);
  return fma2(w, q, f.e[0]);
}
__device__ __forceinline__ uint64_t cap_near1(const CapCoef& f, uint64_t z) { return mul2(z, near1_factor(f, z)); }
__device__ __forceinline__ uint64_t cap_near2(const CapCoef& f, uint64_t z) { return mul2(z, near2_factor(f, z)); }

// tanh(y) = 1 - 2 / (1 + e^(2y)): absolute error about 2^-23, saturating
// exactly; y2 = 2 log2(e) y
__device__ __forceinline__ float tanh_any(float y2) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2(y2)));
  return fmaf(-2.f, r, 1.f);
}
// the capped scores of a pair beyond the polynomials' ranges, and under a large cap
__device__ __forceinline__ uint64_t cap_far(const CapCoef& f, uint64_t z) {
  const float2 v = f2split(z);
  return f2(tanh_any(v.x * f.k2) * f.out, tanh_any(v.y * f.k2) * f.out);
}
__device__ __forceinline__ uint64_t cap_far_large(const CapCoef& f, uint64_t z) {
  const float2 v = f2split(z), near = f2split(cap_near1(f, z)), far = f2split(cap_far(f, z));
  return f2(fabsf(v.x) <= f.near1 ? near.x : far.x, fabsf(v.y) <= f.near1 ? near.y : far.y);
}

// The order of the grid: work items of tiles x heads, the tiles of all heads
// of a group in turn, first tile index first, then the next group, so that a
// group's last, small items balance its large first ones.  A group is as many
// key/value heads (of any sequence) as L2 holds the streams of, or 16: then
// some ten CTAs still share a head's stream as they go.
struct ItemOrder {
  int tiles, per_head, group, kv_heads;  // group: key/value heads in one; kv_heads: b * H_kv
};
struct Item {
  int tile, kv, sub;  // kv: index of the key/value head over all sequences; sub < per_head
};
inline ItemOrder item_order(int64_t tiles, int64_t per_head, int64_t kv_heads, int64_t bytes_per_head) {
  const int64_t fit = std::max<int64_t>(16, (48 << 20) / std::max<int64_t>(1, bytes_per_head));
  ItemOrder o;
  o.tiles = (int)tiles;
  o.per_head = (int)per_head;
  o.kv_heads = (int)kv_heads;
  o.group = (int)std::min(fit, kv_heads);
  return o;
}
__device__ __forceinline__ Item item_of(const ItemOrder& o, int block) {
  const int full = o.group * o.per_head * o.tiles;
  const int g = block / full;
  const int rem = block - g * full;
  const int heads = min(o.group, o.kv_heads - g * o.group) * o.per_head;
  const int head = rem % heads;
  return Item{rem / heads, g * o.group + head / o.per_head, head % o.per_head};
}

// A place in a ring of N and the parity of the round, counted up instead of
// divided: the issuing warps' loops feel every instruction (a remainder by 3 or 5
// in them cost the forward up to a third).
template <int N>
struct RingPos {
  int at = 0;
  uint32_t round = 0;
  __device__ __forceinline__ RingPos next() const {
    RingPos r;
    r.at = at + 1 == N ? 0 : at + 1;
    r.round = at + 1 == N ? round ^ 1 : round;
    return r;
  }
};

// One work item as the scheduling warp of a persistent CTA publishes it; n < 0:
// no more.
struct WorkItem {
  int n, bi, q0, j0, nkv;  // query head, sequence, first row, first key tile, key tiles
};
constexpr int WORK_BYTES = 2 * 16 + 2 * 32;  // two answers, two items
struct WorkQueue {
  uint8_t* mem;          // WORK_BYTES, 16-byte aligned
  uint64_t* full;        // [2], count 1
  uint64_t* empty;       // [2], one arrival per reading warp
  uint64_t* answered;    // count 1
  __device__ __forceinline__ volatile WorkItem* item(int it) const {
    return reinterpret_cast<volatile WorkItem*>(mem + 32 + 32 * (it & 1));
  }
};
// The scheduling warp: publishes describe(block) for this CTA's block and then
// for the blocks it takes over, the next one asked for when every warp has
// begun the current one and the loading warp is through with it: a CTA that
// took an item earlier would hold it back from the others (more = false: no
// further one is asked for).  published(it, item) follows each.  Returns whether
// `last` was among them.
template <class Describe, class Published>
__device__ __forceinline__ bool publish_items(const WorkQueue& q, int block, int last, bool more,
                                              volatile int* abort_flag, unsigned int* err, Describe describe,
                                              Published published) {
  const int lane = lane_id();
  bool asked = false, took_last = false;
  int it = 0;
  while (true) {
    if (block < 0) {
      if (lane == 0) {
        q.item(it)->n = -1;
        mbar_arrive(&q.full[it & 1]);
      }
      break;
    }
    took_last |= block == last;
    const WorkItem w = describe(block);
    if (lane == 0) {
      volatile WorkItem* to = q.item(it);
      to->n = w.n;
      to->bi = w.bi;
      to->q0 = w.q0;
      to->j0 = w.j0;
      to->nkv = w.nkv;
      mbar_arrive(&q.full[it & 1]);
    }
    if (!published(it, w)) break;
    if (!bounded_wait_w(&q.empty[it & 1], (it >> 1) & 1, abort_flag, 252, err)) break;
    block = -1;
    if (more) {
      uint8_t* answer = q.mem + 16 * (it & 1);
      if (lane == 0) request_block(answer, q.answered);
      asked = true;
      if (!bounded_wait_w(q.answered, it & 1, abort_flag, 257, err)) break;
      asked = false;
      block = answered_block(answer);
      fence_proxy_async_smem();
      __syncwarp();
    }
    ++it;
  }
  // a request in flight lands before the shared memory goes
  if (asked) drain_wait(q.answered, it & 1);
  return took_last;
}
__device__ __forceinline__ void release_item(const WorkQueue& q, int it) {
  __syncwarp();
  if (lane_id() == 0) mbar_arrive(&q.empty[it & 1]);
}
// A reading warp's copy of item it; false after a timeout.  The loading warp
// (keep) releases it itself.
template <bool keep = false>
__device__ __forceinline__ bool next_item(const WorkQueue& q, int it, WorkItem* w, volatile int* abort_flag,
                                          unsigned int* err) {
  if (!bounded_wait_w(&q.full[it & 1], (it >> 1) & 1, abort_flag, 250, err)) return false;
  volatile WorkItem* from = q.item(it);
  *w = WorkItem{from->n, from->bi, from->q0, from->j0, from->nkv};
  if (!keep) release_item(q, it);
  return true;
}

// 64 score columns of this thread's row, and the largest of them (of their
// magnitudes: ABS), which the load itself finds
template <bool ABS>
__device__ __forceinline__ float load_scores(uint32_t taddr, uint32_t (&sv)[64]) {
  float a, b;
  if constexpr (ABS) {
    tmem_ld32_amax_nw(taddr, sv, a);
    tmem_ld32_amax_nw(taddr + 32, sv + 32, b);
  } else {
    tmem_ld32_max_nw(taddr, sv, a);
    tmem_ld32_max_nw(taddr + 32, sv + 32, b);
  }
  tmem_wait_ld(sv);
  tmem_wait_max(a);
  tmem_wait_max(b);
  return fmaxf(a, b);
}

// the largest magnitude of the columns that on(i) says, NaN left out
template <class On>
__device__ __forceinline__ float largest_of(const uint32_t (&sv)[64], On on) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 64; ++i)
    if (on(i)) m = fmaxf(m, fabsf(__uint_as_float(sv[i])));
  return m;
}
// of the columns [lo, hi), lo < hi
__device__ __forceinline__ float largest_within(const uint32_t (&sv)[64], int lo, int hi) {
  const uint64_t bits = lo < hi ? ~0ull << lo & ~0ull >> (64 - hi) : 0ull;
  const uint32_t b0 = (uint32_t)bits, b1 = (uint32_t)(bits >> 32);
  return largest_of(sv, [&](int i) { return ((i < 32 ? b0 >> i : b1 >> (i - 32)) & 1u) != 0u; });
}

// The bias -a |i - j| along a run of n consecutive indices from `first`
// against the fixed index `self`, as base + k * step for k < n, unless
// the run passes `self` strictly inside (mixed).  below_only: indices above
// `self` are masked anyway; above_only: those below.
struct BiasLine {
  float base, step;
  bool mixed;
};
// (k, k + 1) as fp32 for even k < 64: operands of packed arithmetic
#define BPT_PAIRS8(k) {k, k + 1}, {k + 2, k + 3}, {k + 4, k + 5}, {k + 6, k + 7}
static __constant__ float2 index_pairs[32] = {BPT_PAIRS8(0.f),  BPT_PAIRS8(8.f),  BPT_PAIRS8(16.f), BPT_PAIRS8(24.f),
                                              BPT_PAIRS8(32.f), BPT_PAIRS8(40.f), BPT_PAIRS8(48.f), BPT_PAIRS8(56.f)};
#undef BPT_PAIRS8
// base + k * step of the pair (k, k + 1)
__device__ __forceinline__ uint64_t on_line(int k, uint64_t step2, uint64_t base2) {
  const float2 i = index_pairs[k / 2];
  return fma2(f2(i.x, i.y), step2, base2);
}
__device__ __forceinline__ BiasLine bias_line(float slope2, int self, int first, int n, bool below_only, bool above_only) {
  BiasLine b;
  const int dist = self - first;  // > 0: the run starts below self
  const bool below = !above_only && dist >= (below_only ? 1 : n - 1);
  b.mixed = dist > 0 && !below && !above_only;
  b.base = below ? -slope2 * (float)dist : slope2 * (float)dist;
  b.step = below ? slope2 : -slope2;
  return b;
}

}  // namespace bpt
