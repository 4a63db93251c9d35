// moe_few.cu -- the experts' network for a few new tokens (serving): so few
// rows that every expert's matrices meet about one of them.
//
// Bound by the weights' bytes: 3 h f values for each chosen expert, one
// multiply each.  Tensor-core tiles gain nothing there, and a tile's set-up
// (barriers, tensor memory, the groups' lists) costs more than its products, so
// the rows go one by one through plain loads: a warp holds a few rows of W at a
// time, 16 bytes a lane, many loads in flight, fp32 throughout.  The second
// product adds a position's k experts in its registers: no rows in between, no
// pass to add them, and the activation stays fp32.
//   one token, 4 of 64 experts of 2048 x 1024 (50 MB, 7.4 us of HBM time):
//   18.5 us in two launches against 29.6 in the grouped GEMM's three.
// Weights that two rows share are read twice, the second time from L2, and long
// streams go faster by TMA: taken up to a quarter as many rows as experts and
// 256 MB (moe_few_rows).  us here and through the grouped GEMM: 64 experts of
// 2048 x 1024, 4 pairs 17 and 25, 16 pairs (201 MB) 42 and 46, 32 pairs 77 and
// 68; 128 of 2560 x 2048, 4 pairs 28 and 43, 16 pairs (503 MB) 92 and 99; 64 of
// 4096 x 2048, 8 pairs (403 MB) 81 and 80; 16 of 4096 x 8192, 2 pairs 85 and 74.
#include <math.h>

#include <algorithm>

#include "../../include/bpt.h"
#include "grouped.h"
#include "internal.h"
#include "moe.h"
#include "ptx.cuh"

namespace bpt {

namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32;

struct FewParams {
  const __nv_bfloat16 *x, *w1, *w3, *w2;
  const int *offsets, *order, *slot;
  const void* weight;
  int weight_f32;
  float* act;  // [pairs, f]
  __nv_bfloat16* y;
  int h, f, E, k, pairs, kind;
  unsigned int* err;
};

// The expert of row r of the order (E: none) into *s, by all threads of the
// block, where no offsets are bad; whether this thread saw bad ones.
__device__ __forceinline__ bool find_expert(const FewParams& p, int r, int* s) {
  bool bad = false;
  for (int e = threadIdx.x; e < p.E; e += THREADS) {
    const int lo = p.offsets[e], hi = p.offsets[e + 1];
    if (bad_offsets(lo, hi, p.pairs)) {
      if (blockIdx.x == 0) report_bad_data(p.err, BPT_GROUPED_BAD_OFFSET_SITE);
      bad = true;
    } else if (r >= lo && r < hi) {
      atomicMin(s, e);
    }
  }
  return bad;
}

__device__ __forceinline__ uint4 load16(const __nv_bfloat16* p, bool in) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (in) asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ float dot8(const uint4& w, const float (&x)[8], float s) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s = fmaf(bf16_lo(u[i]), x[2 * i], s);
    s = fmaf(bf16_hi(u[i]), x[2 * i + 1], s);
  }
  return s;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// act[r, i] of row r of the order for 4 rows of weights a warp: two units with
// gate and up (SwiGLU), or four.
constexpr int STEP = 4;  // blocks of 256 columns whose loads are in flight
template <bool GATED>
__global__ void __launch_bounds__(THREADS) few_act_kernel(const FewParams p) {
  __shared__ int s_e;
  constexpr int UNITS = GATED ? 2 : 4;
  const int lane = lane_id();
  const int chunks = (p.f + WARPS * UNITS - 1) / (WARPS * UNITS);
  const int r = blockIdx.x / chunks;
  const int i0 = ((int)(blockIdx.x % chunks) * WARPS + warp_id()) * UNITS;
  if (threadIdx.x == 0) s_e = p.E;
  wait_for_previous();
  let_next_start();
  const int pair = p.order[r];
  __syncthreads();
  if (__syncthreads_or(find_expert(p, r, &s_e))) {
    if (threadIdx.x == 0) s_e = group_of(p.offsets, p.E, p.pairs, r);
    __syncthreads();
  }
  const int e = s_e;
  if (e == p.E || i0 >= p.f) return;  // f is a multiple of 8: a warp's units are all there or none
  const bool some = pair >= 0 && pair < p.pairs;
  const __nv_bfloat16* x = p.x + (int64_t)(some ? pair / p.k : 0) * p.h;
  const __nv_bfloat16* w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t at = ((int64_t)e * p.f + i0 + (GATED ? q >> 1 : q)) * p.h;
    w[q] = (GATED && (q & 1) ? p.w3 : p.w1) + at;
  }
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  for (int c0 = lane * 8; c0 < p.h; c0 += 256 * STEP) {
    uint4 xv[STEP], wv[STEP][4];
#pragma unroll
    for (int t = 0; t < STEP; ++t) {
      const int c = c0 + 256 * t;
      const bool in = c < p.h;
#pragma unroll
      for (int q = 0; q < 4; ++q) wv[t][q] = load16(w[q] + c, in);
      xv[t] = in && some ? *reinterpret_cast<const uint4*>(x + c) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int t = 0; t < STEP; ++t) {
      const uint32_t u[4] = {xv[t].x, xv[t].y, xv[t].z, xv[t].w};
      float v[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(u[i]), v[2 * i + 1] = bf16_hi(u[i]);
#pragma unroll
      for (int q = 0; q < 4; ++q) s[q] = dot8(wv[t][q], v, s[q]);
    }
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) s[q] = warp_sum(s[q]);
  if (lane < UNITS) {
    float a;
    if constexpr (GATED) {
      const float g = lane ? s[2] : s[0], u = lane ? s[3] : s[1];
      a = g / (1.f + expf(-g)) * u;
    } else {
      const float z = lane == 0 ? s[0] : lane == 1 ? s[1] : lane == 2 ? s[2] : s[3];
      const float c = 0.7978845608028654f;
      a = p.kind == BPT_ACT_GELU_ERF ? 0.5f * z * (1.f + erff(z * 0.70710678118654752f))
                                     : 0.5f * z * (1.f + tanhf(c * (z + 0.044715f * z * z * z)));
    }
    p.act[(int64_t)r * p.f + i0 + lane] = a;
  }
}

// y[t, i] = sum_j w_tj <act of pair (t, j), W2_e[i, :]>: two i a group of JS
// warps, which share the choices out and add their sums in order.  (One warp for
// all of four choices is four round trips to memory in a row.)
constexpr int MAX_TOP_K = 32;
template <int JS>
__global__ void __launch_bounds__(THREADS) few_out_kernel(const FewParams p) {
  constexpr int PAIRS = WARPS / JS;  // row pairs of W2 a block
  __shared__ int s_e[MAX_TOP_K];
  __shared__ float s_sum[WARPS][2];
  const int lane = lane_id(), js = warp_id() % JS;
  const int chunks = (p.h + PAIRS * 2 - 1) / (PAIRS * 2);
  const int t = blockIdx.x / chunks;
  const int i0 = ((int)(blockIdx.x % chunks) * PAIRS + warp_id() / JS) * 2;
  const bool in = i0 < p.h;  // h is even
  if (threadIdx.x < MAX_TOP_K) s_e[threadIdx.x] = p.E;
  // the routes are older than the activations: the kernel before has waited
  // for them before it let this one start
  __syncthreads();
  bool bad = false;
  for (int j = 0; j < p.k; ++j) {
    const int r = p.slot[t * p.k + j];
    if (r >= 0 && r < p.pairs) bad |= find_expert(p, r, &s_e[j]);
  }
  if (__syncthreads_or(bad)) {
    if ((int)threadIdx.x < p.k) s_e[threadIdx.x] = group_of(p.offsets, p.E, p.pairs, p.slot[t * p.k + threadIdx.x]);
    __syncthreads();
  }
  if (in)
    for (int j = js; j < p.k; j += JS)
      if (s_e[j] < p.E)  // on their way to L2 meanwhile
#pragma unroll
        for (int q = 0; q < 2; ++q)
          for (int c = lane * 64; c < p.f; c += 2048)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p.w2 + ((int64_t)s_e[j] * p.h + i0 + q) * p.f + c));
  wait_for_previous();
  let_next_start();
  float s[2] = {0.f, 0.f};
  if (in)
    for (int j = js; j < p.k; j += JS) {
      const int e = s_e[j];
      if (e == p.E) continue;
      const int64_t q = (int64_t)t * p.k + j;
      const float weight = p.weight_f32 ? reinterpret_cast<const float*>(p.weight)[q]
                                        : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.weight)[q]);
      const float* a = p.act + (int64_t)p.slot[q] * p.f;
      const __nv_bfloat16* w0 = p.w2 + ((int64_t)e * p.h + i0) * p.f;
      float d[2] = {0.f, 0.f};
      for (int c0 = lane * 8; c0 < p.f; c0 += 256 * STEP) {
        uint4 wv[STEP][2];
        float4 av[STEP][2];
#pragma unroll
        for (int u = 0; u < STEP; ++u) {
          const int c = c0 + 256 * u;
          const bool some = c < p.f;
          wv[u][0] = load16(w0 + c, some);
          wv[u][1] = load16(w0 + p.f + c, some);
#pragma unroll
          for (int i = 0; i < 2; ++i) av[u][i] = some ? reinterpret_cast<const float4*>(a + c)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int u = 0; u < STEP; ++u) {
          const float v[8] = {av[u][0].x, av[u][0].y, av[u][0].z, av[u][0].w, av[u][1].x, av[u][1].y, av[u][1].z, av[u][1].w};
          d[0] = dot8(wv[u][0], v, d[0]);
          d[1] = dot8(wv[u][1], v, d[1]);
        }
      }
      s[0] = fmaf(weight, d[0], s[0]);
      s[1] = fmaf(weight, d[1], s[1]);
    }
  s[0] = warp_sum(s[0]);
  s[1] = warp_sum(s[1]);
  if constexpr (JS > 1) {
    if (lane < 2) s_sum[warp_id()][lane] = lane ? s[1] : s[0];
    __syncthreads();
    if (js) return;
#pragma unroll
    for (int q = 1; q < JS; ++q) {
      s[0] += s_sum[warp_id() + q][0];
      s[1] += s_sum[warp_id() + q][1];
    }
  }
  if (in && lane == 0) *reinterpret_cast<uint32_t*>(p.y + (int64_t)t * p.h + i0) = pack_bf16(s[0], s[1]);
}

}  // namespace

bool moe_few_rows(const MoeDims& D) {
  const int64_t mats = D.act == BPT_ACT_SWIGLU ? 3 : 2;
  return 4 * D.pairs <= D.E && 2 * D.pairs * mats * D.h * D.f <= (int64_t(256) << 20);
}
size_t moe_few_ws_bytes(const MoeDims& D) { return (size_t)D.pairs * D.f * 4; }

int moe_few_fwd(const MoeDims& D, const bpt_moe_route* r, const void* x, const void* w1, const void* w3, const void* w2, void* y, void* ws,
                cudaStream_t st) {
  FewParams p;
  p.x = reinterpret_cast<const __nv_bfloat16*>(x);
  p.w1 = reinterpret_cast<const __nv_bfloat16*>(w1);
  p.w3 = reinterpret_cast<const __nv_bfloat16*>(w3);
  p.w2 = reinterpret_cast<const __nv_bfloat16*>(w2);
  p.offsets = r->offsets;
  p.order = r->order;
  p.slot = r->slot;
  p.weight = r->weights;
  p.weight_f32 = D.weight_bytes == 4;
  p.act = reinterpret_cast<float*>(ws);
  p.y = reinterpret_cast<__nv_bfloat16*>(y);
  p.h = (int)D.h;
  p.f = (int)D.f;
  p.E = (int)D.E;
  p.k = (int)D.k;
  p.pairs = (int)D.pairs;
  p.kind = D.act;
  p.err = device_error_word();
  if (!p.err) return BPT_ECUDA;
  const bool gated = D.act == BPT_ACT_SWIGLU;
  const int64_t mats = gated ? 3 : 2;
  ProfScope prof(PROF_MISC, 0.0, 2.0 * (double)(D.pairs * mats * D.h * D.f), st);
  const int64_t per = WARPS * (gated ? 2 : 4);
  const int js = D.k >= 4 ? 4 : D.k >= 2 ? 2 : 1;
  const int64_t g1 = D.pairs * ((D.f + per - 1) / per), g2 = D.n * ((D.h + WARPS / js * 2 - 1) / (WARPS / js * 2));
  if (g1 > INT32_MAX || g2 > INT32_MAX) return BPT_EUNSUPPORTED;
  if (launch_dependent(gated ? few_act_kernel<true> : few_act_kernel<false>, (int)g1, 1, dim3(THREADS), 0, st, p) != cudaSuccess)
    return BPT_ECUDA;
  auto out = js == 4 ? few_out_kernel<4> : js == 2 ? few_out_kernel<2> : few_out_kernel<1>;
  return launch_dependent(out, (int)g2, 1, dim3(THREADS), 0, st, p) == cudaSuccess ? BPT_OK : BPT_ECUDA;
}

}  // namespace bpt
