// moe_route.cu -- the router of a mixture-of-experts layer: from the logits of
// every position, its top-k experts, their weights, the order that groups the
// (position, choice) pairs by expert, the balance and z losses, and the
// gradient of the logits.
//
//   p = softmax(z) over the E experts of a row, chosen: the k largest z
//   weights = p at the chosen, or (norm_topk) the softmax over the chosen
//   loss = balance E / (nv k) sum_e count_e mean_t p_te + z_coef mean_t lse_t^2
//
// Memory-bound on paper and bound by latency in fact: 8 MB of logits at
// n = 32768, E = 64 are 1.3 us of HBM time, less than a launch.  So: few
// launches (one for few rows, two else: choosing with counts per block, then
// placing), a row held by G lanes in registers for the whole of the choice and
// the softmax, and every sum in a fixed order.  At that size 15 us choosing, 12
// placing, 10 backward; 35 us for forward and backward in a stream of calls.
#include <math.h>

#include <algorithm>

#include "../../include/bpt.h"
#include "internal.h"
#include "moe.h"
#include "ptx.cuh"

namespace bpt {

namespace {

// Threads a block: 1024 where the registers suffice.  A row's choice is a chain
// of k dependent steps, so the time is that of the rows a warp does in turn: at
// n = 32768, E = 64, k = 6 choosing and placing took 41 and 20 us with 256
// threads in 152 blocks.
constexpr int BWD_THREADS = 256;
constexpr int MAX_BLOCKS = 152;  // of rows: one on each SM
template <int V>
constexpr int choose_threads() {
  return V == 8 ? 1024 : V == 16 ? 512 : 256;
}

struct RouteParams {
  const void* logits;
  int logits_bf16, weights_bf16;
  int64_t n;
  int E, k, norm;
  float balance, zc;
  int32_t *ids, *offsets, *order, *slot;
  void* weights;
  float* loss;
  // per block of rows: rows of each expert, sums of probabilities, of lse^2, routed rows
  int* hist;
  float* psum;
  float* zsum;
  int* live;
  int nblk;
  int64_t per;  // rows a block
  unsigned int* err;
};

// rises with v, equal for equal values; 0: not to be chosen
__device__ __forceinline__ uint32_t sort_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);  // -0 becomes +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// e^x with a relative error of 2^-22 and |x| 2^-24
__device__ __forceinline__ float exp_of(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
  return r;
}

// V consecutive logits from column c of a row (past E: -inf)
template <int V>
__device__ __forceinline__ void load_logits(const void* z, int bf16, int64_t row, int E, int c, float (&v)[V], unsigned int* err) {
  if (c + V <= E && (E & 7) == 0) {
    // whole 16-byte words: rows are multiples of 8 values
#pragma unroll
    for (int i = 0; i < V; i += 8) {
      if (bf16) {
        const uint4 u = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(z) + row * E + c + i);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[i + 2 * j] = bf16_lo(w[j]);
          v[i + 2 * j + 1] = bf16_hi(w[j]);
        }
      } else {
        const float4* q = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(z) + row * E + c + i);
        const float4 a = q[0], b = q[1];
        v[i] = a.x, v[i + 1] = a.y, v[i + 2] = a.z, v[i + 3] = a.w;
        v[i + 4] = b.x, v[i + 5] = b.y, v[i + 6] = b.z, v[i + 7] = b.w;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      v[i] = c + i >= E ? -INFINITY
             : bf16     ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(z)[row * E + c + i])
                        : reinterpret_cast<const float*>(z)[row * E + c + i];
  }
  // a NaN or +inf is recorded and cannot be chosen
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (!(v[i] < INFINITY)) {
      if (err) report_bad_data(err, BPT_MOE_BAD_LOGIT_SITE);
      v[i] = -INFINITY;
    }
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int d = 1; d < G; d <<= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int d = 1; d < G; d <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
  return v;
}

// Rows [r0, r1) of one block: their choice, weights and the block's sums.
// G lanes hold a row, V = 8 or more consecutive logits each.
template <int G, int V, int THREADS>
__device__ void choose_rows(const RouteParams& p, int64_t r0, int64_t r1, int b, int* s_hist, float* s_sum) {
  const int lane = lane_id(), warp = warp_id();
  const int sub = lane % G, c = sub * V;
  constexpr int ROWS = 32 / G;  // rows a warp holds at once
  constexpr int WARPS = THREADS / 32;
  for (int e = threadIdx.x; e < p.E; e += THREADS) s_hist[e] = 0;
  __syncthreads();
  const bool sums = p.balance != 0.f, zsums = p.zc != 0.f;
  float acc[V], zacc = 0.f;
  int live = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  for (int64_t base = r0 + warp * ROWS; base < r1; base += WARPS * ROWS) {
    const int64_t row = base + lane / G;
    const bool in = row < r1;
    float v[V];
    if (in) {
      load_logits<V>(p.logits, p.logits_bf16, row, p.E, c, v, p.err);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = -INFINITY;
    }
    uint32_t key[V];  // 0: taken, or not to be chosen
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = v[i] > -INFINITY ? sort_key(v[i]) : 0u;
    float m = 0.f, total = 0.f, inv = 0.f, top_sum = 0.f, mine = 0.f, first = 0.f;
    for (int j = 0; j < p.k; ++j) {
      // the largest key left; of equals the first lane's, and its first
      uint32_t best = key[0];
#pragma unroll
      for (int i = 1; i < V; ++i) best = max(best, key[i]);
      const uint32_t own = best;
      if constexpr (G == 32) {
        best = __reduce_max_sync(0xffffffffu, best);
      } else {
#pragma unroll
        for (int d = 1; d < G; d <<= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, d));
      }
      int at = 0;
#pragma unroll
      for (int i = V - 1; i >= 0; --i) at = key[i] == best ? i : at;
      const uint32_t holds = __ballot_sync(0xffffffffu, own == best) >> (lane - sub);
      const int from = __ffs(holds) - 1;  // below G: the group's own maximum is among its lanes
      const int idx = from * V + __shfl_sync(0xffffffffu, at, lane - sub + from);
      const bool some = best != 0u;
      const float val = some ? __uint_as_float((best & 0x80000000u) ? (best & 0x7fffffffu) : ~best) : -INFINITY;
      if (j == 0) {
        first = val;
        m = some ? val : 0.f;
        float part = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          v[i] = exp_of(v[i] - m);  // from here on the exponentials; -inf: 0
          part += v[i];
        }
        total = group_sum<G>(part);
        inv = total > 0.f ? 1.f / total : 0.f;
      }
      const float ex = some ? exp_of(val - m) : 0.f;
      top_sum += ex;
      if (sub == from) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (i == at) key[i] = 0u;
      }
      // lane j % G of the group keeps the j-th choice until all are known
      if (in && sub == j % G) {
        p.ids[row * p.k + j] = some ? idx : -1;
        if (some) atomicAdd(&s_hist[idx], 1);
        mine = ex;
        if (!p.norm) {
          const float w = ex * inv;
          if (p.weights_bf16) reinterpret_cast<__nv_bfloat16*>(p.weights)[row * p.k + j] = __float2bfloat16(w);
          else reinterpret_cast<float*>(p.weights)[row * p.k + j] = w;
        } else if (p.k > G) {
          // more choices than lanes: the exponentials wait in place (fp32 weights) or are taken again below
          if (!p.weights_bf16) reinterpret_cast<float*>(p.weights)[row * p.k + j] = ex;
        }
      }
    }
    if (p.norm && in) {
      const float of = top_sum > 0.f ? top_sum : 1.f;  // divided by: a single choice has weight 1 exactly
      if (p.k <= G) {
        if (sub < p.k) {
          const float w = mine / of;
          if (p.weights_bf16) reinterpret_cast<__nv_bfloat16*>(p.weights)[row * p.k + sub] = __float2bfloat16(w);
          else reinterpret_cast<float*>(p.weights)[row * p.k + sub] = w;
        }
      } else {
        for (int j = sub; j < p.k; j += G) {  // written by this very lane above
          if (p.weights_bf16) {
            const int id = p.ids[row * p.k + j];
            const float z = id < 0 ? -INFINITY
                            : p.logits_bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.logits)[row * p.E + id])
                                            : reinterpret_cast<const float*>(p.logits)[row * p.E + id];
            reinterpret_cast<__nv_bfloat16*>(p.weights)[row * p.k + j] = __float2bfloat16(id < 0 ? 0.f : exp_of(z - m) / of);
          } else {
            float* w = reinterpret_cast<float*>(p.weights) + row * p.k + j;
            *w = *w / of;
          }
        }
      }
    }
    const bool routed = in && first > -INFINITY;
    if (routed) {
      live += sub == 0;
      if (sums) {
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(v[i], inv, acc[i]);
      }
      if (zsums && sub == 0) {
        const float lse = m + logf(total);
        zacc = fmaf(lse, lse, zacc);
      }
    }
  }
  // the block's sums, in a fixed order: over the rows a warp held at once, then
  // over the warps
  if (sums) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
      for (int d = G; d < 32; d <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], d);
      if (lane < G && c + i < p.E) s_sum[warp * p.E + c + i] = acc[i];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += THREADS) {
      float t = 0.f;
#pragma unroll 8
      for (int q = 0; q < WARPS; ++q) t += s_sum[q * p.E + e];
      p.psum[(int64_t)b * p.E + e] = t;
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += THREADS) p.hist[(int64_t)b * p.E + e] = s_hist[e];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    live += __shfl_xor_sync(0xffffffffu, live, d);
    zacc += __shfl_xor_sync(0xffffffffu, zacc, d);
  }
  if (lane == 0) {
    s_sum[warp] = zacc;
    reinterpret_cast<int*>(s_sum)[WARPS + warp] = live;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    float z = 0.f;
    int l = 0;
    for (int w = 0; w < WARPS; ++w) {
      z += s_sum[w];
      l += reinterpret_cast<int*>(s_sum)[WARPS + w];
    }
    p.zsum[b] = z;
    p.live[b] = l;
  }
  __syncthreads();
}

// Places of block b's pairs: an expert's rows are those of the blocks before,
// then of this block's warps before, then in the order of the pairs.
// s_count: [WARPS][E]; s_tot, s_base: [E].
template <int THREADS>
__device__ void place_rows(const RouteParams& p, int64_t r0, int64_t r1, int b, int* s_count, int* s_tot, int* s_base) {
  const int lane = lane_id(), warp = warp_id();
  constexpr int WARPS = THREADS / 32;
  __shared__ int s_part[2][THREADS];
  for (int e0 = 0; e0 < p.E; e0 += THREADS) {
    // rows of each expert in all blocks and in those before b: slices of the
    // blocks per expert where the experts leave threads over
    const int span = min(p.E - e0, THREADS);
    const int slices = THREADS / span;
    const int e = e0 + (int)threadIdx.x % span, sl = (int)threadIdx.x / span;
    int before = 0, all = 0;
    if (sl < slices)
      for (int q0 = sl; q0 < p.nblk; q0 += 10 * slices) {
        // ten loads at once, so that few blocks are not one latency each
        int v[10];
#pragma unroll
        for (int i = 0; i < 10; ++i) {
          const int q = q0 + i * slices;
          v[i] = q < p.nblk ? p.hist[q * p.E + e] : 0;
        }
#pragma unroll
        for (int i = 0; i < 10; ++i) {
          all += v[i];
          before += q0 + i * slices < b ? v[i] : 0;
        }
      }
    s_part[0][threadIdx.x] = all;
    s_part[1][threadIdx.x] = before;
    __syncthreads();
    if ((int)threadIdx.x < span) {
      int a = 0, f = 0;
      for (int q = 0; q < slices; ++q) {
        a += s_part[0][q * span + threadIdx.x];
        f += s_part[1][q * span + threadIdx.x];
      }
      s_tot[e0 + threadIdx.x] = a;
      s_base[e0 + threadIdx.x] = f;
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < WARPS * p.E; i += THREADS) s_count[i] = 0;
  __shared__ int s_all;
  if (warp == 0) {
    int run = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      const int t = e < p.E ? s_tot[e] : 0;
      int u = t;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, u, d);
        if (lane >= d) u += o;
      }
      if (e < p.E) {
        s_base[e] += run + u - t;
        if (b == 0) p.offsets[e] = run + u - t;
      }
      run += __shfl_sync(0xffffffffu, u, 31);
    }
    if (lane == 0) {
      s_all = run;
      if (b == 0) p.offsets[p.E] = run;
    }
  }
  __syncthreads();
  const int64_t q0 = r0 * p.k, q1 = r1 * p.k;
  const int64_t share = ((q1 - q0 + WARPS - 1) / WARPS + 31) / 32 * 32;  // pairs a warp
  const int64_t w0 = min(q1, q0 + warp * share), w1 = min(q1, w0 + share);
  int* mine = s_count + warp * p.E;
  for (int64_t q = w0 + lane; q < w1; q += 32) {
    const int id = p.ids[q];
    if (id >= 0) atomicAdd(&mine[id], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += THREADS) {
    int run = s_base[e];
    for (int w = 0; w < WARPS; ++w) {
      const int t = s_count[w * p.E + e];
      s_count[w * p.E + e] = run;
      run += t;
    }
  }
  __syncthreads();
  for (int64_t q = w0; q < w1; q += 32) {
    const bool in = q + lane < w1;
    const int id = in ? p.ids[q + lane] : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, id);
    const int rank = __popc(same & ((1u << lane) - 1u));
    int at = -1;
    if (id >= 0) at = mine[id] + rank;
    __syncwarp();
    if (id >= 0 && rank == 0) mine[id] += __popc(same);
    __syncwarp();
    if (in) {
      p.slot[q + lane] = at;
      if (at >= 0) p.order[at] = (int)(q + lane);
    }
  }
  // behind the last routed row
  const int64_t pairs = p.n * p.k;
  for (int64_t i = s_all + (int64_t)b * THREADS + threadIdx.x; i < pairs; i += (int64_t)p.nblk * THREADS) p.order[i] = -1;
}

// The losses and the number of routed rows, by one block: sums over the
// blocks of rows, in an order fixed by their number.
template <int THREADS>
__device__ void finish_losses(const RouteParams& p) {
  constexpr int WARPS = THREADS / 32;
  __shared__ float s_ps[THREADS];
  __shared__ int s_live[WARPS], s_rows[THREADS];
  const int lane = lane_id(), warp = warp_id();
  int l = 0;
  for (int q = threadIdx.x; q < p.nblk; q += THREADS) l += p.live[q];
  l = __reduce_add_sync(0xffffffffu, l);
  if (lane == 0) s_live[warp] = l;
  __syncthreads();
  l = 0;
  for (int w = 0; w < WARPS; ++w) l += s_live[w];
  if (threadIdx.x == 0) p.offsets[p.E + 1] = l;
  if (!p.loss) return;
  // sum_e count_e sum_t p_te: slices of the blocks per expert, in fp32 by at
  // most 152 blocks and then in fp64 (which this card adds slowly) by one warp
  double t = 0.0;
  if (p.balance != 0.f) {
    for (int e0 = 0; e0 < p.E; e0 += THREADS) {
      const int span = min(p.E - e0, THREADS), slices = THREADS / span;
      const int e = e0 + (int)threadIdx.x % span, sl = (int)threadIdx.x / span;
      int rows = 0;
      float ps = 0.f;
      if (sl < slices)
        for (int q0 = sl; q0 < p.nblk; q0 += 10 * slices) {
          int v[10];
          float f[10];
#pragma unroll
          for (int i = 0; i < 10; ++i) {
            const int q = q0 + i * slices;
            v[i] = q < p.nblk ? p.hist[q * p.E + e] : 0;
            f[i] = q < p.nblk ? p.psum[q * p.E + e] : 0.f;
          }
#pragma unroll
          for (int i = 0; i < 10; ++i) {
            rows += v[i];
            ps += f[i];
          }
        }
      s_rows[threadIdx.x] = rows;
      s_ps[threadIdx.x] = ps;
      __syncthreads();
      if (warp == 0)
        for (int i = lane; i < span; i += 32) {
          int r = 0;
          double sum = 0.0;
          for (int q = 0; q < slices; ++q) {
            r += s_rows[q * span + i];
            sum += (double)s_ps[q * span + i];
          }
          t += sum * (double)r;
        }
      __syncthreads();
    }
  }
  if (warp) return;
  double z = 0.0;
  if (p.zc != 0.f) {
    static_assert(MAX_BLOCKS <= 160, "five of them a lane");
    float f[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) f[i] = lane + 32 * i < p.nblk ? p.zsum[lane + 32 * i] : 0.f;
#pragma unroll
    for (int i = 0; i < 5; ++i) z += (double)f[i];
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    t += __shfl_down_sync(0xffffffffu, t, d);
    z += __shfl_down_sync(0xffffffffu, z, d);
  }
  if (lane == 0) {
    const double nv = l > 0 ? l : 1;
    *p.loss = (float)((double)p.balance * p.E / (nv * nv * p.k) * t + (double)p.zc / nv * z);
  }
}

template <int G, int V>
__global__ void __launch_bounds__(choose_threads<V>()) route_choose_kernel(const RouteParams p) {
  extern __shared__ float s_dyn[];
  int* s_hist = reinterpret_cast<int*>(s_dyn);
  float* s_sum = s_dyn + p.E;
  wait_for_previous();
  let_next_start();
  const int64_t r0 = min(p.n, blockIdx.x * p.per), r1 = min(p.n, r0 + p.per);
  choose_rows<G, V, choose_threads<V>()>(p, r0, r1, blockIdx.x, s_hist, s_sum);
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) route_place_kernel(const RouteParams p) {
  extern __shared__ float s_dyn[];
  constexpr int WARPS = THREADS / 32;
  int* s_count = reinterpret_cast<int*>(s_dyn);
  wait_for_previous();
  let_next_start();
  if ((int)blockIdx.x == p.nblk) return finish_losses<THREADS>(p);
  const int64_t r0 = min(p.n, blockIdx.x * p.per), r1 = min(p.n, r0 + p.per);
  place_rows<THREADS>(p, r0, r1, blockIdx.x, s_count, s_count + WARPS * p.E, s_count + (WARPS + 1) * p.E);
}

// Few rows: one block does both
constexpr int ONE_THREADS = 256;
template <int G, int V>
__global__ void __launch_bounds__(ONE_THREADS) route_one_kernel(const RouteParams p) {
  extern __shared__ float s_dyn[];
  constexpr int WARPS = ONE_THREADS / 32;
  int* s_int = reinterpret_cast<int*>(s_dyn);
  wait_for_previous();
  let_next_start();
  choose_rows<G, V, ONE_THREADS>(p, 0, p.n, 0, s_int, s_dyn + p.E);
  place_rows<ONE_THREADS>(p, 0, p.n, 0, s_int, s_int + WARPS * p.E, s_int + (WARPS + 1) * p.E);
  finish_losses<ONE_THREADS>(p);
}

struct RouteBwdParams {
  const void* logits;
  int logits_bf16, weights_bf16;
  int64_t n;
  int E, k, norm;
  float balance, zc;  // times the loss's gradient
  const int32_t *ids, *offsets;
  const void* dweights;
  void* dlogits;
};

// dz of a row: through the weights, q the softmax they are taken of (over the
// chosen, or over all): dz_e = q_e (g_e - sum_e' g_e' q_e'), g the weights'
// gradients at the chosen; the balance loss: the same with p and
// g_e = balance E count_e / (nv^2 k); the z loss: 2 z_coef lse / nv p_e.
template <int G, int V>
__global__ void __launch_bounds__(BWD_THREADS) route_bwd_kernel(const RouteBwdParams p) {
  const int lane = lane_id();
  const int sub = lane % G, c = sub * V;
  constexpr int ROWS = 32 / G, WARPS = BWD_THREADS / 32;
  wait_for_previous();
  let_next_start();
  const int nv_i = p.offsets[p.E + 1];
  const float nv = nv_i > 0 ? (float)nv_i : 1.f;
  const bool aux = p.balance != 0.f || p.zc != 0.f;
  float share[V];
  const float each = p.balance * (float)p.E / nv / (nv * (float)p.k);
#pragma unroll
  for (int i = 0; i < V; ++i)
    share[i] = p.balance != 0.f && c + i < p.E ? each * (float)(p.offsets[c + i + 1] - p.offsets[c + i]) : 0.f;
  const int64_t step = (int64_t)gridDim.x * WARPS * ROWS;
  for (int64_t base = ((int64_t)blockIdx.x * WARPS + warp_id()) * ROWS; base < p.n; base += step) {
    const int64_t row = base + lane / G;
    const bool in = row < p.n;
    float v[V], g[V];
    if (in) {
      load_logits<V>(p.logits, p.logits_bf16, row, p.E, c, v, nullptr);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = -INFINITY;
    }
    uint32_t chosen = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) g[i] = 0.f;
    for (int j0 = 0; j0 < p.k; j0 += G) {
      // a choice a lane, then handed round the row's lanes
      int id = -1;
      float d = 0.f;
      if (in && j0 + sub < p.k) {
        const int64_t q = row * p.k + j0 + sub;
        id = p.ids[q];
        d = p.weights_bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.dweights)[q])
                           : reinterpret_cast<const float*>(p.dweights)[q];
      }
      const int left = min(G, p.k - j0);
      for (int j = 0; j < left; ++j) {
        const int at = __shfl_sync(0xffffffffu, id, lane - sub + j) - c;
        const float dj = __shfl_sync(0xffffffffu, d, lane - sub + j);
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (at == i) {
            g[i] += dj;
            chosen |= 1u << i;
          }
      }
    }
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, v[i]);
    m = group_max<G>(m);
    const bool live = m > -INFINITY;
    if (!live) m = 0.f;
    float ex[V], all = 0.f, some = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      ex[i] = exp_of(v[i] - m);
      all += ex[i];
      some += (chosen >> i) & 1u ? ex[i] : 0.f;
    }
    all = group_sum<G>(all);
    if (p.norm) some = group_sum<G>(some);
    const float inv_p = live ? 1.f / all : 0.f;
    // over the chosen: a division, so that a single choice has weight 1 exactly
    float q[V], gq = 0.f, sp = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      q[i] = !p.norm ? ex[i] * inv_p : ((chosen >> i) & 1u) && some > 0.f ? ex[i] / some : 0.f;
      gq = fmaf(g[i], q[i], gq);
      sp = fmaf(share[i], ex[i] * inv_p, sp);
    }
    gq = group_sum<G>(gq);
    float zt = 0.f;
    if (aux) {
      sp = group_sum<G>(sp);
      zt = live ? 2.f * p.zc / nv * (m + logf(all)) - sp : 0.f;
    }
    if (in) {
      float dz[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        dz[i] = q[i] * (g[i] - gq);
        if (aux) dz[i] = fmaf(ex[i] * inv_p, share[i] + zt, dz[i]);
      }
      if (c + V <= p.E && (p.E & 7) == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 8) {
          if (p.logits_bf16) {
            uint4 u;
            u.x = pack_bf16(dz[i], dz[i + 1]);
            u.y = pack_bf16(dz[i + 2], dz[i + 3]);
            u.z = pack_bf16(dz[i + 4], dz[i + 5]);
            u.w = pack_bf16(dz[i + 6], dz[i + 7]);
            *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.dlogits) + row * p.E + c + i) = u;
          } else {
            float4* o = reinterpret_cast<float4*>(reinterpret_cast<float*>(p.dlogits) + row * p.E + c + i);
            o[0] = make_float4(dz[i], dz[i + 1], dz[i + 2], dz[i + 3]);
            o[1] = make_float4(dz[i + 4], dz[i + 5], dz[i + 6], dz[i + 7]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (c + i < p.E) {
            if (p.logits_bf16) reinterpret_cast<__nv_bfloat16*>(p.dlogits)[row * p.E + c + i] = __float2bfloat16(dz[i]);
            else reinterpret_cast<float*>(p.dlogits)[row * p.E + c + i] = dz[i];
          }
      }
    }
  }
}

// lanes that hold a row (by_width)
int row_lanes(int E) { return E <= 16 ? 2 : E <= 32 ? 4 : E <= 64 ? 8 : E <= 128 ? 16 : 32; }

// One block does it all in one launch up to the rows its warps hold at once
// (three times that where a warp holds one row, whose placing in a launch of its
// own takes longer): 64 experts, 16 rows 9.0 us, 64 rows 11.6 in one block and
// 128 rows 9.7 in two launches; 256 experts, 64 rows 31 and 128 rows 17.
bool one_block(int64_t n, int E) {
  const int g = row_lanes(E);
  return n <= ONE_THREADS / g * (g == 32 ? 3 : 1);
}
// blocks of rows of the two-launch form
int route_blocks(int64_t n) { return (int)std::max<int64_t>(1, std::min<int64_t>(MAX_BLOCKS, (n + 63) / 64)); }

template <int G, int V>
int route_launch(const RouteParams& p, cudaStream_t st) {
  // shared memory: the choice's counts and sums, then the placing's counts
  auto choose = [&](int warps) { return (size_t)(p.E + std::max(warps * p.E, 2 * warps)) * 4; };
  auto place = [&](int warps) { return (size_t)(warps + 2) * p.E * 4; };
  if (one_block(p.n, p.E)) {
    constexpr int W = ONE_THREADS / 32;
    return launch_dependent(route_one_kernel<G, V>, 1, 1, dim3(ONE_THREADS), std::max(choose(W), place(W)), st, p) == cudaSuccess ? BPT_OK
                                                                                                                                : BPT_ECUDA;
  }
  constexpr int T = choose_threads<V>(), PT = V == 8 ? 1024 : 256;
  if (launch_dependent(route_choose_kernel<G, V>, p.nblk, 1, dim3(T), choose(T / 32), st, p) != cudaSuccess) return BPT_ECUDA;
  auto k = route_place_kernel<PT>;
  static std::atomic<uint64_t> attr{0};
  if (smem_limit_once(reinterpret_cast<const void*>(k), 48 * 1024, &attr)) return BPT_ECUDA;
  return launch_dependent(k, p.nblk + 1, 1, dim3(PT), place(PT / 32), st, p) == cudaSuccess ? BPT_OK : BPT_ECUDA;
}

// G lanes of V logits hold a row: 8 a lane (a 32- or 16-byte load) as long as
// a warp's lanes suffice
template <class F>
int by_width(int E, F&& f) {
  if (E <= 16) return f(std::integral_constant<int, 2>(), std::integral_constant<int, 8>());
  if (E <= 32) return f(std::integral_constant<int, 4>(), std::integral_constant<int, 8>());
  if (E <= 64) return f(std::integral_constant<int, 8>(), std::integral_constant<int, 8>());
  if (E <= 128) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 8>());
  if (E <= 256) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 8>());
  if (E <= 512) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 16>());
  return f(std::integral_constant<int, 32>(), std::integral_constant<int, 32>());
}

struct RouteWs {
  int* hist;
  float* psum;
  float* zsum;
  int* live;
};
size_t plan_route(const MoeDims& D, void* base, RouteWs* w) {
  const int nb = one_block(D.n, (int)D.E) ? 1 : route_blocks(D.n);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) / 256 * 256;
    return at;
  };
  const size_t h = take((size_t)nb * D.E * 4), s = take((size_t)nb * D.E * 4), z = take((size_t)nb * 4), l = take((size_t)nb * 4);
  if (base) {
    uint8_t* b = reinterpret_cast<uint8_t*>(base);
    w->hist = reinterpret_cast<int*>(b + h);
    w->psum = reinterpret_cast<float*>(b + s);
    w->zsum = reinterpret_cast<float*>(b + z);
    w->live = reinterpret_cast<int*>(b + l);
  }
  return off;
}

bool aligned(const void* p, int a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace

}  // namespace bpt

using namespace bpt;

extern "C" {

size_t bpt_moe_route_workspace_bytes(const bpt_moe_config* cfg) {
  MoeDims D;
  if (moe_dims(cfg, &D)) return 0;
  return plan_route(D, nullptr, nullptr);
}

int bpt_moe_route_fwd(const bpt_moe_config* cfg, const void* logits, const bpt_moe_route* r, float* loss, void* ws, size_t ws_bytes,
                      void* stream) {
  MoeDims D;
  int rc = moe_dims(cfg, &D);
  if (rc) return rc;
  if (!logits || !r || !r->ids || !r->weights || !r->offsets || !r->order || !r->slot || !ws) return BPT_EINVAL;
  if (!loss && (cfg->balance_coef != 0.f || cfg->z_coef != 0.f)) return BPT_EINVAL;
  if (!aligned(logits, 16) || !aligned(r->ids, 4) || !aligned(r->weights, 4) || !aligned(r->offsets, 4) || !aligned(r->order, 4) ||
      !aligned(r->slot, 4) || !aligned(loss, 4) || !aligned(ws, 16))
    return BPT_EINVAL;
  const size_t need = plan_route(D, nullptr, nullptr);
  if (ws_bytes < need) return BPT_ENOSPC;
  const Span sp[] = {{logits, D.n * D.E * D.logit_bytes}, {r->ids, D.pairs * 4},   {r->weights, D.pairs * D.weight_bytes},
                     {r->offsets, (D.E + 2) * 4},         {r->order, D.pairs * 4}, {r->slot, D.pairs * 4},
                     {ws, (int64_t)need},                 {loss, loss ? 4 : 0}};
  for (int i = 1; i < 8; ++i)
    if (sp[i].p && overlaps(sp[i], sp, i)) return BPT_EINVAL;
  if (D.debug && debug_spans(sp, 8)) return BPT_EINVAL;
  RouteWs W;
  plan_route(D, ws, &W);
  RouteParams p;
  p.logits = logits;
  p.logits_bf16 = D.logit_bytes == 2;
  p.weights_bf16 = D.weight_bytes == 2;
  p.n = D.n;
  p.E = (int)D.E;
  p.k = (int)D.k;
  p.norm = cfg->norm_topk;
  p.balance = cfg->balance_coef;
  p.zc = cfg->z_coef;
  p.ids = r->ids;
  p.offsets = r->offsets;
  p.order = r->order;
  p.slot = r->slot;
  p.weights = r->weights;
  p.loss = loss;
  p.hist = W.hist;
  p.psum = W.psum;
  p.zsum = W.zsum;
  p.live = W.live;
  p.nblk = one_block(D.n, p.E) ? 1 : route_blocks(D.n);
  p.per = (D.n + p.nblk - 1) / p.nblk;
  p.err = device_error_word();
  if (!p.err) return BPT_ECUDA;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  {
    ProfScope prof(PROF_MISC, 0.0, (double)D.n * D.E * D.logit_bytes + 16.0 * (double)D.pairs, st);
    rc = by_width(p.E, [&](auto g, auto v) { return route_launch<g.value, v.value>(p, st); });
  }
  if (rc) return rc;
  return D.debug ? debug_finish(st) : BPT_OK;
}

int bpt_moe_route_bwd(const bpt_moe_config* cfg, const void* logits, const bpt_moe_route* r, const void* dweights, float dloss,
                      void* dlogits, void* stream) {
  MoeDims D;
  int rc = moe_dims(cfg, &D);
  if (rc) return rc;
  if (!logits || !r || !r->ids || !r->offsets || !dweights || !dlogits) return BPT_EINVAL;
  if (!aligned(logits, 16) || !aligned(r->ids, 4) || !aligned(r->offsets, 4) || !aligned(dweights, 4) || !aligned(dlogits, 16))
    return BPT_EINVAL;
  if (!(fabsf(dloss) < INFINITY)) return BPT_EINVAL;
  const Span in[] = {{logits, D.n * D.E * D.logit_bytes}, {r->ids, D.pairs * 4}, {r->offsets, (D.E + 2) * 4},
                     {dweights, D.pairs * D.weight_bytes}, {dlogits, D.n * D.E * D.logit_bytes}};
  if (overlaps(in[4], in, 4)) return BPT_EINVAL;
  if (D.debug && debug_spans(in, 5)) return BPT_EINVAL;
  RouteBwdParams p;
  p.logits = logits;
  p.logits_bf16 = D.logit_bytes == 2;
  p.weights_bf16 = D.weight_bytes == 2;
  p.n = D.n;
  p.E = (int)D.E;
  p.k = (int)D.k;
  p.norm = cfg->norm_topk;
  p.balance = cfg->balance_coef * dloss;
  p.zc = cfg->z_coef * dloss;
  p.ids = r->ids;
  p.offsets = r->offsets;
  p.dweights = dweights;
  p.dlogits = dlogits;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int sms = sm_count();
  if (sms <= 0) return BPT_ECUDA;
  {
    ProfScope prof(PROF_MISC, 0.0, 2.0 * (double)D.n * D.E * D.logit_bytes + 8.0 * (double)D.pairs, st);
    rc = by_width(p.E, [&](auto g, auto v) {
      constexpr int per = BWD_THREADS / 32 * (32 / g.value);
      const int grid = (int)std::min<int64_t>((D.n + per - 1) / per, 8 * (int64_t)sms);
      return launch_dependent(route_bwd_kernel<g.value, v.value>, grid, 1, dim3(BWD_THREADS), 0, st, p) == cudaSuccess ? BPT_OK : BPT_ECUDA;
    });
  }
  if (rc) return rc;
  return D.debug ? debug_finish(st) : BPT_OK;
}

}  // extern "C"
