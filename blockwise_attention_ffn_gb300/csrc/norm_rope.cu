// norm_rope.cu -- the norm of every query and key head with the rotary
// position embedding in the same pass, on the packed projection buffer
// [rows, (H + 2 H_kv) d], forward and backward.
//
// With x one head's d values of one row, w the head norm's weight (one vector
// for all query heads, one for all key heads) and R(p) the rotation of the
// pairs (i, i + d/2) by p * base^(-2i/d):
//   r = (mean x^2 + eps)^(-1/2),  n = x r,  y = R(p) (n * w)
// and for an upstream gradient dy
//   dn = R(p)^T dy,  dw = sum over rows and heads of dn * n,
//   g = dn * w,  dx = r (g - n mean(g * n)).
// V's columns pass through (copied where the output is another buffer).
//
// HBM-bound: one read of each input and one write of the output.  A lane
// takes 8 consecutive elements of a head's first half and the 8 they are
// paired with in its second half, two 16-byte loads, so L = d/16 lanes hold a
// head and a warp takes 32/L heads at a time, neighbours in memory.  All
// statistics, angles' sines and sums are fp32; each output is rounded once.
//
// Angles: p * theta in turns, as a 64-bit fraction of a turn.  The product of
// the integer position with the frequency's fraction, modulo 2^64, is the
// angle reduced exactly, whatever the position; its upper 32 bits give the
// argument of one sincospi.  A row's angles are the same for all its heads,
// so a lane keeps its 8 sines and cosines until its row changes.
//
// The weights' gradients: fp32 sums per lane over the heads it meets, per
// block over its lanes in shared memory, one partial per block, added in
// block order by a second kernel: no atomics, one summation order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <string.h>

#include <algorithm>

#include "../../include/bpt.h"
#include "internal.h"
#include "ptx.cuh"

namespace bpt {
namespace {

constexpr int NR_THREADS = 256;
constexpr int NR_WARPS = NR_THREADS / 32;
constexpr int NR_MAX_BLOCKS = 152 * 4;  // partials of the weight gradients

struct NormRopeParams {
  const __nv_bfloat16 *x, *dy;  // dy: backward only
  __nv_bfloat16* out;
  const __nv_bfloat16 *wq, *wk;  // null: no norm
  const int32_t* pos;            // null: the row's index in its sequence
  float* part;                   // [blocks][2 d], or null
  int64_t rows;
  int s, H, K, d, width, rope, copy_v;
  float eps;
  uint64_t turn[64];  // base^(-2i/d) / (2 pi) as a fraction of 2^64
};

// sum over the L lanes that hold one head (lanes slot * L .. slot * L + L-1)
template <int L>
__device__ __forceinline__ float head_sum(float v, int base, int idx) {
  if constexpr ((L & (L - 1)) == 0) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  } else {
    float s = v;
#pragma unroll
    for (int k = 1; k < L; ++k) {
      const int j = idx + k;
      s += __shfl_sync(0xffffffffu, v, base + (j >= L ? j - L : j));
    }
    return s;
  }
}

__device__ __forceinline__ void unpack8(uint4 v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

// One section of the columns (the query heads, or the key heads): n heads
// from column col0.  Items are the rows * n (row, head) pairs in memory
// order; a warp takes 32/L neighbouring ones per step and `steps` steps in a
// row, then moves on by the whole grid.
template <int L, bool BWD>
__device__ __forceinline__ void section(const NormRopeParams& p, int n, int col0, const __nv_bfloat16* w, int steps,
                                        float (&acc)[16]) {
  constexpr int HPW = 32 / L;
  const int lane = lane_id();
  const int slot = lane / L, idx = lane % L, base = slot * L;
  const bool lane_on = slot < HPW;
  const int half = p.d / 2;
  const int64_t items = p.rows * n;
  const int64_t per_run = (int64_t)HPW * steps;
  const int64_t warps = (int64_t)gridDim.x * NR_WARPS;
  const float inv_d = 1.f / (float)p.d;
  const int step_rows = HPW / n, step_heads = HPW % n;
  uint4 wa = make_uint4(0u, 0u, 0u, 0u), wb = wa;
  if (w && lane_on) {
    wa = *reinterpret_cast<const uint4*>(w + 8 * idx);
    wb = *reinterpret_cast<const uint4*>(w + half + 8 * idx);
  }
  float cs[8], sn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    cs[i] = 1.f;
    sn[i] = 0.f;
  }
  for (int64_t run = (int64_t)blockIdx.x * NR_WARPS + warp_id(); run * per_run < items; run += warps) {
    int64_t it = run * per_run + slot;
    const int64_t end = min(items, (run + 1) * per_run);
    int64_t row = it / n;
    int head = (int)(it - row * n);
    int64_t angles_of = -1;
    for (int st = 0; st < steps; ++st, it += HPW) {
      const bool on = lane_on && it < end;
      const int64_t at = row * p.width + col0 + (int64_t)head * p.d + 8 * idx;
      uint4 xa = make_uint4(0u, 0u, 0u, 0u), xb = xa, ya = xa, yb = xa;
      if (on && (!BWD || w)) {
        xa = *reinterpret_cast<const uint4*>(p.x + at);
        xb = *reinterpret_cast<const uint4*>(p.x + at + half);
      }
      if (BWD && on) {
        ya = *reinterpret_cast<const uint4*>(p.dy + at);
        yb = *reinterpret_cast<const uint4*>(p.dy + at + half);
      }
      if (p.rope && on && row != angles_of) {
        angles_of = row;
        const int64_t pos = p.pos ? (int64_t)p.pos[row] : row % p.s;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint64_t t = (uint64_t)pos * p.turn[8 * idx + i];
          sincospif((float)(int32_t)(t >> 32) * 0x1p-31f, &sn[i], &cs[i]);
        }
      }
      float a[8], b[8];
      unpack8(xa, a);
      unpack8(xb, b);
      float r = 1.f;
      if (w) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(a[i], a[i], fmaf(b[i], b[i], s));
        s = head_sum<L>(s, base, idx);
        r = rsqrtf(s * inv_d + p.eps);
      }
      float oa[8], ob[8];
      if constexpr (!BWD) {
        if (w) {
          float ua[8], ub[8];
          unpack8(wa, ua);
          unpack8(wb, ub);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            a[i] = a[i] * r * ua[i];
            b[i] = b[i] * r * ub[i];
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          oa[i] = a[i] * cs[i] - b[i] * sn[i];
          ob[i] = a[i] * sn[i] + b[i] * cs[i];
        }
      } else {
        float da[8], db[8];
        unpack8(ya, da);
        unpack8(yb, db);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          oa[i] = da[i] * cs[i] + db[i] * sn[i];
          ob[i] = db[i] * cs[i] - da[i] * sn[i];
        }
        if (w) {
          float ua[8], ub[8];
          unpack8(wa, ua);
          unpack8(wb, ub);
          float s = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            a[i] *= r;  // n
            b[i] *= r;
            acc[i] = fmaf(oa[i], a[i], acc[i]);
            acc[8 + i] = fmaf(ob[i], b[i], acc[8 + i]);
            oa[i] *= ua[i];  // g
            ob[i] *= ub[i];
            s = fmaf(oa[i], a[i], fmaf(ob[i], b[i], s));
          }
          s = head_sum<L>(s, base, idx) * inv_d;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            oa[i] = r * (oa[i] - a[i] * s);
            ob[i] = r * (ob[i] - b[i] * s);
          }
        }
      }
      if (on) {
        *reinterpret_cast<uint4*>(p.out + at) = pack8(oa);
        *reinterpret_cast<uint4*>(p.out + at + half) = pack8(ob);
      }
      row += step_rows;
      head += step_heads;
      if (head >= n) {
        head -= n;
        ++row;
      }
    }
  }
}

// steps a warp takes in a row: up to 8, so that a row's angles serve many
// heads, but no more than leaves every warp of the grid some work
__device__ __forceinline__ int steps_for(int64_t items, int hpw) {
  const int64_t per = items / ((int64_t)hpw * gridDim.x * NR_WARPS);
  return (int)(per < 1 ? 1 : per > 8 ? 8 : per);
}

template <int L, bool BWD>
__global__ void __launch_bounds__(NR_THREADS, BWD ? 2 : 3) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int HPW = 32 / L;
  constexpr int D = 16 * L;
  __shared__ float red[BWD ? NR_WARPS * HPW * D : 1];
#pragma unroll 1
  for (int sec = 0; sec < 2; ++sec) {
    const int n = sec ? p.K : p.H;
    float acc[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
    section<L, BWD>(p, n, sec ? p.H * D : 0, sec ? p.wk : p.wq, steps_for(p.rows * n, HPW), acc);
    if constexpr (BWD) {
      if (p.part) {
        const int lane = lane_id(), slot = lane / L, idx = lane % L;
        if (slot < HPW) {
          float* dst = red + (warp_id() * HPW + slot) * D;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dst[8 * idx + i] = acc[i];
            dst[D / 2 + 8 * idx + i] = acc[8 + i];
          }
        }
        __syncthreads();
        if (threadIdx.x < D) {
          float s = 0.f;
          for (int k = 0; k < NR_WARPS * HPW; ++k) s += red[k * D + threadIdx.x];
          p.part[((int64_t)blockIdx.x * 2 + sec) * D + threadIdx.x] = s;
        }
        __syncthreads();
      }
    }
  }
  if (BWD) let_next_start();
  if (p.copy_v) {
    const __nv_bfloat16* src = BWD ? p.dy : p.x;
    const int per = p.K * D / 8;  // 16-byte units of a row
    const int64_t total = p.rows * per;
    const int64_t stride = (int64_t)gridDim.x * NR_THREADS;
#pragma unroll 4
    for (int64_t u = (int64_t)blockIdx.x * NR_THREADS + threadIdx.x; u < total; u += stride) {
      const int64_t row = u / per;
      const int64_t at = row * p.width + (int64_t)(p.H + p.K) * D + (u - row * per) * 8;
      *reinterpret_cast<uint4*>(p.out + at) = *reinterpret_cast<const uint4*>(src + at);
    }
  }
}

// dw[c] (+)= sum over blocks of part[block][c], c < 2 d, in a fixed order:
// 32 columns per block, 32 threads per column
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(const float* part, int nparts, int d, float* dwq,
                                                            float* dwk, int accumulate) {
  __shared__ float red[32][33];
  wait_for_previous();
  const int c = blockIdx.x * 32 + threadIdx.x;
  float s = 0.f;
  for (int i = threadIdx.y; i < nparts; i += 32) s += part[(int64_t)i * 2 * d + c];
  red[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0) {
    s = 0.f;
    for (int k = 0; k < 32; ++k) s += red[k][threadIdx.x];
    float* out = c < d ? dwq + c : dwk + (c - d);
    *out = accumulate ? *out + s : s;
  }
}

template <bool BWD>
int launch(const NormRopeParams& p, int blocks, cudaStream_t st) {
  switch (p.d) {
    case 64: norm_rope_kernel<4, BWD><<<blocks, NR_THREADS, 0, st>>>(p); break;
    case 80: norm_rope_kernel<5, BWD><<<blocks, NR_THREADS, 0, st>>>(p); break;
    case 96: norm_rope_kernel<6, BWD><<<blocks, NR_THREADS, 0, st>>>(p); break;
    case 112: norm_rope_kernel<7, BWD><<<blocks, NR_THREADS, 0, st>>>(p); break;
    case 128: norm_rope_kernel<8, BWD><<<blocks, NR_THREADS, 0, st>>>(p); break;
    default: return BPT_EUNSUPPORTED;
  }
  return cudaGetLastError() == cudaSuccess ? BPT_OK : BPT_ECUDA;
}

// blocks: enough for one step of every warp, at most what the SMs hold
int blocks_for(const PackedDims& D, int per_sm) {
  const int nsm = sm_count();
  if (nsm <= 0) return 0;
  const int hpw = 32 / (int)(D.d / 16);
  const int64_t want = (D.rows * D.H + (int64_t)hpw * NR_WARPS - 1) / ((int64_t)hpw * NR_WARPS);
  return (int)std::min<int64_t>(std::min<int64_t>(want, (int64_t)nsm * per_sm), NR_MAX_BLOCKS);
}

int fill(const bpt_config* cfg, const PackedDims& D, const void* wq, const void* wk, const int32_t* pos,
         NormRopeParams* p) {
  memset(p, 0, sizeof(*p));
  p->wq = reinterpret_cast<const __nv_bfloat16*>(wq);
  p->wk = reinterpret_cast<const __nv_bfloat16*>(wk);
  p->pos = pos;
  p->rows = D.rows;
  p->s = (int)D.s;
  p->H = (int)D.H;
  p->K = (int)D.Hkv;
  p->d = (int)D.d;
  p->width = (int)D.width;
  p->eps = cfg->norm_eps;
  p->rope = cfg->rope_base > 0.f;
  if (p->rope)
    for (int i = 0; i < D.d / 2; ++i) {
      const double turns = pow((double)cfg->rope_base, -2.0 * i / (double)D.d) * 0.15915494309189535;
      p->turn[i] = (uint64_t)ldexp(turns, 64);
    }
  return BPT_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// two buffers of n bytes that overlap without being the same one
bool part_overlap(const void* a, const void* b, int64_t n) {
  const intptr_t x = reinterpret_cast<intptr_t>(a), y = reinterpret_cast<intptr_t>(b);
  return x != y && x < y + n && y < x + n;
}

// what both directions check: the config, the weights, the positions
int check_common(const bpt_config* cfg, const void* wq, const void* wk, const int32_t* pos, PackedDims* D) {
  const int rc = packed_dims(cfg, D);
  if (rc) return rc;
  if ((wq == nullptr) != (wk == nullptr) || !aligned16(wq) || !aligned16(wk)) return BPT_EINVAL;
  if (reinterpret_cast<uintptr_t>(pos) & 3) return BPT_EINVAL;
  if (!wq && !(cfg->rope_base > 0.f)) return BPT_EINVAL;  // neither a norm nor a rotation
  if (D->width > INT32_MAX) return BPT_EUNSUPPORTED;
  return BPT_OK;
}

size_t ws_need(const PackedDims& D) { return (size_t)NR_MAX_BLOCKS * 2 * D.d * sizeof(float); }

}  // namespace
}  // namespace bpt

using namespace bpt;

extern "C" {

size_t bpt_qk_norm_rope_workspace_bytes(const bpt_config* cfg) {
  PackedDims D;
  return packed_dims(cfg, &D) ? 0 : ws_need(D);
}

int bpt_qk_norm_rope_fwd(const bpt_config* cfg, const void* qkv, const void* wq, const void* wk,
                         const int32_t* positions, void* out, void* stream) {
  PackedDims D;
  int rc = check_common(cfg, wq, wk, positions, &D);
  if (rc) return rc;
  if (!qkv || !out || !aligned16(qkv) || !aligned16(out)) return BPT_EINVAL;
  const int64_t bytes = D.rows * D.width * 2;
  if (part_overlap(qkv, out, bytes)) return BPT_EINVAL;
  if (D.debug) {
    const Span sp[] = {{qkv, bytes}, {out, bytes}, {wq, wq ? D.d * 2 : 0}, {wk, wk ? D.d * 2 : 0},
                       {positions, positions ? D.rows * 4 : 0}};
    if (debug_spans(sp, 5)) return BPT_EINVAL;
  }
  NormRopeParams p;
  fill(cfg, D, wq, wk, positions, &p);
  p.x = reinterpret_cast<const __nv_bfloat16*>(qkv);
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.copy_v = qkv != out;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int blocks = blocks_for(D, 3);
  if (blocks <= 0) return BPT_ECUDA;
  {
    ProfScope prof(PROF_NORM, 0.0, 2.0 * (p.copy_v ? bytes : bytes - D.rows * D.Hkv * D.d * 2), st);
    rc = launch<false>(p, blocks, st);
  }
  if (rc) return rc;
  return D.debug ? debug_finish(st) : BPT_OK;
}

int bpt_qk_norm_rope_bwd(const bpt_config* cfg, const void* qkv, const void* wq, const void* wk,
                         const int32_t* positions, const void* dout, void* dqkv, float* dwq, float* dwk, void* ws,
                         size_t ws_bytes, void* stream) {
  PackedDims D;
  int rc = check_common(cfg, wq, wk, positions, &D);
  if (rc) return rc;
  if (!dout || !dqkv || !aligned16(dout) || !aligned16(dqkv) || !aligned16(qkv)) return BPT_EINVAL;
  const int64_t bytes = D.rows * D.width * 2;
  if (part_overlap(dout, dqkv, bytes)) return BPT_EINVAL;
  if (wq) {
    if (!qkv || !dwq || !dwk || !ws || !aligned16(ws)) return BPT_EINVAL;
    if ((reinterpret_cast<uintptr_t>(dwq) & 3) || (reinterpret_cast<uintptr_t>(dwk) & 3)) return BPT_EINVAL;
    if (qkv == dqkv || part_overlap(qkv, dqkv, bytes)) return BPT_EINVAL;
    if (ws_bytes < ws_need(D)) return BPT_ENOSPC;
  }
  if (D.debug) {
    const int64_t dw = wq ? D.d * 4 : 0;
    const Span sp[] = {{qkv, wq ? bytes : 0}, {dout, bytes}, {dqkv, bytes}, {wq, dw / 2}, {wk, dw / 2}, {dwq, dw},
                       {dwk, dw}, {ws, wq ? (int64_t)ws_need(D) : 0}, {positions, positions ? D.rows * 4 : 0}};
    if (debug_spans(sp, 9)) return BPT_EINVAL;
  }
  NormRopeParams p;
  fill(cfg, D, wq, wk, positions, &p);
  p.x = reinterpret_cast<const __nv_bfloat16*>(qkv);
  p.dy = reinterpret_cast<const __nv_bfloat16*>(dout);
  p.out = reinterpret_cast<__nv_bfloat16*>(dqkv);
  p.part = wq ? reinterpret_cast<float*>(ws) : nullptr;
  p.copy_v = dout != dqkv;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int blocks = blocks_for(D, 2);
  if (blocks <= 0) return BPT_ECUDA;
  {
    const double v = (double)D.rows * D.Hkv * D.d * 2;
    ProfScope prof(PROF_NORM, 0.0, (wq ? 3.0 : 2.0) * (bytes - v) + (p.copy_v ? 2 * v : 0.0), st);
    rc = launch<true>(p, blocks, st);
    if (!rc && wq) {
      if (launch_dependent(norm_rope_dw_kernel, (int)(2 * D.d / 32), 1, dim3(32, 32), 0, st, (const float*)p.part,
                           blocks, (int)D.d, dwq, dwk, (int)D.accum) != cudaSuccess)
        rc = BPT_ECUDA;
    }
  }
  if (rc) return rc;
  return D.debug ? debug_finish(st) : BPT_OK;
}

}  // extern "C"
