// lm_distill.cu -- training on a teacher's stored top logits: the divergence
// of the teacher's distribution over its k entries from the student's over the
// whole vocabulary, blockwise through the vocabulary projection as lm_loss.cu,
// and its gradients.
//
//   z = x W^T / T,  q = softmax(z),  p of the entries (see bpt.h),  P = sum_j p_j
//   loss = T^2 sum_i c_i sum_j p_ij (log p_ij - z_i,id + lse_i)
//   dz (by the logits x W^T) = T dloss c_i (P_i q_iv - p_iv)
//   dx = dz W,  dW = dz^T x
//
// The entries are sorted by id once (prepare_kernel), with the place where
// each 128 columns' entries begin; the GEMM's epilogue then meets the few
// entries of a tile as it passes (EPI_KD_LSE) and keeps their logits.  The
// backward writes P q for every column (EPI_KD_GRAD) and a small kernel puts
// P q - p, formed in fp32 from the kept logits and rounded once, at the
// entries.  No n x V logits: one n x c_v bf16 block.
// Bound by the tensor cores: 2 n h V FLOPs forward, 6 backward.  8000 rows of
// 2560 against 50257 words, 32 entries: 5.5 ms for both (1500 TFLOP/s).
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>

#include "../../include/bpt.h"
#include "internal.h"
#include "ptx.cuh"

namespace bpt {

namespace {

constexpr int TILE_N = 256;
constexpr int PART = 128;  // columns of one (max, sum) pair
constexpr int MAX_K = 128;
constexpr int NO_ID = 0x7fffffff;

struct KdDims {
  int64_t n, h, V, cv, nparts, nblk, k;
  int teacher;
  float T;
  bool det, debug, accum, f32;
};

int kd_validate(const bpt_distill_config* c, KdDims* D) {
  if (!c) return BPT_EINVAL;
  if (c->n < 1 || c->h < 8 || (c->h % 8) || c->vocab < 1) return BPT_EINVAL;
  if (c->vocab_block < 0 || (c->vocab_block % TILE_N)) return BPT_EINVAL;
  if (c->top_k < 1 || c->top_k > MAX_K) return BPT_EINVAL;
  if (c->teacher != BPT_TEACHER_LOGITS && c->teacher != BPT_TEACHER_LOGPROBS) return BPT_EINVAL;
  if (c->grads_dtype != BPT_DTYPE_F32 && c->grads_dtype != BPT_DTYPE_BF16) return BPT_EINVAL;
  if (!(c->temperature >= 0x1p-10f && c->temperature <= 0x1p10f)) return BPT_EINVAL;
  if (c->flags & ~(BPT_FLAG_ACCUM_GRADS | BPT_FLAG_DETERMINISTIC | BPT_FLAG_DEBUG_CHECKS)) return BPT_EINVAL;
  D->n = c->n;
  D->h = c->h;
  D->V = c->vocab;
  D->k = c->top_k;
  D->teacher = c->teacher;
  D->T = c->temperature;
  const int64_t vpad = (D->V + TILE_N - 1) / TILE_N * TILE_N;
  D->cv = c->vocab_block ? std::min<int64_t>(c->vocab_block, vpad) : std::min<int64_t>(8192, vpad);
  D->nparts = vpad / PART;
  D->nblk = (D->V + D->cv - 1) / D->cv;
  D->det = (c->flags & BPT_FLAG_DETERMINISTIC) != 0;
  D->debug = (c->flags & BPT_FLAG_DEBUG_CHECKS) != 0;
  D->accum = (c->flags & BPT_FLAG_ACCUM_GRADS) != 0;
  D->f32 = c->grads_dtype == BPT_DTYPE_F32;
  if (D->accum && !D->f32) return BPT_EINVAL;  // a running sum is not kept in 8 bits of mantissa
  return BPT_OK;
}

struct Planner {
  uint8_t* base;
  size_t off = 0;
  template <class T>
  T* take(int64_t count) {
    T* p = base ? reinterpret_cast<T*>(base + off) : nullptr;
    off += ((size_t)count * sizeof(T) + 255) / 256 * 256;
    return p;
  }
};

// What the forward leaves for the backward (and its own later steps).
struct Saved {
  int* id;            // [n, k] entries' columns, rising; NO_ID: none
  float* p;           // [n, k] their probabilities
  float* z;           // [n, k] the student's logits / T there
  float *lse, *mass;  // [n]
  float* ent;         // [n] sum p log p
  unsigned char* at;  // [nparts + 1, n] first entry at or past each 128 columns
};
size_t plan_saved(const KdDims& D, void* base, Saved* s) {
  Planner pl{reinterpret_cast<uint8_t*>(base)};
  s->id = pl.take<int>(D.n * D.k);
  s->p = pl.take<float>(D.n * D.k);
  s->z = pl.take<float>(D.n * D.k);
  s->lse = pl.take<float>(D.n);
  s->mass = pl.take<float>(D.n);
  s->ent = pl.take<float>(D.n);
  s->at = pl.take<unsigned char>((D.nparts + 1) * D.n);
  return pl.off;
}
struct FwdWs {
  float2* part;
  double* term;
};
size_t plan_fwd(const KdDims& D, void* base, FwdWs* w) {
  Planner pl{reinterpret_cast<uint8_t*>(base)};
  w->part = pl.take<float2>(D.nparts * D.n);
  w->term = pl.take<double>(D.n);
  return pl.off;
}
// K ranges of dx = dz W that run side by side: a product of few tiles over
// thousands of words would leave most SMs idle (100 rows of 256 against 5000
// words took 36 us in one tile).  Each range's product has a place of its own
// and they are added in order, so the sum does not depend on the run.
int dx_slabs(const KdDims& D, int64_t nv) {
  const int64_t tiles = ((D.n + 255) / 256) * ((D.h + 255) / 256), kt = (nv + 63) / 64;
  const int want = tiles <= 9 ? 8 : tiles <= 19 ? 4 : tiles <= 38 ? 2 : 1;
  return (int)std::max<int64_t>(1, std::min<int64_t>(want, kt / 4));
}

struct BwdWs {
  __nv_bfloat16* dz;
  float *dx_acc, *slabs;
};
size_t plan_bwd(const KdDims& D, void* base, BwdWs* w) {
  Planner pl{reinterpret_cast<uint8_t*>(base)};
  w->dz = pl.take<__nv_bfloat16>(D.n * D.cv);
  w->dx_acc = D.nblk > 1 ? pl.take<float>(D.n * D.h) : nullptr;
  const int s = dx_slabs(D, std::min(D.cv, D.V));
  w->slabs = s > 1 ? pl.take<float>(s * D.n * D.h) : nullptr;
  return pl.off;
}

// The teacher's entries of 32 rows a block, a warp a row at a time: their
// probabilities, sorted by (id, place); then, a lane a row, where each 128
// columns' entries begin.
struct PrepParams {
  const int* ids;
  const float* v;
  int64_t n, V, nparts;
  int k, teacher;
  float inv_t;
  Saved s;
  unsigned int* err;
};
constexpr int PREP_ROWS = 32, PREP_WARPS = 32;  // a row a warp: 59 us for 4001 rows of 64 entries with 8 warps

template <int C>  // entries a lane holds
__global__ void __launch_bounds__(32 * PREP_WARPS) prepare_kernel(const PrepParams q) {
  extern __shared__ int s_id[];  // [PREP_ROWS][k | 1]
  const int lane = lane_id(), warp = warp_id();
  const int ld = q.k | 1;
  const int64_t r0 = (int64_t)blockIdx.x * PREP_ROWS;
  wait_for_previous();
  let_next_start();
  static_assert(PREP_ROWS == PREP_WARPS, "a row a warp");
  if (const int64_t row = r0 + warp; row < q.n) {
    const int i = warp;
    int id[C], rank[C];
    float v[C];
    float m = -INFINITY;
    bool bad = false;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = c * 32 + lane;
      id[c] = NO_ID;
      rank[c] = 0;
      v[c] = -INFINITY;
      if (j < q.k) {
        const int t = q.ids[row * q.k + j];
        const float x = q.v[row * q.k + j];
        if (t >= 0) {
          if ((int64_t)t < q.V && x < INFINITY) {
            id[c] = t;
            v[c] = x;
          } else {
            bad = true;
          }
        }
      }
      m = fmaxf(m, v[c]);
    }
    if (bad) report_bad_data(q.err, BPT_DISTILL_BAD_ENTRY_SITE);
    float total = 1.f;
    if (q.teacher == BPT_TEACHER_LOGITS) {
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
      if (m == -INFINITY) m = 0.f;
      total = 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        v[c] = (v[c] - m) * q.inv_t;  // the difference first: values / T may be beyond fp32, or have no digits left for it
        total += expf(v[c]);
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
    }
    const float log_total = total > 0.f ? logf(total) : 0.f;
    float mass = 0.f, ent = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float lp = v[c] - log_total;
      const float p = expf(lp);
      v[c] = p;
      mass += p;
      ent += p > 0.f ? p * lp : 0.f;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      mass += __shfl_xor_sync(0xffffffffu, mass, d);
      ent += __shfl_xor_sync(0xffffffffu, ent, d);
    }
    if (lane == 0) {
      q.s.mass[row] = mass;
      q.s.ent[row] = ent;
    }
    // an entry's rank: how many come before it
#pragma unroll
    for (int o = 0; o < C; ++o) {
      if (o * 32 >= q.k) break;
      for (int l = 0; l < min(32, q.k - o * 32); ++l) {
        const int other = __shfl_sync(0xffffffffu, id[o], l);
#pragma unroll
        for (int c = 0; c < C; ++c) rank[c] += other < id[c] || (other == id[c] && o * 32 + l < c * 32 + lane);
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (c * 32 + lane < q.k) {
        s_id[i * ld + rank[c]] = id[c];
        q.s.id[row * q.k + rank[c]] = id[c];
        q.s.p[row * q.k + rank[c]] = v[c];
      }
  }
  __syncthreads();
  const int64_t row = r0 + lane;
  if (row >= q.n) return;
  const int* mine = s_id + lane * ld;
  for (int64_t part = warp; part <= q.nparts; part += PREP_WARPS) {
    const int64_t col = part * PART;
    int lo = 0, hi = q.k;  // the first entry at or past col
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (mine[mid] < col) lo = mid + 1;
      else hi = mid;
    }
    // the last part's end leaves out what is no entry
    q.s.at[part * q.n + row] = (unsigned char)lo;
  }
}

// Rows' log-sum-exp from their pairs, 32 rows a block with the parts in 32
// slices, and their terms of the loss, sum p z by a warp a row.
struct RowParams {
  const float2* part;
  int64_t n, nparts;
  int k;
  float scale;  // T^2, over n without row weights
  const float* weight;
  Saved s;
  double* term;
};
constexpr int ROW_SLICES = 32;
__global__ void __launch_bounds__(32 * ROW_SLICES) rows_kernel(const RowParams q) {
  wait_for_previous();
  let_next_start();
  __shared__ float s_m[ROW_SLICES][32], s_l[ROW_SLICES][32], s_dot[32];
  const int lane = lane_id(), sl = warp_id();
  const int64_t r0 = (int64_t)blockIdx.x * 32, row = r0 + lane;
  const bool in = row < q.n;
  float m = -INFINITY, l = 0.f;
  for (int64_t p0 = sl; p0 < q.nparts; p0 += 8 * ROW_SLICES) {
    // eight pairs on their way at once; those past the last are (-inf, 0) like
    // the pairs of columns past the vocabulary
    float2 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t p = p0 + i * ROW_SLICES;
      v[i] = in && p < q.nparts ? q.part[p * q.n + row] : make_float2(-INFINITY, 0.f);
    }
    float top = m;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, v[i].x);
    if (top > -INFINITY) {
      l *= expf(m - top);
#pragma unroll
      for (int i = 0; i < 8; ++i) l += v[i].y * expf(v[i].x - top);
      m = top;
    }
  }
  s_m[sl][lane] = m;
  s_l[sl][lane] = l;
  static_assert(ROW_SLICES == 32, "a warp a row");
  float dot = 0.f;
  if (r0 + sl < q.n)
    for (int j = lane; j < q.k; j += 32) {
      const int64_t at = (r0 + sl) * q.k + j;
      const float p = q.s.p[at], z = q.s.z[at];  // z holds nothing where there is no entry
      dot += p > 0.f ? p * z : 0.f;
    }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
  if (lane == 0) s_dot[sl] = dot;
  __syncthreads();
  if (sl || !in) return;
  float top = s_m[0][lane];
#pragma unroll
  for (int i = 1; i < ROW_SLICES; ++i) top = fmaxf(top, s_m[i][lane]);
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < ROW_SLICES; ++i) sum += s_l[i][lane] * expf(s_m[i][lane] - top);
  const float lse = top + logf(sum);
  q.s.lse[row] = lse;
  const float w = q.weight ? q.weight[row] : 1.f;
  // the divergence is a small difference of these: in fp64
  q.term[row] =
      w != 0.f && q.s.mass[row] != 0.f ? (double)q.scale * w * ((double)q.s.ent[row] - (double)s_dot[lane] + (double)q.s.mass[row] * lse) : 0.0;
}

// loss = the rows' terms, added in a fixed order
__global__ void __launch_bounds__(1024) total_kernel(int64_t n, const double* term, float* loss) {
  __shared__ double acc[32];
  wait_for_previous();
  let_next_start();
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += 1024) s += term[i];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  if (lane_id() == 0) acc[warp_id()] = s;
  __syncthreads();
  if (warp_id()) return;
  s = acc[lane_id()];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  if (threadIdx.x == 0) *loss = (float)s;
}

// dz at the entries of columns [v0, v1): T dloss c (P q - p), the p of an id
// that appears more than once added up by the first of them.
__global__ void __launch_bounds__(256) entries_kernel(int64_t n, int k, int64_t v0, int64_t v1, const Saved s, const float* weight,
                                                      float scale, __nv_bfloat16* dz, int64_t ld) {
  wait_for_previous();
  let_next_start();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n * k) return;
  const int id = s.id[i];
  if (id < v0 || id >= v1) return;
  const int64_t row = i / k;
  const int j = (int)(i - row * k);
  if (j > 0 && s.id[i - 1] == id) return;
  float p = s.p[i];
  for (int o = 1; j + o < k && s.id[i + o] == id; ++o) p += s.p[i + o];
  const float w = scale * (weight ? weight[row] : 1.f);
  const float q = expf(s.z[i] - s.lse[row]);
  // a row without mass gives nothing, whatever its logits (and q) are
  const float mass = s.mass[row];
  dz[row * ld + (id - v0)] = __float2bfloat16(w != 0.f && mass != 0.f ? w * (mass * q - p) : 0.f);
}

// sum over the slabs in order, onto acc (NULL: 0): fp32 out, or bf16
__global__ void __launch_bounds__(256) slabs_kernel(int64_t n4, int slabs, const float4* s, const float4* acc, float4* out_f32,
                                                    uint2* out_bf16) {
  wait_for_previous();
  let_next_start();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n4) return;
  float4 t = acc ? acc[i] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int q = 0; q < slabs; ++q) {
    const float4 v = s[q * n4 + i];
    t.x += v.x, t.y += v.y, t.z += v.z, t.w += v.w;
  }
  if (out_f32) out_f32[i] = t;
  else out_bf16[i] = make_uint2(pack_bf16(t.x, t.y), pack_bf16(t.z, t.w));
}

bool al(const void* p, int a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace
}  // namespace bpt

using namespace bpt;

extern "C" {

size_t bpt_lm_distill_saved_bytes(const bpt_distill_config* cfg) {
  KdDims D;
  if (kd_validate(cfg, &D)) return 0;
  Saved s;
  return plan_saved(D, nullptr, &s);
}

size_t bpt_lm_distill_workspace_bytes(const bpt_distill_config* cfg, int pass) {
  KdDims D;
  if (kd_validate(cfg, &D)) return 0;
  FwdWs f;
  BwdWs b;
  return pass == BPT_PASS_FWD ? plan_fwd(D, nullptr, &f) : pass == BPT_PASS_BWD ? plan_bwd(D, nullptr, &b) : 0;
}

int bpt_lm_distill_fwd(const bpt_distill_config* cfg, const void* x, const void* w, const int32_t* ids, const float* teacher,
                       const float* row_weight, float* loss, void* saved, void* ws, size_t ws_bytes, void* stream) {
  KdDims D;
  int rc = kd_validate(cfg, &D);
  if (rc) return rc;
  if (!x || !w || !ids || !teacher || !loss || !saved || !ws) return BPT_EINVAL;
  if (!al(x, 16) || !al(w, 16) || !al(ids, 4) || !al(teacher, 4) || !al(row_weight, 4) || !al(loss, 4) || !al(saved, 16) || !al(ws, 16))
    return BPT_EINVAL;
  FwdWs W;
  Saved S;
  const size_t need = plan_fwd(D, nullptr, &W), keep = plan_saved(D, nullptr, &S);
  if (ws_bytes < need) return BPT_ENOSPC;
  const Span sp[] = {{x, D.n * D.h * 2}, {w, D.V * D.h * 2}, {ids, D.n * D.k * 4}, {teacher, D.n * D.k * 4},
                     {row_weight, row_weight ? D.n * 4 : 0}, {loss, 4}, {saved, (int64_t)keep}, {ws, (int64_t)need}};
  for (int i = 5; i < 8; ++i)
    if (overlaps(sp[i], sp, i)) return BPT_EINVAL;
  if (D.debug && debug_spans(sp, 8)) return BPT_EINVAL;
  plan_fwd(D, ws, &W);
  plan_saved(D, saved, &S);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  unsigned int* err = device_error_word();
  if (!err) return BPT_ECUDA;
  {
    PrepParams q{ids, teacher, D.n, D.V, D.nparts, (int)D.k, D.teacher, 1.f / D.T, S, err};
    ProfScope prof(PROF_MISC, 0.0, (double)D.n * (20.0 * D.k + D.nparts), st);
    const size_t smem = (size_t)PREP_ROWS * (D.k | 1) * 4;
    auto k = D.k <= 32 ? prepare_kernel<1> : D.k <= 64 ? prepare_kernel<2> : prepare_kernel<4>;
    if (launch_dependent(k, (int)((D.n + PREP_ROWS - 1) / PREP_ROWS), 1, dim3(32 * PREP_WARPS), smem, st, q) != cudaSuccess)
      return BPT_ECUDA;
  }
  {
    MatView A{x, D.n, D.h, D.h};
    MatView B{w, D.V, D.h, D.h};
    Epilogue e;
    e.kind = EPI_KD_LSE;
    e.out = W.part;
    e.ldo = D.n;
    e.out2 = S.z;
    e.ent_id = S.id;
    e.ent_at = S.at;
    e.ent_k = (int)D.k;
    e.inv_t = 1.f / D.T;
    const int64_t K = D.h;
    if ((rc = gemm(D.n, D.V, D.h, A, false, &B, &K, 1, false, nullptr, e, st))) return rc;
  }
  {
    ProfScope prof(PROF_MISC, 0.0, (double)D.n * (D.nparts * 8.0 + 8.0 * D.k), st);
    const float scale = row_weight ? D.T * D.T : D.T * D.T / (float)D.n;
    RowParams q{W.part, D.n, D.nparts, (int)D.k, scale, row_weight, S, W.term};
    if (launch_dependent(rows_kernel, (int)((D.n + 31) / 32), 1, dim3(32 * ROW_SLICES), 0, st, q) != cudaSuccess) return BPT_ECUDA;
    if (launch_dependent(total_kernel, 1, 1, dim3(1024), 0, st, D.n, (const double*)W.term, loss) != cudaSuccess) return BPT_ECUDA;
  }
  return D.debug ? debug_finish(st) : BPT_OK;
}

int bpt_lm_distill_bwd(const bpt_distill_config* cfg, const void* x, const void* w, const float* row_weight, const void* saved,
                       float dloss, void* dx, void* dw, void* ws, size_t ws_bytes, void* stream) {
  KdDims D;
  int rc = kd_validate(cfg, &D);
  if (rc) return rc;
  if (!x || !w || !saved || !dx || !dw || !ws) return BPT_EINVAL;
  if (!al(x, 16) || !al(w, 16) || !al(row_weight, 4) || !al(saved, 16) || !al(dx, 16) || !al(dw, 16) || !al(ws, 16)) return BPT_EINVAL;
  if (!(fabsf(dloss) < INFINITY)) return BPT_EINVAL;
  BwdWs W;
  Saved S;
  const size_t need = plan_bwd(D, nullptr, &W), keep = plan_saved(D, nullptr, &S);
  if (ws_bytes < need) return BPT_ENOSPC;
  const int64_t elem = D.f32 ? 4 : 2;
  const Span sp[] = {{x, D.n * D.h * 2}, {w, D.V * D.h * 2}, {row_weight, row_weight ? D.n * 4 : 0}, {saved, (int64_t)keep},
                     {dx, D.n * D.h * 2}, {dw, D.V * D.h * elem}, {ws, (int64_t)need}};
  for (int i = 4; i < 7; ++i)
    if (overlaps(sp[i], sp, i)) return BPT_EINVAL;
  if (D.debug && debug_spans(sp, 7)) return BPT_EINVAL;
  plan_bwd(D, ws, &W);
  plan_saved(D, const_cast<void*>(saved), &S);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const float scale = row_weight ? D.T * dloss : D.T * dloss / (float)D.n;
  for (int64_t b = 0; b < D.nblk; ++b) {
    const int64_t v0 = b * D.cv, nv = std::min(D.cv, D.V - v0);
    const void* wb = reinterpret_cast<const uint8_t*>(w) + v0 * D.h * 2;
    const int64_t K = D.h, Kn = D.n, Kv = nv;
    MatView X{x, D.n, D.h, D.h}, Wb{wb, nv, D.h, D.h}, Z{W.dz, D.n, nv, D.cv};
    {
      Epilogue e;
      e.kind = EPI_KD_GRAD;
      e.out = W.dz;
      e.ldo = D.cv;
      e.rowf = S.lse;
      e.rowp = S.mass;
      e.roww = row_weight;
      e.scale = scale;
      e.inv_t = 1.f / D.T;
      if ((rc = gemm(D.n, nv, D.h, X, false, &Wb, &K, 1, false, nullptr, e, st))) return rc;
    }
    {
      ProfScope prof(PROF_MISC, 0.0, 4.0 * (double)D.n * D.k, st);
      if (launch_dependent(entries_kernel, (int)((D.n * D.k + 255) / 256), 1, dim3(256), 0, st, D.n, (int)D.k, v0, v0 + nv, S, row_weight,
                           scale, W.dz, D.cv) != cudaSuccess)
        return BPT_ECUDA;
    }
    {
      Epilogue e;
      e.kind = D.f32 ? EPI_F32 : EPI_BF16;
      e.out = reinterpret_cast<uint8_t*>(dw) + v0 * D.h * elem;
      e.ldo = D.h;
      e.beta = D.accum ? 1.f : 0.f;
      e.deterministic = D.det;
      if ((rc = gemm(nv, D.h, D.n, Z, true, &X, &Kn, 1, true, nullptr, e, st))) return rc;
    }
    const int slabs = dx_slabs(D, nv);
    const bool last = b == D.nblk - 1;
    if (slabs > 1) {
      Epilogue e;
      e.kind = EPI_SLABS;
      e.out = W.slabs;
      e.ldo = D.h;
      e.slabs = slabs;
      e.slab = D.n * D.h;
      if ((rc = gemm(D.n, D.h, nv, Z, false, &Wb, &Kv, 1, true, nullptr, e, st))) return rc;
      const int64_t n4 = D.n * D.h / 4;
      ProfScope prof(PROF_MISC, 0.0, 16.0 * (double)n4 * (slabs + 1), st);
      if (launch_dependent(slabs_kernel, (int)((n4 + 255) / 256), 1, dim3(256), 0, st, n4, slabs,
                           reinterpret_cast<const float4*>(W.slabs),
                           b > 0 ? reinterpret_cast<const float4*>(W.dx_acc) : (const float4*)nullptr,
                           last ? (float4*)nullptr : reinterpret_cast<float4*>(W.dx_acc), reinterpret_cast<uint2*>(dx)) != cudaSuccess)
        return BPT_ECUDA;
    } else {
      // dx: fp32 over the blocks, the last one rounds to bf16
      Epilogue e;
      e.deterministic = D.det;
      e.ldo = D.h;
      if (last) {
        e.kind = EPI_BF16;
        e.out = dx;
        if (b > 0) {
          e.res = W.dx_acc;
          e.res_f32 = 1;
          e.ldr = D.h;
        }
      } else {
        e.kind = EPI_F32;
        e.out = W.dx_acc;
        e.beta = b > 0 ? 1.f : 0.f;
      }
      if ((rc = gemm(D.n, D.h, nv, Z, false, &Wb, &Kv, 1, true, nullptr, e, st))) return rc;
    }
  }
  return D.debug ? debug_finish(st) : BPT_OK;
}

}  // extern "C"
