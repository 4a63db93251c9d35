// moe_ffn.cu -- the feed-forward network of a mixture-of-experts layer, over
// the rows as the router left them, and the public products over ragged
// groups.
//
//   y_t = sum_j w_tj W2_e act(x_t W1_e^T [, x_t W3_e^T]),  e = ids[t, j]
//
// Forward, in the groups' order of the pairs (moe_route.cu): the first product
// gathers the rows of x by copying warps and applies the activation in its
// epilogue, the second multiplies by W2, and a last pass adds each position's k
// rows with their weights.  Backward, with da = dy W2 (dy gathered):
//   dg, du = w da dact/dg, dact/du    aw = w act    dw = <act, da>   (epilogue)
//   dx rows = dg W1 + du W3 (one accumulator), added over the k choices
//   dW1 = dg^T x, dW3 = du^T x (x gathered), dW2 = dy^T aw (dy gathered)
// The weight's own gradient <W2 act, dy> is taken as <act, dy W2>, so the
// second product is not formed again.
//
// Between the kernels act, dg, du, aw and the rows before the last sum are
// bf16 (2^-9 of each value on average less): the tensor core's operands.
// Every sum is fp32 in a fixed order: no atomics.
//
// Bound by the tensor cores: 4096 rows, 2 of 8 experts of 4096 x 14336, 1.9 ms
// forward and 3.9 backward (in one call after another 6.7 ms in all, under the
// power cap: 1290 TFLOP/s); a few rows by the weights' bytes (48 rows over 32
// experts of 2560 x 2048: 158 us, 6.4 TB/s).
#include <math.h>

#include <algorithm>

#include "../../include/bpt.h"
#include "gemm_kernel.cuh"
#include "grouped.h"
#include "internal.h"
#include "moe.h"
#include "ptx.cuh"

namespace bpt {

int moe_dims(const bpt_moe_config* c, MoeDims* D) {
  if (!c) return BPT_EINVAL;
  if (c->n < 1 || c->h < 8 || (c->h % 8) || c->ffn_dim < 8 || (c->ffn_dim % 8)) return BPT_EINVAL;
  if (c->n_experts < 1 || c->n_experts > GROUPED_MAX_GROUPS || c->top_k < 1 || c->top_k > 32 || c->top_k > c->n_experts) return BPT_EINVAL;
  if (c->act < BPT_ACT_GELU_ERF || c->act > BPT_ACT_SWIGLU) return BPT_EINVAL;
  for (int32_t t : {c->logits_dtype, c->weights_dtype, c->grads_dtype})
    if (t != BPT_DTYPE_F32 && t != BPT_DTYPE_BF16) return BPT_EINVAL;
  if (c->norm_topk != 0 && c->norm_topk != 1) return BPT_EINVAL;
  if (!(fabsf(c->balance_coef) < INFINITY) || !(fabsf(c->z_coef) < INFINITY)) return BPT_EINVAL;
  if (c->flags & ~(BPT_FLAG_ACCUM_GRADS | BPT_FLAG_DETERMINISTIC | BPT_FLAG_DEBUG_CHECKS)) return BPT_EINVAL;
  D->n = c->n;
  D->h = c->h;
  D->f = c->ffn_dim;
  D->E = c->n_experts;
  D->k = c->top_k;
  D->pairs = D->n * D->k;
  D->act = c->act;
  D->logit_bytes = c->logits_dtype == BPT_DTYPE_F32 ? 4 : 2;
  D->weight_bytes = c->weights_dtype == BPT_DTYPE_F32 ? 4 : 2;
  D->grads_f32 = c->grads_dtype == BPT_DTYPE_F32;
  D->debug = (c->flags & BPT_FLAG_DEBUG_CHECKS) != 0;
  D->accum = (c->flags & BPT_FLAG_ACCUM_GRADS) != 0;
  if (D->accum && !D->grads_f32) return BPT_EINVAL;  // a running sum is not kept in 8 bits of mantissa
  if (D->pairs > (int64_t(1) << 26)) return BPT_EUNSUPPORTED;
  return BPT_OK;
}

namespace {

// One sum over each position's choices: out[t, :] = sum_j w_tj rows[slot_tj, :]
// (w NULL: 1), j in order.  8 columns a thread; behind those blocks, with
// `part`, the weights' gradients: dw[pair] = sum over the parts in order.  Rows
// that no expert's offsets hold were not written: their pairs add nothing.
struct CombineParams {
  const __nv_bfloat16* rows;
  const int *slot, *offsets;
  const void* weight;
  int weight_f32;
  __nv_bfloat16* out;
  int64_t n, pairs;
  int h8, k, E;
  const int2* span;  // rows that the offsets hold; x < 0: some of them are bad
  int64_t blocks;  // of the sum
  const float* part;
  int nparts;
  void* dweight;
};

constexpr int CT = 128;

// The same where some offsets are bad, one value at a time: rows of the groups
// that are left.
static __device__ __noinline__ void combine_odd(const CombineParams& p) {
  auto row = [&](int64_t q) {  // of pair q; -1: none
    const int at = p.slot[q];
    return group_of(p.offsets, p.E, p.pairs, at) < p.E ? at : -1;
  };
  if (blockIdx.x < p.blocks) {
    const int64_t i = (int64_t)blockIdx.x * CT + threadIdx.x;
    if (i >= p.n * p.h8) return;
    const int64_t t = i / p.h8, c = (i - t * p.h8) * 8;
    for (int q = 0; q < 8; ++q) {
      float s = 0.f;
      for (int64_t j = t * p.k; j < (t + 1) * p.k; ++j) {
        const int at = row(j);
        const float w = !p.weight     ? 1.f
                        : p.weight_f32 ? reinterpret_cast<const float*>(p.weight)[j]
                                       : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.weight)[j]);
        if (at >= 0) s = fmaf(w, __bfloat162float(p.rows[at * (int64_t)p.h8 * 8 + c + q]), s);
      }
      p.out[i * 8 + q] = __float2bfloat16(s);
    }
    return;
  }
  const int64_t q = ((int64_t)blockIdx.x - p.blocks) * CT + threadIdx.x;
  if (q >= p.pairs) return;
  const int at = row(q);
  float s = 0.f;
  for (int i = 0; i < p.nparts && at >= 0; ++i) s += p.part[(int64_t)i * p.pairs + at];
  if (p.weight_f32) reinterpret_cast<float*>(p.dweight)[q] = s;
  else reinterpret_cast<__nv_bfloat16*>(p.dweight)[q] = __float2bfloat16(s);
}

template <int ROWS>
__global__ void __launch_bounds__(CT) combine_kernel(const __grid_constant__ CombineParams p) {
  wait_for_previous();
  let_next_start();
  const int2 span = *p.span;
  if (span.x < 0) return combine_odd(p);
  if (blockIdx.x < p.blocks) {
    const int64_t i = (int64_t)blockIdx.x * CT + threadIdx.x;
    if (i >= p.n * p.h8) return;
    const int64_t t = i / p.h8;
    const int c = (int)(i - t * p.h8);
    float s[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) s[q] = 0.f;
    const int* slot = p.slot + t * p.k;
    for (int j0 = 0; j0 < p.k; j0 += ROWS) {
      // ROWS rows on their way at once
      int at[ROWS];
      uint4 u[ROWS];
      float w[ROWS];
#pragma unroll
      for (int j = 0; j < ROWS; ++j) at[j] = j0 + j < p.k ? slot[j0 + j] : -1;
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        const bool some = at[j] >= span.x && at[j] < span.y;
        // without a row: the first one, not used
        asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(u[j].x), "=r"(u[j].y), "=r"(u[j].z), "=r"(u[j].w)
                     : "l"(reinterpret_cast<const uint4*>(p.rows) + (some ? at[j] : 0) * (int64_t)p.h8 + c));
        w[j] = !some         ? 0.f
               : !p.weight   ? 1.f
               : p.weight_f32 ? reinterpret_cast<const float*>(p.weight)[t * p.k + j0 + j]
                              : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.weight)[t * p.k + j0 + j]);
      }
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        const bool some = at[j] >= span.x && at[j] < span.y;
        const uint32_t v[4] = {some ? u[j].x : 0u, some ? u[j].y : 0u, some ? u[j].z : 0u, some ? u[j].w : 0u};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          s[2 * q] = fmaf(w[j], bf16_lo(v[q]), s[2 * q]);
          s[2 * q + 1] = fmaf(w[j], bf16_hi(v[q]), s[2 * q + 1]);
        }
      }
    }
    uint4 o;
    o.x = pack_bf16(s[0], s[1]);
    o.y = pack_bf16(s[2], s[3]);
    o.z = pack_bf16(s[4], s[5]);
    o.w = pack_bf16(s[6], s[7]);
    reinterpret_cast<uint4*>(p.out)[i] = o;
    return;
  }
  const int64_t q = ((int64_t)blockIdx.x - p.blocks) * CT + threadIdx.x;
  if (q >= p.pairs) return;
  const int at = p.slot[q];
  float s = 0.f;
  if (at >= span.x && at < span.y)
    for (int i = 0; i < p.nparts; ++i) s += p.part[(int64_t)i * p.pairs + at];
  if (p.weight_f32) reinterpret_cast<float*>(p.dweight)[q] = s;
  else reinterpret_cast<__nv_bfloat16*>(p.dweight)[q] = __float2bfloat16(s);
}

int combine(const MoeDims& D, const void* rows, const bpt_moe_route* r, const int2* span, const void* weight, void* out, const float* part,
            int nparts, void* dweight, cudaStream_t st) {
  CombineParams p;
  p.rows = reinterpret_cast<const __nv_bfloat16*>(rows);
  p.slot = r->slot;
  p.offsets = r->offsets;
  p.span = span;
  p.weight = weight;
  p.weight_f32 = D.weight_bytes == 4;
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.n = D.n;
  p.pairs = D.pairs;
  p.h8 = (int)(D.h / 8);
  p.k = (int)D.k;
  p.E = (int)D.E;
  p.blocks = (D.n * p.h8 + CT - 1) / CT;
  p.part = part;
  p.nparts = nparts;
  p.dweight = dweight;
  const int64_t grid = p.blocks + (part ? (D.pairs + CT - 1) / CT : 0);
  if (grid > INT32_MAX) return BPT_EUNSUPPORTED;
  ProfScope prof(PROF_MISC, 0.0, 2.0 * (double)(D.pairs + D.n) * D.h, st);
  auto kern = D.k <= 2 ? combine_kernel<2> : D.k <= 4 ? combine_kernel<4> : combine_kernel<8>;
  return launch_dependent(kern, (int)grid, 1, dim3(CT), 0, st, p) == cudaSuccess ? BPT_OK : BPT_ECUDA;
}

struct Planner {
  uint8_t* base;
  size_t off = 0;
  void* take(int64_t bytes) {
    void* p = base ? base + off : nullptr;
    off += ((size_t)bytes + 255) / 256 * 256;
    return p;
  }
};

// What the backward takes back: SwiGLU the gate and up products, GeLU the
// product; pairs * f bf16 values each, in the grouped GEMM's own layout.
struct Saved {
  void *s0, *s1;
};
size_t plan_saved(const MoeDims& D, void* base, Saved* s) {
  Planner pl{reinterpret_cast<uint8_t*>(base)};
  s->s0 = pl.take(D.pairs * D.f * 2);
  s->s1 = D.act == BPT_ACT_SWIGLU ? pl.take(D.pairs * D.f * 2) : nullptr;
  return pl.off;
}
struct FwdWs {
  void *act, *ys;
  int2* span;
};
size_t plan_fwd(const MoeDims& D, void* base, FwdWs* w) {
  Planner pl{reinterpret_cast<uint8_t*>(base)};
  w->act = pl.take(D.pairs * D.f * 2);
  w->ys = pl.take(D.pairs * D.h * 2);
  w->span = reinterpret_cast<int2*>(pl.take(8));
  return moe_few_rows(D) ? std::max(pl.off, moe_few_ws_bytes(D)) : pl.off;
}
struct BwdWs {
  void *dg, *du, *aw, *dxs;
  float* part;
  int2* span;
};
size_t plan_bwd(const MoeDims& D, void* base, BwdWs* w) {
  Planner pl{reinterpret_cast<uint8_t*>(base)};
  w->dg = pl.take(D.pairs * D.f * 2);
  w->du = D.act == BPT_ACT_SWIGLU ? pl.take(D.pairs * D.f * 2) : nullptr;
  w->aw = pl.take(D.pairs * D.f * 2);
  w->dxs = pl.take(D.pairs * D.h * 2);
  w->part = reinterpret_cast<float*>(pl.take(2 * grouped_part_tiles(D.f) * D.pairs * 4));
  w->span = reinterpret_cast<int2*>(pl.take(8));
  return pl.off;
}

bool al(const void* p, int a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

GroupedOp op_base(const MoeDims& D, const bpt_moe_route* r) {
  GroupedOp op;
  op.rows = D.pairs;
  op.groups = (int)D.E;
  op.offsets = r->offsets;
  op.mean_rows = D.pairs / D.E;
  op.top_k = (int)D.k;
  op.act = D.act;
  return op;
}

bool route_ok(const bpt_moe_route* r) {
  return r && r->weights && r->offsets && r->order && r->slot && al(r->weights, 4) && al(r->offsets, 4) && al(r->order, 4) && al(r->slot, 4);
}

}  // namespace
}  // namespace bpt

using namespace bpt;

extern "C" {

size_t bpt_moe_saved_bytes(const bpt_moe_config* cfg) {
  MoeDims D;
  if (moe_dims(cfg, &D)) return 0;
  Saved s;
  return plan_saved(D, nullptr, &s);
}

size_t bpt_moe_ffn_workspace_bytes(const bpt_moe_config* cfg, int pass) {
  MoeDims D;
  if (moe_dims(cfg, &D)) return 0;
  FwdWs f;
  BwdWs b;
  return pass == BPT_PASS_FWD ? plan_fwd(D, nullptr, &f) : pass == BPT_PASS_BWD ? plan_bwd(D, nullptr, &b) : 0;
}

int bpt_moe_ffn_fwd(const bpt_moe_config* cfg, const bpt_moe_route* r, const void* x, const void* w1, const void* w3, const void* w2,
                    void* y, void* saved, void* ws, size_t ws_bytes, void* stream) {
  MoeDims D;
  int rc = moe_dims(cfg, &D);
  if (rc) return rc;
  const bool swiglu = D.act == BPT_ACT_SWIGLU;
  if (!route_ok(r) || !x || !w1 || !w2 || (w3 != nullptr) != swiglu || !y || !ws) return BPT_EINVAL;
  if (!al(x, 16) || !al(w1, 16) || !al(w3, 16) || !al(w2, 16) || !al(y, 16) || !al(saved, 16) || !al(ws, 16)) return BPT_EINVAL;
  FwdWs W;
  Saved S;
  const size_t need = plan_fwd(D, nullptr, &W), keep = plan_saved(D, nullptr, &S);
  if (ws_bytes < need) return BPT_ENOSPC;
  const int64_t mat = D.E * D.f * D.h * 2;
  const Span sp[] = {{r->weights, D.pairs * D.weight_bytes}, {r->offsets, (D.E + 2) * 4}, {r->order, D.pairs * 4},
                     {r->slot, D.pairs * 4}, {x, D.n * D.h * 2}, {w1, mat}, {w3, w3 ? mat : 0}, {w2, mat},
                     {y, D.n * D.h * 2}, {saved, saved ? (int64_t)keep : 0}, {ws, (int64_t)need}};
  for (int i = 8; i < 11; ++i)
    if (sp[i].p && overlaps(sp[i], sp, i)) return BPT_EINVAL;
  if (D.debug && debug_spans(sp, 11)) return BPT_EINVAL;
  plan_fwd(D, ws, &W);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (!saved && moe_few_rows(D)) {
    if ((rc = moe_few_fwd(D, r, x, w1, w3, w2, y, ws, st))) return rc;
    return D.debug ? debug_finish(st) : BPT_OK;
  }
  {
    GroupedOp op = op_base(D, r);
    op.form = GROUPED_NT;
    op.epi = GROUPED_ACT;
    op.N = D.f;
    op.K = D.h;
    op.a = x;
    op.a_rows = D.n;
    op.a_gather = true;
    op.order = r->order;
    op.w = w1;
    op.w2 = w3;
    op.out = W.act;
    if (saved) {
      plan_saved(D, saved, &S);
      op.out2 = S.s0;
      op.out3 = S.s1;
    }
    if ((rc = grouped_gemm(op, st))) return rc;
  }
  {
    GroupedOp op = op_base(D, r);
    op.form = GROUPED_NT;
    op.N = D.h;
    op.K = D.f;
    op.a = W.act;
    op.a_rows = D.pairs;
    op.w = w2;
    op.out = W.ys;
    op.span = W.span;
    if ((rc = grouped_gemm(op, st))) return rc;
  }
  if ((rc = combine(D, W.ys, r, W.span, r->weights, y, nullptr, 0, nullptr, st))) return rc;
  return D.debug ? debug_finish(st) : BPT_OK;
}

int bpt_moe_ffn_bwd(const bpt_moe_config* cfg, const bpt_moe_route* r, const void* x, const void* w1, const void* w3, const void* w2,
                    const void* saved, const void* dy, void* dx, void* dweights, void* dw1, void* dw3, void* dw2, void* ws,
                    size_t ws_bytes, void* stream) {
  MoeDims D;
  int rc = moe_dims(cfg, &D);
  if (rc) return rc;
  const bool swiglu = D.act == BPT_ACT_SWIGLU;
  if (!route_ok(r) || !x || !w1 || !w2 || (w3 != nullptr) != swiglu || (dw3 != nullptr) != swiglu || !saved || !dy || !dx || !dweights ||
      !dw1 || !dw2 || !ws)
    return BPT_EINVAL;
  for (const void* q : {x, w1, w3, w2, saved, dy, (const void*)dx, (const void*)dw1, (const void*)dw3, (const void*)dw2, (const void*)ws})
    if (!al(q, 16)) return BPT_EINVAL;
  if (!al(dweights, 4)) return BPT_EINVAL;
  BwdWs W;
  Saved S;
  const size_t need = plan_bwd(D, nullptr, &W), keep = plan_saved(D, nullptr, &S);
  if (ws_bytes < need) return BPT_ENOSPC;
  const int64_t mat = D.E * D.f * D.h * 2, grad = D.E * D.f * D.h * (D.grads_f32 ? 4 : 2);
  const Span sp[] = {{r->weights, D.pairs * D.weight_bytes}, {r->offsets, (D.E + 2) * 4}, {r->order, D.pairs * 4},
                     {r->slot, D.pairs * 4}, {x, D.n * D.h * 2}, {w1, mat}, {w3, w3 ? mat : 0}, {w2, mat}, {saved, (int64_t)keep},
                     {dy, D.n * D.h * 2}, {dx, D.n * D.h * 2}, {dweights, D.pairs * D.weight_bytes}, {dw1, grad}, {dw3, dw3 ? grad : 0},
                     {dw2, grad}, {ws, (int64_t)need}};
  for (int i = 10; i < 16; ++i)
    if (sp[i].p && overlaps(sp[i], sp, i)) return BPT_EINVAL;
  if (D.debug && debug_spans(sp, 16)) return BPT_EINVAL;
  plan_bwd(D, ws, &W);
  plan_saved(D, const_cast<void*>(saved), &S);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  {
    GroupedOp op = op_base(D, r);
    op.form = GROUPED_NN;
    op.epi = GROUPED_ACT_BWD;
    op.N = D.f;
    op.K = D.h;
    op.a = dy;
    op.a_rows = D.n;
    op.a_gather = true;
    op.order = r->order;
    op.w = w2;
    op.aux = S.s0;
    op.aux2 = S.s1;
    op.row_weight = r->weights;
    op.row_weight_f32 = D.weight_bytes == 4;
    op.out = W.dg;
    op.out2 = W.du;
    op.out3 = W.aw;
    op.part = W.part;
    if ((rc = grouped_gemm(op, st))) return rc;
  }
  {
    GroupedOp op = op_base(D, r);
    op.form = GROUPED_NN;
    op.N = D.h;
    op.K = D.f;
    op.a = W.dg;
    op.a2 = W.du;
    op.a_rows = D.pairs;
    op.w = w1;
    op.w2 = w3;
    op.out = W.dxs;
    op.span = W.span;
    if ((rc = grouped_gemm(op, st))) return rc;
  }
  {
    GroupedOp op = op_base(D, r);
    op.form = GROUPED_TN;
    op.M = D.f;
    op.N = D.h;
    op.a = W.dg;
    op.a2 = W.du;
    op.a_rows = D.pairs;
    op.b = x;
    op.b_rows = D.n;
    op.b_gather = true;
    op.order = r->order;
    op.out = dw1;
    op.out2 = dw3;
    op.out_f32 = D.grads_f32;
    op.beta = D.accum ? 1.f : 0.f;
    if ((rc = grouped_gemm(op, st))) return rc;
  }
  {
    GroupedOp op = op_base(D, r);
    op.form = GROUPED_TN;
    op.M = D.h;
    op.N = D.f;
    op.a = dy;
    op.a_rows = D.n;
    op.a_gather = true;
    op.b = W.aw;
    op.b_rows = D.pairs;
    op.order = r->order;
    op.out = dw2;
    op.out_f32 = D.grads_f32;
    op.beta = D.accum ? 1.f : 0.f;
    if ((rc = grouped_gemm(op, st))) return rc;
  }
  if ((rc = combine(D, W.dxs, r, W.span, nullptr, dx, W.part, (int)(2 * grouped_part_tiles(D.f)), dweights, st))) return rc;
  return D.debug ? debug_finish(st) : BPT_OK;
}

int bpt_grouped_gemm(const bpt_grouped_config* c, const void* a, const void* b, const int32_t* offsets, void* out, void* stream) {
  if (!c) return BPT_EINVAL;
  if (c->rows < 1 || c->n < 8 || (c->n % 8) || c->k < 8 || (c->k % 8) || c->groups < 1 || c->groups > GROUPED_MAX_GROUPS) return BPT_EINVAL;
  if (c->form < BPT_GROUPED_NT || c->form > BPT_GROUPED_TN) return BPT_EINVAL;
  if (c->out_dtype != BPT_DTYPE_F32 && c->out_dtype != BPT_DTYPE_BF16) return BPT_EINVAL;
  if (c->flags & ~(BPT_FLAG_ACCUM_GRADS | BPT_FLAG_DETERMINISTIC | BPT_FLAG_DEBUG_CHECKS)) return BPT_EINVAL;
  const bool f32 = c->out_dtype == BPT_DTYPE_F32, tn = c->form == BPT_GROUPED_TN;
  if ((c->flags & BPT_FLAG_ACCUM_GRADS) && !f32) return BPT_EINVAL;
  if (c->rows > (1 << 29)) return BPT_EUNSUPPORTED;
  if (!a || !b || !offsets || !out || !al(a, 16) || !al(b, 16) || !al(offsets, 4) || !al(out, 16)) return BPT_EINVAL;
  const int64_t rows = c->rows, n = c->n, k = c->k, g = c->groups;
  const Span sp[] = {{a, rows * k * 2}, {b, (tn ? rows * n : g * n * k) * 2}, {offsets, (g + 1) * 4},
                     {out, (tn ? g * n * k : rows * n) * (f32 ? 4 : 2)}};
  if (overlaps(sp[3], sp, 3)) return BPT_EINVAL;
  const bool debug = (c->flags & BPT_FLAG_DEBUG_CHECKS) != 0;
  if (debug && debug_spans(sp, 4)) return BPT_EINVAL;
  GroupedOp op;
  op.form = c->form;
  op.rows = rows;
  op.N = n;
  op.groups = c->groups;
  op.offsets = offsets;
  op.mean_rows = rows / g;
  op.a = a;
  op.a_rows = rows;
  if (tn) {
    op.M = k;
    op.b = b;
    op.b_rows = rows;
  } else {
    op.K = k;
    op.w = b;
  }
  op.out = out;
  op.out_f32 = f32;
  op.beta = (c->flags & BPT_FLAG_ACCUM_GRADS) ? 1.f : 0.f;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int rc = grouped_gemm(op, st);
  if (rc) return rc;
  return debug ? debug_finish(st) : BPT_OK;
}

}  // extern "C"
