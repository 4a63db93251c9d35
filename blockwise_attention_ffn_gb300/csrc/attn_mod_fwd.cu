// attn_mod_fwd.cu -- attention forward with a key window per query row, capped
// scores and a distance bias, on tcgen05 (bpt_attention_mod_fwd).
//
// The recurrence is that of the plain forward: for the key tiles j of a query
// tile, S = Q K_j^T, y = modified scores, m' = max(m, rowmax y),
// l = l 2^(m - m') + rowsum 2^(y - m'), O = O 2^(m - m') + 2^(y - m') V_j; at
// the end O / l and the log-sum-exp.  What differs:
//  * A tile's first and last key tile come from its rows' windows, so packed
//    documents, prefixes and padding cost only the tiles that some row sees.
//  * Scores are modified between the tensor core and the softmax. With a cap
//    of at most 44 (2^64 in the exponent's units) and no bias the scores are
//    bounded, so the running maximum is dropped: every row keeps m = 0.
//  * Row sums are fp32 sums of the fp32 exponentials, so the log-sum-exp is an
//    fp32-exact output; the tensor core's row sums of bf16 P would be off by
//    up to 2^-9.
//
// One CTA = one 128-row query tile of one head, heaviest tiles first; the 128
// keys of a tile are split in two halves, each with its own softmax warps
// (2..5, 6..9), MMA-issuing warp (1, 10), running maximum and O accumulator,
// merged at the end by the log-sum-exp rule.  All head dims take this form
// here, unlike the plain forward: the modified softmax, not the tensor core,
// bounds the loop, and two warps per SM sub-partition hide each other's
// latency.  Q sits in TMEM where it fits beside both O's (d <= 96), else in
// shared memory.
#include <math.h>
#include <string.h>

#include "../../include/bpt.h"
#include "attn_mod.cuh"
#include "internal.h"

namespace bpt {
int make_attn_map(CUtensorMap* map, const void* qkv, int b, int s, int64_t ld, int d);

namespace {

struct ModFwdParams {
  CUtensorMap map_qkv;  // 3-D {width, s, b}, box {CW, 128, 1}
  int s, s_pad, H, G, causal;
  int k_col, v_col, n_qt;
  __nv_bfloat16* o;
  float* lse;
  const __nv_bfloat16* qkv;
  long long width;
  const int32_t *row_begin, *row_end;
  const float* slopes;
  float scale, scale_log2;  // 1/sqrt(d), log2(e)/sqrt(d)
  float inv_cap, cap_log2;  // scale / cap, cap log2(e)
  int fixed_max;
  unsigned int* err;
};

// TMEM: S of half b as two 64-column buffers at 128 b, O_b at 256 + b D, Q at
// 256 + 2 D (d <= 96).  Shared memory: Q (d > 96), the K/V ring, the merge's
// maxima, barriers.
template <int D>
struct ModFwdCfg {
  using T = TileGeom<D>;
  static constexpr bool Q_TMEM = D <= 96;
  static constexpr int STAGE = 2 * T::TILE;
  static constexpr int QB = Q_TMEM ? 0 : T::TILE;
  static constexpr int RED = 2 * 128 * 4;
  static constexpr int FIT = (232448 - QB - RED - 1280) / STAGE;
  static constexpr int KVS = FIT > 5 ? 5 : FIT;
  static constexpr int SMEM = QB + KVS * STAGE + RED + 1024 + 256;
  static constexpr uint32_t COL_O = 256, COL_Q = 256 + 2 * D;
};

template <int D, bool CAP>
__global__ void __launch_bounds__(352, 1) attn_mod_fwd_kernel(const __grid_constant__ ModFwdParams p) {
  using T = TileGeom<D>;
  using C = ModFwdCfg<D>;
  constexpr int KVS = C::KVS, STAGE = C::STAGE;
  static_assert(C::COL_O + 2 * D + (C::Q_TMEM ? D / 2 : 0) <= 512, "TMEM columns");
  constexpr uint32_t IDESC_S = idesc_bf16(128, 64, false, false);
  constexpr uint32_t IDESC_PV = idesc_bf16(128, D, false, true);
  constexpr float NEG_INF = -INFINITY;
  constexpr float LN2 = 0.6931471805599453f;

  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + C::QB;
  float* red = reinterpret_cast<float*>(sKV + KVS * STAGE);
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(red) + C::RED);
  uint64_t* q_ready = bars;             // Q in TMEM (4 warps) or in shared memory (TMA)
  uint64_t* kv_full = bars + 1;         // [KVS]
  uint64_t* kv_empty = kv_full + KVS;   // [KVS], both issuers
  uint64_t* s_full = kv_empty + KVS;    // [half][buffer]
  uint64_t* p_full = s_full + 4;        // [half][buffer], 4 warps
  uint64_t* pv_done = p_full + 4;       // [half]
  uint64_t* drain = pv_done + 2;        // [half]
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* range = reinterpret_cast<int*>(tmem_holder + 2);  // [4] least lo, [4] largest hi of a warp's rows

  const int warp = warp_id();
  const int lane = lane_id();
  const int pair = blockIdx.x / p.n_qt;
  const int qt = p.n_qt - 1 - (int)(blockIdx.x % p.n_qt);
  const int n = pair % p.H;
  const int bi = pair / p.H;
  const int q0 = qt * 128;
  const int g = n / p.G;

  // this softmax thread's row and its window
  const int quarter = warp & 3;
  const int r = quarter * 32 + lane;
  const int qpos = q0 + r;
  int2 win = make_int2(0, 0);
  if (warp >= 2 && warp < 10) {
    win = key_window(p.row_begin, p.row_end, p.causal, p.s, bi, qpos);
    if (warp < 6) {
      const int lo = __reduce_min_sync(0xffffffffu, win.x < win.y ? win.x : INT32_MAX);
      const int hi = __reduce_max_sync(0xffffffffu, win.y);
      if (lane == 0) {
        range[quarter] = lo;
        range[4 + quarter] = hi;
      }
    }
  }
  if (threadIdx.x == 0) {
    mbar_init(q_ready, C::Q_TMEM ? 4 : 1);
    for (int i = 0; i < KVS; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 2);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&pv_done[b], 1);
      mbar_init(&drain[b], 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) tma_prefetch(&p.map_qkv);
  if (warp == 1) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const uint32_t tQA = tmem + C::COL_Q;
  // key tiles [j0, j0 + nkv) hold every key that some row sees
  const int lo_all = min(min(range[0], range[1]), min(range[2], range[3]));
  const int hi_all = max(max(range[4], range[5]), max(range[6], range[7]));
  const int j0 = lo_all < hi_all ? lo_all / 128 : 0;
  const int nkv = lo_all < hi_all ? (hi_all + 127) / 128 - j0 : 0;

  if (warp == 0) {
    if (lane == 0 && nkv > 0) {
      // ------------------------------------------------ TMA producer
      if constexpr (!C::Q_TMEM) {
        mbar_expect_tx(q_ready, T::TILE);
#pragma unroll
        for (int c = 0; c < T::NCH; ++c) tma_load_3d(sQ + c * T::CHUNK, &p.map_qkv, q_ready, n * D + c * T::CW, q0, bi);
      }
      int issued = 0;
      for (int j = 0; j < nkv; ++j) {
        const int st = j % KVS;
        if (j >= KVS && !bounded_wait(&kv_empty[st], ((j / KVS) & 1) ^ 1, abort_flag, 251, p.err)) break;
        uint8_t* sK = sKV + st * STAGE;
        uint8_t* sV = sK + T::TILE;
        mbar_expect_tx(&kv_full[st], 2 * T::TILE);
#pragma unroll
        for (int c = 0; c < T::NCH; ++c)
          tma_load_3d(sK + c * T::CHUNK, &p.map_qkv, &kv_full[st], p.k_col + g * D + c * T::CW, (j0 + j) * 128, bi);
#pragma unroll
        for (int c = 0; c < T::NCH; ++c)
          tma_load_3d(sV + c * T::CHUNK, &p.map_qkv, &kv_full[st], p.v_col + g * D + c * T::CW, (j0 + j) * 128, bi);
        issued = j + 1;
      }
      if (*abort_flag) {
        if constexpr (!C::Q_TMEM) drain_wait(q_ready, 0);
        for (int j = (issued > KVS ? issued - KVS : 0); j < issued; ++j) drain_wait(&kv_full[j % KVS], (j / KVS) & 1);
      }
    }
  } else if (warp == 1 || warp == 10) {
    // ------------------------------------------------ MMA issuers (the
    // whole warp runs the loop, one elected lane issues): S_b(j+1) = Q
    // K_{j+1}[64b..]^T into buffer (j+1) % 2, then O_b += P_b(j) V_j[64b..];
    // S_b(j+1) overwrites P_b(j-1) after PV_b(j-1) from the same thread
    if (nkv > 0) {
      const int b = warp == 1 ? 0 : 1;
      const uint32_t uKV = smem_u32(sKV), uQ = smem_u32(sQ);
      const uint32_t tSb = tmem + 128 * b;
      const uint32_t tOb = tmem + C::COL_O + b * D;
      auto issue_s = [&](int j) -> bool {
        if (!bounded_wait_w(&kv_full[j % KVS], (j / KVS) & 1, abort_flag, 253, p.err)) return false;
        tc_fence_after();
        const uint32_t kt = uKV + (j % KVS) * STAGE + 64 * T::SWB * b;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          if constexpr (C::Q_TMEM)
            umma_bf16_tmem_a_w(tSb + (j & 1) * 64, tQA + kk * 8, T::kmajor(kt, kk), IDESC_S, kk > 0);
          else
            umma_bf16_w(tSb + (j & 1) * 64, T::kmajor(uQ, kk), T::kmajor(kt, kk), IDESC_S, kk > 0);
        }
        umma_commit_w(&s_full[2 * b + (j & 1)]);
        return true;
      };
      bool ok = bounded_wait_w(q_ready, 0, abort_flag, 254, p.err) && issue_s(0);
      for (int j = 0; ok && j < nkv; ++j) {
        if (j + 1 < nkv && !issue_s(j + 1)) { ok = false; break; }
        if (!bounded_wait_w(&p_full[2 * b + (j & 1)], (j >> 1) & 1, abort_flag, 255, p.err)) { ok = false; break; }
        tc_fence_after();
        const uint32_t vt = uKV + (j % KVS) * STAGE + T::TILE;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_bf16_tmem_a_w(tOb, tSb + (j & 1) * 64 + kk * 8, T::mnmajor(vt, 4 * b + kk), IDESC_PV, (j > 0 || kk > 0));
        umma_commit_w(&kv_empty[j % KVS]);
        umma_commit_w(&pv_done[b]);
      }
      if (!ok) {
        umma_commit_w(&drain[b]);
        drain_wait(&drain[b], 0);
      }
    }
  } else {
    // ------------------------------------------------ softmax (warps 2..9)
    const int b = (warp - 2) >> 2;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t tSb = tmem + 128 * b;
    const uint32_t tOb = tmem + C::COL_O + b * D;
    const bool valid = qpos < p.s;
    __nv_bfloat16* orow = p.o + ((long long)bi * p.s + qpos) * p.H * D + (long long)n * D;
    float* lse = p.lse ? p.lse + ((long long)bi * p.H + n) * p.s_pad + qpos : nullptr;
    if constexpr (C::Q_TMEM) if (b == 0 && nkv > 0) {
      // this thread's Q row into TMEM as bf16 pairs (zero past the sequence)
      uint32_t w[D / 2];
      const __nv_bfloat16* src = p.qkv + ((long long)bi * p.s + qpos) * p.width + (long long)n * D;
#pragma unroll
      for (int cc = 0; cc < D / 8; ++cc) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (valid) v = *reinterpret_cast<const uint4*>(src + cc * 8);
        w[4 * cc] = v.x;
        w[4 * cc + 1] = v.y;
        w[4 * cc + 2] = v.z;
        w[4 * cc + 3] = v.w;
      }
      tmem_store_row<D / 2>(tQA + lane_off, w);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_ready);
    }
    const float slope2 = p.slopes ? p.slopes[n] * 1.4426950408889634f : 0.f;
    const bool bias = p.slopes != nullptr;
    // the units of m and of the scores when exponentiated: raw scores times
    // log2(e)/sqrt(d) without a modifier, else already log2
    const float ce = (CAP || bias) ? 1.f : p.scale_log2;
    const bool fixed = CAP && p.fixed_max;
    float m_run = fixed ? 0.f : NEG_INF, l_run = 0.f;
    bool ok = true;
    for (int j = 0; j < nkv; ++j) {
      const int sb = j & 1;
      const uint32_t tb = tSb + sb * 64 + lane_off;
      ok = bounded_wait(&s_full[2 * b + sb], (j >> 1) & 1, abort_flag, 261, p.err);
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      tc_fence_after();
      // this half's key columns [klo, khi) of the 64 are visible
      const int kv0 = (j0 + j) * 128 + 64 * b;
      const int klo = max(win.x - kv0, 0), khi = min(win.y - kv0, 64);
      const bool full = klo == 0 && khi == 64;
      uint32_t pk[32];
      bool rescale = false;
      float alpha = 1.f;
      if (!__any_sync(0xffffffffu, klo < khi)) {
        // nothing of this half is visible to the warp's rows
#pragma unroll
        for (int i = 0; i < 32; ++i) pk[i] = 0u;
      } else {
        uint32_t sv[64];
        tmem_ld32_nw(tb, sv);
        tmem_ld32_nw(tb + 32, sv + 32);
        tmem_wait_ld(sv);
        if constexpr (CAP) {
          const bool small = amax_of(sv) * p.inv_cap <= TANH_SMALL;
          if (__all_sync(0xffffffffu, small)) {
            const uint64_t ic2 = f2(p.inv_cap, p.inv_cap), cl2 = f2(p.cap_log2, p.cap_log2);
#pragma unroll
            for (int i = 0; i < 64; i += 2) {
              const float2 t = f2split(
                  mul2(tanh2_small(mul2(f2(__uint_as_float(sv[i]), __uint_as_float(sv[i + 1])), ic2)), cl2));
              sv[i] = __float_as_uint(t.x);
              sv[i + 1] = __float_as_uint(t.y);
            }
          } else {
            const float y2 = p.inv_cap * 2.8853900817779268f;
#pragma unroll
            for (int i = 0; i < 64; ++i) sv[i] = __float_as_uint(tanh_any(__uint_as_float(sv[i]) * y2) * p.cap_log2);
          }
        }
        if (bias) {
          const float cs = CAP ? 1.f : p.scale_log2;
          const BiasLine bl = bias_line(slope2, qpos, kv0, p.causal != 0, false);
          if (!__any_sync(0xffffffffu, bl.mixed)) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
              sv[i] = __float_as_uint(fmaf(__uint_as_float(sv[i]), cs, fmaf(bl.step, (float)i, bl.base)));
          } else {
            const float dist = (float)(qpos - kv0);
#pragma unroll
            for (int i = 0; i < 64; ++i)
              sv[i] = __float_as_uint(fmaf(__uint_as_float(sv[i]), cs, -slope2 * fabsf(dist - (float)i)));
          }
        }
        if (!fixed) {
          float mx = NEG_INF;
          if (full) {
            float m4[4] = {NEG_INF, NEG_INF, NEG_INF, NEG_INF};
#pragma unroll
            for (int i = 0; i < 64; i += 2)
              m4[(i >> 1) & 3] = max3f(m4[(i >> 1) & 3], __uint_as_float(sv[i]), __uint_as_float(sv[i + 1]));
            mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          } else {
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (i >= klo && i < khi) mx = fmaxf(mx, __uint_as_float(sv[i]));
          }
          const float m_new = fmaxf(m_run, mx);
          // the maximum is left stale while it moves by less than 2^8 (O and
          // l are scaled alike, so the result does not change)
          rescale = __any_sync(0xffffffffu, (m_new - m_run) * ce > 8.f);
          if (rescale) {
            alpha = (m_run == NEG_INF) ? 0.f : ex2((m_run - m_new) * ce);
            m_run = m_new;
          }
        }
        // a row that has seen no key keeps m = -inf: offset 0, P masked to 0
        const float mc = (m_run == NEG_INF) ? 0.f : m_run * ce;
        const uint64_t c2 = f2(ce, ce), nmc2 = f2(-mc, -mc);
        uint64_t rs[2] = {0ull, 0ull};
        if (full) {
#pragma unroll
          for (int i = 0; i < 64; i += 2) {
            const float2 e = f2split(fma2(f2(__uint_as_float(sv[i]), __uint_as_float(sv[i + 1])), c2, nmc2));
            const float e0 = ex2(e.x), e1 = ex2(e.y);
            rs[(i >> 1) & 1] = add2(rs[(i >> 1) & 1], f2(e0, e1));
            pk[i / 2] = pack_bf16(e0, e1);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 64; i += 2) {
            const float2 e = f2split(fma2(f2(__uint_as_float(sv[i]), __uint_as_float(sv[i + 1])), c2, nmc2));
            const float e0 = (i >= klo && i < khi) ? ex2(e.x) : 0.f;
            const float e1 = (i + 1 >= klo && i + 1 < khi) ? ex2(e.y) : 0.f;
            rs[(i >> 1) & 1] = add2(rs[(i >> 1) & 1], f2(e0, e1));
            pk[i / 2] = pack_bf16(e0, e1);
          }
        }
        const float2 rsum = f2split(add2(rs[0], rs[1]));
        l_run = fmaf(l_run, alpha, rsum.x + rsum.y);
      }
      // P over the first 32 columns of its own S buffer (all read above)
      tmem_st32(tb, pk);
      // PV(j-1) must be done before O is rescaled.  Having seen S(j), which
      // was issued after PV(j-2), these warps know pv_done is in phase j-1 or
      // j, so a wait on the parity of j - 1 is exact however many phases went
      // by unwaited; the last step always waits, so the wait after the loop
      // is exact too.
      if (j > 0 && (rescale || j == nkv - 1)) {
        ok = bounded_wait(&pv_done[b], (j - 1) & 1, abort_flag, 262, p.err);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        tc_fence_after();
        if (rescale) {
          uint32_t ro[D];
#pragma unroll
          for (int cc = 0; cc < D / 16; ++cc) tmem_ld16_nw(tOb + lane_off + cc * 16, ro + cc * 16);
          tmem_wait_ld(ro);
#pragma unroll
          for (int i = 0; i < D; ++i) ro[i] = __float_as_uint(__uint_as_float(ro[i]) * alpha);
#pragma unroll
          for (int cc = 0; cc < D / 16; ++cc) tmem_st16_nw(tOb + lane_off + cc * 16, ro + cc * 16);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[2 * b + sb]);
    }
    if (nkv == 0) {
      // no row of the tile sees a key
      if (b == 0) {
        if (valid) {
#pragma unroll
          for (int cc = 0; cc < D / 8; ++cc) reinterpret_cast<uint4*>(orow)[cc] = make_uint4(0u, 0u, 0u, 0u);
        }
        if (lse) *lse = valid ? NEG_INF : 0.f;
      }
    } else {
      if (ok) ok = __all_sync(0xffffffffu, bounded_wait(&pv_done[b], (nkv - 1) & 1, abort_flag, 263, p.err));
      // merge: both halves' warps of this lane quarter always reach this
      // barrier, which also ANDs their status; each leaves its maximum and
      // row sum for the other
      red[b * 128 + r] = m_run;
      bool merge = named_bar_and(1 + quarter, 64, ok);
      if (merge)
        merge = __all_sync(0xffffffffu, bounded_wait(&pv_done[b ^ 1], (nkv - 1) & 1, abort_flag, 264, p.err));
      const float m_o = red[(b ^ 1) * 128 + r];
      named_bar(1 + quarter, 64);
      red[b * 128 + r] = l_run;
      named_bar(1 + quarter, 64);
      if (merge) {
        tc_fence_after();
        const float l_o = red[(b ^ 1) * 128 + r];
        const float m = fmaxf(m_run, m_o);
        const float a_self = (m_run == NEG_INF) ? 0.f : ex2((m_run - m) * ce);
        const float a_o = (m_o == NEG_INF) ? 0.f : ex2((m_o - m) * ce);
        const float l = l_run * a_self + l_o * a_o;
        const float inv_l = l == 0.f ? 0.f : 1.f / l;  // nothing visible: O = 0
        const float w_self = a_self * inv_l, w_o = a_o * inv_l;
        const uint32_t tOo = tmem + C::COL_O + (b ^ 1) * D;
        // each half writes half of the row's 16-column chunks
        constexpr int NC = D / 16;
        constexpr int NC0 = (NC + 1) / 2;
        const int cbeg = b == 0 ? 0 : NC0, cend = b == 0 ? NC0 : NC;
        for (int cc = cbeg; cc < cend; ++cc) {
          uint32_t vs[16], vo[16];
          tmem_ld16_nw(tOb + lane_off + cc * 16, vs);
          tmem_ld16_nw(tOo + lane_off + cc * 16, vo);
          tmem_wait_ld(vs);
          tmem_wait_ld(vo);
          uint32_t vm[16];
#pragma unroll
          for (int k = 0; k < 16; ++k)
            vm[k] = __float_as_uint(__uint_as_float(vs[k]) * w_self + __uint_as_float(vo[k]) * w_o);
          if (valid) store_row16(orow + cc * 16, vm, 1.f);
        }
        if (b == 0 && lse) *lse = !valid ? 0.f : l == 0.f ? NEG_INF : fmaf(m * ce, LN2, logf(l));
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool CAP>
int launch_mod_fwd(const ModFwdParams& prm, int grid, cudaStream_t st) {
  constexpr int SMEM = ModFwdCfg<D>::SMEM;
  static_assert(SMEM <= 232448, "attention forward tile set exceeds shared memory");
  static std::atomic<uint64_t> attr{0};  // devices whose limit is set
  if (smem_limit_once(reinterpret_cast<const void*>(attn_mod_fwd_kernel<D, CAP>), SMEM, &attr)) return BPT_ECUDA;
  attn_mod_fwd_kernel<D, CAP><<<grid, 352, SMEM, st>>>(prm);
  return cudaGetLastError() == cudaSuccess ? BPT_OK : BPT_ECUDA;
}

}  // namespace

int attention_mod_fwd(const PackedDims& D, int causal, const bpt_score_mod& mod, const void* qkv, void* o, float* lse,
                      cudaStream_t st) {
  ModFwdParams p;
  memset(&p, 0, sizeof(p));
  if (make_attn_map(&p.map_qkv, qkv, (int)D.b, (int)D.s, D.width, (int)D.d)) return BPT_EINVAL;
  p.s = (int)D.s;
  p.s_pad = (int)D.s_pad;
  p.H = (int)D.H;
  p.G = (int)D.G;
  p.causal = causal;
  p.k_col = (int)(D.H * D.d);
  p.v_col = (int)((D.H + D.Hkv) * D.d);
  p.n_qt = (int)(D.s_pad / 128);
  p.o = reinterpret_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.qkv = reinterpret_cast<const __nv_bfloat16*>(qkv);
  p.width = D.width;
  p.row_begin = mod.row_begin;
  p.row_end = mod.row_end;
  p.slopes = mod.slopes;
  p.scale = 1.f / sqrtf((float)D.d);
  p.scale_log2 = p.scale * 1.4426950408889634f;
  const bool cap = mod.softcap > 0.f;
  if (cap) {
    p.inv_cap = p.scale / mod.softcap;
    p.cap_log2 = mod.softcap * 1.4426950408889634f;
    p.fixed_max = !mod.slopes && p.cap_log2 <= 64.f;
  }
  p.err = device_error_word();
  if (!p.err) return BPT_ECUDA;
  const int grid = (int)(p.n_qt * D.H * D.b);
  // credited as without windows, which live on the device
  const double pairs = causal ? (double)D.s * (D.s + 1) / 2 : (double)D.s * D.s;
  ProfScope prof(PROF_ATTN_FWD, 4.0 * D.d * pairs * D.H * D.b, 0.0, st);
  switch (D.d) {
    case 64: return cap ? launch_mod_fwd<64, true>(p, grid, st) : launch_mod_fwd<64, false>(p, grid, st);
    case 80: return cap ? launch_mod_fwd<80, true>(p, grid, st) : launch_mod_fwd<80, false>(p, grid, st);
    case 96: return cap ? launch_mod_fwd<96, true>(p, grid, st) : launch_mod_fwd<96, false>(p, grid, st);
    case 112: return cap ? launch_mod_fwd<112, true>(p, grid, st) : launch_mod_fwd<112, false>(p, grid, st);
    case 128: return cap ? launch_mod_fwd<128, true>(p, grid, st) : launch_mod_fwd<128, false>(p, grid, st);
    default: return BPT_EUNSUPPORTED;
  }
}

}  // namespace bpt
