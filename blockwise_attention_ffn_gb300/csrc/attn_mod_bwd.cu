// attn_mod_bwd.cu -- attention backward with a key window per query row, capped
// scores and a distance bias (bpt_attention_mod_bwd).
//
// With x = q.k / sqrt(d), u = tanh(x / C), y = C u - a |i - j| (or y = x - ...
// without a cap), P = exp(y - LSE) on the visible pairs and 0 elsewhere,
//   dV = P^T dO,  dP = dO V^T,  D = rowsum(dO * O),
//   dx = P * (dP - D) * (1 - u^2),  dQ = dx K / sqrt(d),  dK = dx^T Q / sqrt(d).
// The bias has no gradient here (the slopes are constants).
//
// Two kernels after one that prepares the rows, in the form of the plain
// backward: dK/dV with the key tile outermost, dQ with the query tile
// outermost, both rebuilding their scores in 64-wide sub-tiles that two groups
// of compute warps take in turn; no atomics.  What differs:
//  * The query tiles that see a key tile, and the key tiles that a query tile
//    sees, come from the windows; tiles outside are never loaded.
//  * Without a cap, -LSE enters dK/dV's scores through the product, as before,
//    but in three bf16 terms (24 bits: a biased LSE can be large); with one it
//    has to be added after the tanh, and travels with the query stage as 128
//    floats.  D's three terms enter through the product in both.
//  * dK/dV's masks are per column: a stage carries its queries' windows, read
//    only in sub-tiles that some window cuts.
//  * P stays fp32 for dx; P (1 - u^2) replaces it in place, so the cap costs
//    no registers.
// P and dx are rounded to bf16 where they are operands of a tensor-core product
// (dV, dQ, dK), as in the plain backward: each by at most 2^-8 of its value, with
// signs that do not build up; dqkv is off by 2.5e-3 to 3.3e-3 (relative norm, its
// own bf16 rounding of 1.7e-3 included).
//
// Measured at 8192 rows of 32 + 8 + 8 heads of 128, causal: dK/dV 791 us, dQ 457,
// capped 904 and 563, capped and biased 948 and 568, in fixed order 1,031 and 626;
// documents of 1500: 204 and 141, capped 237 and 168.  dK/dV is bound by its four
// products (tensor core 57 to 70% busy: at head dims above 80 S^T and dP^T take
// both operands from shared memory, and 64 columns of them cost 48 cycles a step of
// 16 where 32 are arithmetic) and by the chain between them; one product of 128
// columns for both groups saves a fifth of the tensor core's time but makes the
// groups run in step: 774 us plain (against 807 then), 1,064 capped (against 901).
// The capped dK/dV kernels hold more than their 168 registers and spill 20 to 84
// bytes a thread.
#include <math.h>
#include <string.h>

#include <algorithm>

#include "../../include/bpt.h"
#include "attn_mod.cuh"
#include "internal.h"

namespace bpt {
int make_attn_map(CUtensorMap* map, const void* qkv, int b, int s, int64_t ld, int d, int box_rows);

namespace {

// The windows of one 128-query tile as the dK/dV kernel's stage takes them:
// per row (lo, hi - lo), then per 64-row half the bounds that tell a sub-tile
// that no window cuts.
struct __align__(16) WinRecord {
  int2 row[128];
  int2 cut[2];  // (largest lo, least hi)
  int4 unused;
};
static_assert(sizeof(WinRecord) % 16 == 0, "bulk copies move 16-byte units");

struct ModBwdParams {
  CUtensorMap map_qkv;  // 3-D {width, s, b}, box {CW, 128, 1}
  CUtensorMap map_do;   // 3-D {H d, s, b}, box {CW, 128, 1}
  CUtensorMap map_out;  // 3-D {width, s, b}, box {CW, 32, 1}: dqkv
  CUtensorMap map_aux;  // 2-D {8, b*H*s_pad} bf16, box {8, 128}, no swizzle
  int s, s_pad, H, Hkv, G, causal, n_t;
  ItemOrder order_kv, order_q;
  int k_col, v_col;
  const float *dsum, *nl2;  // [b, H, s_pad]: dO . O and -LSE log2(e) (0 for a row that sees nothing)
  const WinRecord* rec;     // [b, n_t]
  const int2* span;         // [b, n_t]: least lo and largest hi of a query tile's rows
  const __nv_bfloat16 *qkv, *dout;
  __nv_bfloat16* dqkv;
  long long width;
  const int32_t *row_begin, *row_end;
  const float* slopes;
  float scale, scale_log2, cap_log2;
  CapCoef cap;  // tanh of the raw scores
  int one_issuer;  // fixed-order mode: warp 1 issues both groups' products
  unsigned int* err;
};

// exp2 of 64 modified scores in log2 units and what dx multiplies (dP - D)
// with: sv in, am their largest magnitude, pe = P (1 - u^2) out, pk = P as
// bf16 pairs (WANT_P).  add(k): what is added to the scaled scores of the pair
// (k, k + 1), the bias and -LSE; on(k): visible; all: every element is; seen(sv):
// the largest magnitude of the visible ones.
// A masked u is replaced by one whose exponential is 0 and whose square is
// finite, in a pass of its own, so that unmasked sub-tiles pay nothing for it.
template <bool CAP, bool WANT_P, class Add, class On, class Seen>
__device__ __forceinline__ void probabilities(const ModBwdParams& p, uint32_t (&sv)[64], float am, float (&pe)[64],
                                              uint32_t (&pk)[32], bool all, Add add, On on, Seen seen) {
  if constexpr (CAP) {
    // u over sv
    auto put = [&](int k, uint64_t v) {
      const float2 x = f2split(v);
      sv[k] = __float_as_uint(x.x);
      sv[k + 1] = __float_as_uint(x.y);
    };
    if (__all_sync(0xffffffffu, am <= p.cap.near1)) {
#pragma unroll
      for (int k = 0; k < 64; k += 2) put(k, cap_near1(p.cap, f2(__uint_as_float(sv[k]), __uint_as_float(sv[k + 1]))));
    } else {
      // masked scores have no say in the form that the others take, as in the
      // forward (tiles beyond C/4: 4% of the whole backward at documents of 4000,
      // cap 30, 794 us without, 826 so; a form of its own for masked tiles 840)
      if (!all) am = seen(sv);
      if (__all_sync(0xffffffffu, am <= p.cap.near1)) {
#pragma unroll
        for (int k = 0; k < 64; k += 2) put(k, cap_near1(p.cap, f2(__uint_as_float(sv[k]), __uint_as_float(sv[k + 1]))));
      } else if (__all_sync(0xffffffffu, am <= p.cap.near2)) {
#pragma unroll
        for (int k = 0; k < 64; k += 2) put(k, cap_near2(p.cap, f2(__uint_as_float(sv[k]), __uint_as_float(sv[k + 1]))));
      } else if (!p.cap.large) {
#pragma unroll
        for (int k = 0; k < 64; k += 2) put(k, cap_far(p.cap, f2(__uint_as_float(sv[k]), __uint_as_float(sv[k + 1]))));
      } else {
#pragma unroll
        for (int k = 0; k < 64; k += 2)
          put(k, cap_far_large(p.cap, f2(__uint_as_float(sv[k]), __uint_as_float(sv[k + 1]))));
      }
    }
  }
  if (!all) {
#pragma unroll
    for (int k = 0; k < 64; ++k)
      if (!on(k)) sv[k] = __float_as_uint(-1e18f);
  }
  const float cs = CAP ? p.cap_log2 : p.scale_log2;
  const uint64_t cs2 = both(cs), one2 = both(1.f);
#pragma unroll
  for (int k = 0; k < 64; k += 2) {
    const uint64_t u2 = f2(__uint_as_float(sv[k]), __uint_as_float(sv[k + 1]));
    const float2 e = f2split(fma2(u2, cs2, add(k)));
    const float p0 = ex2(e.x), p1 = ex2(e.y);
    if constexpr (WANT_P) pk[k / 2] = pack_bf16(p0, p1);
    if constexpr (CAP) {
      const float2 f = f2split(mul2(f2(p0, p1), fma2(u2 ^ 0x8000000080000000ull, u2, one2)));
      pe[k] = f.x;
      pe[k + 1] = f.y;
    } else {
      pe[k] = p0;
      pe[k + 1] = p1;
    }
  }
}

// A masked dP may be infinite (a value that no window reaches is anything
// finite, and its product with dO is not); 0 times it would be NaN.
__device__ __forceinline__ void mask_gradient(uint32_t (&dr)[64], const float (&pe)[64]) {
#pragma unroll
  for (int k = 0; k < 64; ++k)
    if (pe[k] == 0.f) dr[k] = 0u;
}

// ===========================================================================
// dK / dV
// ===========================================================================
// Shared memory of dK/dV: K and V, (d > 80) their extra chunks; dK and dV on
// their way out, for d > 80 in K's and V's place; the stages of Q, dO, the 128
// queries' 16-byte extra rows, their windows and (with a cap) -LSE log2(e); then
// zeros, the upper half of the extra contraction step.
// TMEM: S^T [0, 128) and dP^T [128, 256) as two 64-column buffers each, dV at
// 256, dK at 256 + D, and for d <= 80 K and V with their extra chunks.
template <int D>
struct ModDkdvCfg {
  using T = TileGeom<D>;
  static constexpr bool KV_TMEM = D <= 80;
  static constexpr int AUX = 128 * 16;                 // 128 rows x 8 bf16
  static constexpr int KV = 2 * T::TILE + (KV_TMEM ? 2 * T::TILE : 2 * AUX);  // K, V, then results or extra chunks
  static constexpr int OUT = KV_TMEM ? 2 * T::TILE : 0;
  static constexpr int CTL = 512;
  static constexpr int REC = 2 * T::TILE + AUX;        // offset of the windows
  static constexpr int NL2 = REC + (int)sizeof(WinRecord);
  static constexpr int STAGE = REC + 2048;             // 1024-byte aligned tiles
  static_assert(sizeof(WinRecord) + 128 * 4 <= 2048, "the stage's tail");
  static constexpr int ZERO = 2048;                    // the upper 8 columns
  static constexpr int QS_FIT = (232448 - KV - ZERO - CTL) / STAGE;
  static constexpr int QS = QS_FIT > 4 ? 4 : QS_FIT;
  static constexpr int SMEM = KV + QS * STAGE + ZERO + CTL;
  static constexpr uint32_t COL_DV = 256, COL_DK = 256 + D, COL_K = 256 + 2 * D, COL_V = 256 + 2 * D + D / 2 + 8;
};

// One CTA per 128-row key tile of one key/value head, over the G query heads of
// its group and the query tiles that see it.  A step covers 64 queries:
// sub-tile u is the half u % 2 of stage u / 2 and uses buffer u % 2; compute
// warps 2..5 take the even sub-tiles, 6..9 the odd ones, with issuing warps 1
// and 10, in the order S(u), dP(u), dV(u) (after P^T(u)), S(u+2), dK(u) (after
// dS^T(u)), dP(u+2): what overwrites a buffer comes after its reader from the
// same thread.  P^T is written over S^T and dS^T over dP^T as bf16 pairs, the
// A operands of dV = P^T dO and dK = dS^T Q.  Both issuers add into dV and dK,
// which the compute warps zero first.
// Persistent like the forward: warp 11 takes the items and loads their K and V,
// warp 0 the stages.
//
// Few key tiles (short sequences, few key/value heads) leave SMs idle, or the
// last round of CTAs a poor fill.  Then a cluster of CTAs shares one item: each
// takes an equal part of its (query head, query tile) stream, leaves its dV and
// dK as fp32 in its own shared memory, and sums a share of the rows of all of
// them in rank order through distributed shared memory.
template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(384, 1) attn_mod_dkdv_kernel(const __grid_constant__ ModBwdParams p) {
  using T = TileGeom<D>;
  using C = ModDkdvCfg<D>;
  constexpr int QS = C::QS;
  constexpr int STAGE = C::STAGE;
  static_assert(C::COL_DK + D <= 512, "TMEM columns");
  static_assert(!C::KV_TMEM || C::COL_V + D / 2 + 8 <= 512, "TMEM columns");
  static_assert(QS >= 2, "Q/dO ring");
  constexpr uint32_t ID_S = idesc_bf16(128, 64, false, false);
  constexpr uint32_t ID_KV = idesc_bf16(128, D, false, true);

  static_assert((2 * QS + 19) * 8 + WORK_BYTES + 8 <= C::CTL, "control block");
  // the tiles' swizzle needs 1024-byte alignment, which the declaration gives
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sKV = smem;                  // K, V, their extra chunks (head dims above 80)
  uint8_t* sOut = smem + C::OUT;        // dV, dK
  uint8_t* sStage = smem + C::KV;
  uint8_t* sZero = sStage + QS * STAGE;
  uint8_t* control = sZero + C::ZERO;
  uint64_t* bars = reinterpret_cast<uint64_t*>(control + WORK_BYTES);
  // (read by 8 compute warps, 2 issuers, the loads)
  const WorkQueue queue{control, bars, bars + 2, bars + 4};
  uint64_t* kv_full = bars + 5;         // K, V landed, of every item
  uint64_t* kv_free = bars + 6;         // and their place free again (8 compute warps)
  uint64_t* kv_ready = bars + 7;        // K', V' in place, dV, dK zeroed (8 compute warps), of items with pairs
  uint64_t* all_done = bars + 8;        // both issuers' last products of an item with pairs done
  uint64_t* s_full = bars + 9;          // [2] S^T(u) in buffer u % 2
  uint64_t* dp_full = bars + 11;        // [2]
  uint64_t* p_full = bars + 13;         // [2] P^T(u) written (4 warps of the group)
  uint64_t* ds_full = bars + 15;        // [2] dS^T(u) written (4 warps)
  uint64_t* drain = bars + 17;          // [2], one per issuer
  uint64_t* qdo_full = bars + 19;       // [QS]
  uint64_t* qdo_empty = qdo_full + QS;  // [QS], both issuers
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(qdo_empty + QS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = warp_id();
  const int lane = lane_id();
  // the first (with a causal mask heaviest) key tiles first; a cluster's item
  // is its only one
  const int split = (int)cluster_size(), rank = (int)cluster_rank();
  const int nq_total = p.n_t;
  auto part = [&](int pairs, int r) { return (int)((long long)pairs * r / split); };

  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    mbar_init(kv_free, 8);
    mbar_init(kv_ready, 8);
    mbar_init(all_done, 2);
    mbar_init(queue.answered, 1);
    for (int i = 0; i < QS; ++i) {
      mbar_init(&qdo_full[i], 1);
      mbar_init(&qdo_empty[i], 2);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&queue.full[b], 1);
      mbar_init(&queue.empty[b], 11);
      mbar_init(&s_full[b], 1);
      mbar_init(&dp_full[b], 1);
      mbar_init(&p_full[b], 4);
      mbar_init(&ds_full[b], 4);
      mbar_init(&drain[b], 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch(&p.map_qkv);
    tma_prefetch(&p.map_do);
    tma_prefetch(&p.map_aux);
    tma_prefetch(&p.map_out);
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  if (threadIdx.x < C::ZERO / 16) {
    reinterpret_cast<uint4*>(sZero)[threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  auto load_kv = [&](int g, int bi, int j) {
    if (lane != 0) return;
    mbar_expect_tx(kv_full, 2 * T::TILE);
#pragma unroll
    for (int c = 0; c < T::NCH; ++c) {
      tma_load_3d(sKV + c * T::CHUNK, &p.map_qkv, kv_full, p.k_col + g * D + c * T::CW, j * 128, bi);
      tma_load_3d(sKV + T::TILE + c * T::CHUNK, &p.map_qkv, kv_full, p.v_col + g * D + c * T::CW, j * 128, bi);
    }
  };
  if (warp == 11) {
    // the first K and V, of which the preparation writes nothing
    const Item item = item_of(p.order_kv, blockIdx.x / split);
    load_kv(item.kv % p.Hkv, item.kv / p.Hkv, item.tile);
  }
  // what the preparation wrote; the dQ kernel, which needs nothing of this
  // one, fills the SMs that this one's last round leaves idle
  wait_for_previous();
  let_next_start();
  const uint32_t tS = tmem;          // + 64 b
  const uint32_t tdP = tmem + 128;   // + 64 b
  const uint32_t tdV = tmem + C::COL_DV;
  const uint32_t tdK = tmem + C::COL_DK;
  const uint32_t tKA = tmem + C::COL_K;
  const uint32_t tVA = tmem + C::COL_V;

  // a published item: key/value head n, sequence bi, key tile q0, and the query
  // tiles [j0, j0 + nkv) with a row that may see it
  if (warp == 11) {
    // ------------------------------------------------ items, K and V (the whole warp)
    int loads = 1;
    publish_items(queue, blockIdx.x / split, -1, split == 1, abort_flag, p.err, [&](int block) {
      const Item item = item_of(p.order_kv, block);
      const int bi = item.kv / p.Hkv, j = item.tile;
      // tiles between the first and the last that see nothing of it are masked
      // like any other
      int first = INT32_MAX, last = -1;
#pragma unroll 4
      for (int i = lane; i < nq_total; i += 32) {
        const int2 w = p.span[(long long)bi * nq_total + i];
        if (w.x < (j + 1) * 128 && w.y > j * 128) {
          first = min(first, i);
          last = max(last, i);
        }
      }
      first = __reduce_min_sync(0xffffffffu, first);
      last = __reduce_max_sync(0xffffffffu, last);
      return WorkItem{item.kv % p.Hkv, bi, j, first, last < 0 ? 0 : last - first + 1};
    }, [&](int it, const WorkItem& w) {
      if (it == 0) return true;
      if (!bounded_wait_w(kv_free, (it - 1) & 1, abort_flag, 702, p.err)) return false;
      load_kv(w.n, w.bi, w.q0);
      loads = it + 1;
      return true;
    });
    // every copy lands before the shared memory goes
    drain_wait(kv_full, (loads - 1) & 1);
  } else if (warp == 0) {
    // ------------------------------------------------ Q/dO stages (the whole
    // warp runs the loop, one lane issues)
    int c = 0;  // stages loaded
    bool ok = true;
    for (int it = 0; ok; ++it) {
      WorkItem w;
      if (!next_item<true>(queue, it, &w, abort_flag, p.err) || w.n < 0) break;
      const int pairs = p.G * w.nkv, t1 = part(pairs, rank + 1);
      for (int t = part(pairs, rank); t < t1; ++t, ++c) {
        const int st = c % QS;
        ok = c < QS || bounded_wait_w(&qdo_empty[st], ((c / QS) & 1) ^ 1, abort_flag, 701, p.err);
        if (!ok) break;
        if (lane == 0) {
          const int hn = w.n * p.G + t / w.nkv, i = w.j0 + t % w.nkv, bi = w.bi;
          uint8_t* sQ = sStage + st * STAGE;
          uint8_t* sdO = sQ + T::TILE;
          mbar_expect_tx(&qdo_full[st], C::REC + (int)sizeof(WinRecord) + (CAP ? 512 : 0));
#pragma unroll
          for (int k = 0; k < T::NCH; ++k) {
            tma_load_3d(sQ + k * T::CHUNK, &p.map_qkv, &qdo_full[st], hn * D + k * T::CW, i * 128, bi);
            tma_load_3d(sdO + k * T::CHUNK, &p.map_do, &qdo_full[st], hn * D + k * T::CW, i * 128, bi);
          }
          const int row = (bi * p.H + hn) * p.s_pad + i * 128;
          tma_load_2d(sQ + 2 * T::TILE, &p.map_aux, &qdo_full[st], 0, row);
          bulk_load(sQ + C::REC, p.rec + (long long)bi * nq_total + i, sizeof(WinRecord), &qdo_full[st]);
          if constexpr (CAP) bulk_load(sQ + C::NL2, p.nl2 + row, 512, &qdo_full[st]);
        }
        __syncwarp();
      }
      if (ok) release_item(queue, it);
    }
    // every copy lands before the shared memory goes, also when a wait
    // elsewhere in the block gives up later
    for (int k = (c > QS ? c - QS : 0); k < c; ++k) drain_wait(&qdo_full[k % QS], (k / QS) & 1);
  } else if (warp == 1 || warp == 10) {
    // the whole warp runs the issue loop, one elected lane issues.  One
    // issuer (fixed-order mode): warp 1 issues every sub-tile's products
    // in sub-tile order, so dV and dK take their products in a fixed order,
    // and warp 10 only reads the items
    // ------------------------------------------------ MMA issuers
    const bool issues = !(p.one_issuer && warp == 10);
    const int b0 = warp == 1 ? 0 : 1;  // this issuer's first sub-tile
    const int ustep = p.one_issuer ? 1 : 2;
    const uint32_t uZero = smem_u32(sZero);
    int tg = 0, ki = 0;  // stages, items with pairs before this one
    RingPos<QS> c;       // the sub-tile's stage
    const bool leader = elected();
    bool ok = true;
    // the 64 query rows of sub-tile half b start 64 b rows into every
    // chunk of the stage's tiles (whole swizzle atoms), and 64 b rows into
    // its extra rows; sub-tile u uses buffer b = u % 2
    auto stage_at = [&](RingPos<QS> c) { return smem_u32(sStage) + c.at * STAGE; };
    // K, V and their extra chunks in shared memory (head dims above 80):
    // the extra chunk is 128 rows of 16 bytes, K-major core matrices
    // without swizzle, its upper 8 columns the zeros
    const uint32_t uK = smem_u32(sKV), uV = uK + T::TILE;
    const uint32_t uKx = uK + 2 * T::TILE, uVx = uKx + C::AUX;
    const uint64_t dK = T::kmajor(uK, 0), dV = T::kmajor(uV, 0);
    const uint64_t dKx = sdesc(uKx, uZero - uKx, 128, 0u), dVx = sdesc(uVx, uZero - uVx, 128, 0u);
    auto issue_s = [&](int b, RingPos<QS> c) {
      const uint32_t tSb = tS + 64 * b;
      const uint64_t q = T::kmajor(stage_at(c) + 64 * T::SWB * b, 0);
      const uint32_t uA = stage_at(c) + 2 * T::TILE + 64 * 16 * b;
      if (leader) {
        if constexpr (C::KV_TMEM) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            umma_bf16_tmem_a_1(tSb, tKA + kk * 8, q + T::kmajor_step(kk), ID_S, kk > 0);
          umma_bf16_tmem_a_1(tSb, tKA + D / 2, sdesc(uA, uZero - uA, 128, 0u), ID_S, 1);
        } else {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            umma_bf16_1(tSb, dK + T::kmajor_step(kk), q + T::kmajor_step(kk), ID_S, kk > 0);
          umma_bf16_1(tSb, dKx, sdesc(uA, uZero - uA, 128, 0u), ID_S, 1);
        }
        umma_commit_1(&s_full[b]);
      }
      __syncwarp();
    };
    auto issue_dp = [&](int b, RingPos<QS> c) {
      const uint32_t tdPb = tdP + 64 * b;
      const uint64_t o = T::kmajor(stage_at(c) + T::TILE + 64 * T::SWB * b, 0);
      const uint32_t uA = stage_at(c) + 2 * T::TILE + 64 * 16 * b;
      if (leader) {
        if constexpr (C::KV_TMEM) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            umma_bf16_tmem_a_1(tdPb, tVA + kk * 8, o + T::kmajor_step(kk), ID_S, kk > 0);
          umma_bf16_tmem_a_1(tdPb, tVA + D / 2, sdesc(uA, uZero - uA, 128, 0u), ID_S, 1);
        } else {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            umma_bf16_1(tdPb, dV + T::kmajor_step(kk), o + T::kmajor_step(kk), ID_S, kk > 0);
          umma_bf16_1(tdPb, dVx, sdesc(uA, uZero - uA, 128, 0u), ID_S, 1);
        }
        umma_commit_1(&dp_full[b]);
      }
      __syncwarp();
    };
    auto wait_stage = [&](RingPos<QS> c) {
      return bounded_wait_w(&qdo_full[c.at], c.round, abort_flag, 711, p.err);
    };
    for (int it = 0; ok; ++it) {
      WorkItem w;
      if (!next_item(queue, it, &w, abort_flag, p.err)) { ok = false; break; }
      if (w.n < 0) break;
      const int pairs = p.G * w.nkv, T_iter = part(pairs, rank + 1) - part(pairs, rank), U = 2 * T_iter;
      if (U == 0 || !issues) continue;
      ok = bounded_wait_w(kv_ready, ki & 1, abort_flag, 712, p.err) &&
           (C::KV_TMEM || bounded_wait_w(kv_full, it & 1, abort_flag, 716, p.err)) && wait_stage(c);
      if (!ok) break;
      tc_fence_after();
      // sub-tiles 0 and 1 share the first stage (U is even)
      for (int u = b0; u < 2; u += ustep) {
        issue_s(u, c);
        issue_dp(u, c);
      }
      for (int u = b0; u < U; u += ustep) {
        const int b = u & 1;
        const uint32_t phase = (tg + (u >> 1)) & 1;
        const uint32_t tSb = tS + 64 * b, tdPb = tdP + 64 * b;
        const uint64_t dQm = T::mnmajor(stage_at(c), 4 * b), dOm = T::mnmajor(stage_at(c) + T::TILE, 4 * b);
        const bool more = u + 2 < U;
        const RingPos<QS> ahead = c.next();
        // dV += P^T(u) dO(u): the P^T pairs sit over the first 32 columns of
        // buffer b; dO rows 64b.. are K blocks 4b..4b+3 of the stage's tile
        ok = bounded_wait_w(&p_full[b], phase, abort_flag, 713, p.err);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16_tmem_a_1(tdV, tSb + kk * 8, dOm + T::mnmajor_step(kk), ID_KV, 1);
        }
        __syncwarp();
        if (more) {
          // S(u+2) overwrites P^T(u), after dV(u) in issue order
          ok = wait_stage(ahead);
          if (!ok) break;
          tc_fence_after();
          issue_s(b, ahead);
        }
        // dK += dS^T(u) Q(u)
        ok = bounded_wait_w(&ds_full[b], phase, abort_flag, 714, p.err);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16_tmem_a_1(tdK, tdPb + kk * 8, dQm + T::mnmajor_step(kk), ID_KV, 1);
          umma_commit_1(&qdo_empty[c.at]);
        }
        __syncwarp();
        // dP(u+2) overwrites dS^T(u), after dK(u) in issue order
        if (more) issue_dp(b, ahead);
        if (ustep == 2 || b == 1) c = ahead;
      }
      if (!ok) break;
      // all_done counts two commits: one per issuer, or both from one
      if (leader) {
        umma_commit_1(all_done);
        if (p.one_issuer) umma_commit_1(all_done);
      }
      __syncwarp();
      tg += T_iter;
      ++ki;
    }
    if (!ok) {
      if (leader) umma_commit_1(&drain[b0]);
      drain_wait(&drain[b0], 0);
    }
  } else {
    // ------------------------------------------------ compute (warps 2..9)
    const int quarter = warp & 3;
    const int b = (warp - 2) >> 2;  // group = buffer = sub-tile parity
    const int r = quarter * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t tSb = tS + 64 * b, tdPb = tdP + 64 * b;
    const uint32_t tOut = (b == 0 ? tdV : tdK) + lane_off;  // this group's accumulator
    uint32_t zero[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) zero[c] = 0u;
#pragma unroll
    for (int cc = 0; cc < D / 16; ++cc) tmem_st16_nw(tOut + cc * 16, zero);
    if constexpr (!C::KV_TMEM) {
      // the extra chunk of this thread's K row (group 0: 1 in columns 0..2)
      // or V row (group 1: in columns 3..5), which pick the three terms of
      // -LSE sqrt(d) and of -D from the query's extra row
      reinterpret_cast<uint4*>(sKV + 2 * T::TILE + b * C::AUX)[r] =
          b ? make_uint4(0u, 0x3F800000u, 0x3F803F80u, 0u) : make_uint4(0x3F803F80u, 0x00003F80u, 0u, 0u);
      fence_proxy_async_smem();
    }
    int tg = 0, ki = 0;  // stages, items with pairs before this one
    bool ok = true;
    for (int it = 0; ok; ++it) {
      WorkItem item;
      if (!next_item(queue, it, &item, abort_flag, p.err) || item.n < 0) break;
      const int g = item.n, bi = item.bi, j = item.q0, i0 = item.j0, n_i = item.nkv;
      const int kvp = j * 128 + r;
      const int t0 = part(p.G * n_i, rank), T_iter = part(p.G * n_i, rank + 1) - t0;
      if (T_iter == 0) {
        ok = __all_sync(0xffffffffu, bounded_wait(kv_full, it & 1, abort_flag, 725, p.err));
        if (!ok) break;
        if (lane == 0) mbar_arrive(kv_free);
        if (n_i == 0 && rank == 0 && kvp < p.s) {
          // nothing sees this key tile
          uint4* row = reinterpret_cast<uint4*>(p.dqkv + ((long long)bi * p.s + kvp) * p.width +
                                                (b == 0 ? p.v_col : p.k_col) + (long long)g * D);
#pragma unroll
          for (int cc = 0; cc < D / 8; ++cc) row[cc] = make_uint4(0u, 0u, 0u, 0u);
        }
        continue;
      }
      if constexpr (C::KV_TMEM) {
        // K (group 0) or V (group 1) row of this thread (zeros past the
        // sequence) into TMEM with the extra chunk: K picks the three terms of
        // -LSE sqrt(d) (columns 0..2 of the query's extra row), V those of -D
        // (columns 3..5)
        uint32_t w[D / 2 + 8];
        ok = __all_sync(0xffffffffu, bounded_wait(kv_full, it & 1, abort_flag, 725, p.err));
        if (!ok) break;
        load_tile_row<D>(sKV + b * T::TILE, r, w);
        w[D / 2] = b ? 0u : 0x3F803F80u;
        w[D / 2 + 1] = b ? 0x3F800000u : 0x00003F80u;
        w[D / 2 + 2] = b ? 0x3F803F80u : 0u;
#pragma unroll
        for (int c = 3; c < 8; ++c) w[D / 2 + c] = 0u;
        tmem_store_row<D / 2 + 8>((b ? tVA : tKA) + lane_off, w);
        __syncwarp();
        if (lane == 0) mbar_arrive(kv_free);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(kv_ready);
      for (int u = b; u < 2 * T_iter; u += 2) {
        const int t = u >> 1;
        const int q0 = (i0 + (t0 + t) % n_i) * 128 + 64 * b;
        const int tt = tg + t;
        const uint8_t* stage = sStage + (tt % QS) * STAGE;
        // the stage's windows and (with a cap) -LSE's, read while the scores are
        // still being made: the products take most of the shared memory's
        // bandwidth, and loads among the exponentials waited for it (dK/dV of
        // 8192 x (32 + 8 + 8) heads of 128, capped: 963 us, 930 so).  With K and V
        // in TMEM there is room for them there and the registers are worth more
        // (32 heads of 80: 768 us, 869 so).
        constexpr bool EARLY = CAP && !C::KV_TMEM;
        ok = bounded_wait(&qdo_full[tt % QS], (tt / QS) & 1, abort_flag, 724, p.err);
        const WinRecord* rec = reinterpret_cast<const WinRecord*>(stage + C::REC);
        const int2 cut = rec->cut[b];
        const uint64_t* late = reinterpret_cast<const uint64_t*>(stage + C::NL2) + 32 * b;
        uint64_t nl2[EARLY ? 32 : 1];
        if constexpr (EARLY) {
          const ulonglong2* from = reinterpret_cast<const ulonglong2*>(stage + C::NL2) + 16 * b;
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const ulonglong2 v = from[k];
            nl2[2 * k] = v.x;
            nl2[2 * k + 1] = v.y;
          }
        }
        ok = ok && bounded_wait(&s_full[b], tt & 1, abort_flag, 721, p.err);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        tc_fence_after();
        // ---- phase 1: P^T = exp2 of the modified scores - LSE log2(e)
        const bool all = cut.x <= j * 128 && cut.y >= j * 128 + 128;
        const int2* win = rec->row + 64 * b;
        auto on = [&](int x) {
          const int2 w = win[x];
          return (unsigned)(kvp - w.x) < (unsigned)w.y;
        };
        auto seen = [&](const uint32_t (&sv)[64]) { return largest_of(sv, on); };
        float pe[64];
        uint32_t pk[32];
        {
          uint32_t sv[64];
          const float am = load_scores<true>(tSb + lane_off, sv);
          auto lse2 = [&](int x) -> uint64_t {
            if constexpr (EARLY) return nl2[x / 2];
            else if constexpr (CAP) return late[x / 2];
            else return 0ull;
          };
          if constexpr (!BIAS) {
            probabilities<CAP, true>(p, sv, am, pe, pk, all, lse2, on, seen);
          } else {
            const float slope2 = p.slopes[g * p.G + (t0 + t) / n_i] * 1.4426950408889634f;
            // along the queries; with a causal mask those before the key are masked
            const BiasLine bl = bias_line(slope2, kvp, q0, 64, false, p.causal != 0);
            if (!__any_sync(0xffffffffu, bl.mixed)) {
              const uint64_t step2 = both(bl.step), base2 = both(bl.base);
              auto add = [&](int x) {
                return CAP ? add2(lse2(x), on_line(x, step2, base2)) : on_line(x, step2, base2);
              };
              probabilities<CAP, true>(p, sv, am, pe, pk, all, add, on, seen);
            } else {
              const float dist = (float)(kvp - q0);
              auto add = [&](int x) {
                return add2(lse2(x), f2(-slope2 * fabsf(dist - (float)x), -slope2 * fabsf(dist - (float)(x + 1))));
              };
              probabilities<CAP, true>(p, sv, am, pe, pk, all, add, on, seen);
            }
          }
        }
        tmem_st32(tSb + lane_off, pk);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[b]);
        // ---- phase 2: dx^T = P^T (1 - u^2) dP'^T (dP' offset by -D)
        ok = bounded_wait(&dp_full[b], tt & 1, abort_flag, 722, p.err);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        tc_fence_after();
        uint32_t dr[64];
        tmem_ld32_nw(tdPb + lane_off, dr);
        tmem_ld32_nw(tdPb + lane_off + 32, dr + 32);
        tmem_wait_ld(dr);
        if (!all) mask_gradient(dr, pe);
        uint32_t o[32];
#pragma unroll
        for (int k = 0; k < 64; k += 2) {
          const float2 v = f2split(mul2(f2(pe[k], pe[k + 1]), f2(__uint_as_float(dr[k]), __uint_as_float(dr[k + 1]))));
          o[k / 2] = pack_bf16(v.x, v.y);
        }
        tmem_st32(tdPb + lane_off, o);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ds_full[b]);
      }
      tg += T_iter;
      // epilogue: group 0 writes dV, group 1 dK, once both issuers' products
      // are done (TMEM loads by every lane, stores only for rows inside the
      // sequence), and zeroes its accumulator for the next item
      if (ok) ok = __all_sync(0xffffffffu, bounded_wait(all_done, ki & 1, abort_flag, 723, p.err));
      if (!ok) break;
      ++ki;
      tc_fence_after();
      // stored by TMA: whole lines, rows past the sequence left out (for the
      // cluster's sum: units of four fp32 columns by 128 rows, in the stages,
      // which every product has read)
      uint8_t* tile = sOut + b * T::TILE;
      uint4* sums = reinterpret_cast<uint4*>(sStage) + b * (D / 4) * 128;
      const float sc = b == 0 ? 1.f : p.scale;
      if (C::KV_TMEM && lane == 0) bulk_wait_read0();  // this warp's part of the tile is free
      __syncwarp();
#pragma unroll
      for (int cc = 0; cc < D / 16; ++cc) {
        uint32_t v[16];
        tmem_ld16_nw(tOut + cc * 16, v);
        tmem_wait_ld(v);
        tmem_st16_nw(tOut + cc * 16, zero);
        if (split == 1) {
          store_tile16<D>(tile, r, cc, v, sc);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            sums[(4 * cc + k) * 128 + r] = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (split == 1 && kvp < p.s) {
          for (int c = 0; c < T::NCH; ++c)
            tma_store_3d(&p.map_out, tile + c * T::CHUNK + quarter * 32 * T::SWB,
                         (b == 0 ? p.v_col : p.k_col) + g * D + c * T::CW, kvp, bi);
          bulk_commit();
        }
        if (!C::KV_TMEM) {
          bulk_wait_read0();
          mbar_arrive(kv_free);
        }
      }
      __syncwarp();
    }
    if (lane == 0) bulk_wait0();  // before the shared memory goes
  }

  if (split > 1) {
    // every CTA comes here, also after a timeout
    static_assert(QS * STAGE >= 128 * 2 * D * 4, "the sums' columns");
    __syncwarp();
    cluster_sync_all();
    const volatile WorkItem* item = queue.item(0);
    const int T_all = p.G * item->nkv, j = item->q0, bi = item->bi, g = item->n;
    if (warp >= 2 && warp < 10 && T_all > 0) {
      const int rows = 128 / split, r0 = rank * rows;
      const uint32_t mine = smem_u32(sStage);
      for (int unit = threadIdx.x - 64; unit < rows * (2 * D / 16); unit += 256) {
        const int row = r0 + unit % rows, cc = unit / rows;  // 16 columns of dV, then of dK
        float acc[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) acc[k] = 0.f;
        for (int c = 0; c < split; ++c) {
          if (part(T_all, c + 1) == part(T_all, c)) continue;  // it had no pairs
          const uint32_t from = cluster_addr(mine, c) + (4 * cc * 128 + row) * 16;
          float4 v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = ld_cluster_f32x4(from + k * 2048);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            acc[4 * k] += v[k].x;
            acc[4 * k + 1] += v[k].y;
            acc[4 * k + 2] += v[k].z;
            acc[4 * k + 3] += v[k].w;
          }
        }
        const int kv_row = j * 128 + row;
        if (kv_row < p.s) {
          const bool is_v = cc < D / 16;
          __nv_bfloat16* dst = p.dqkv + ((long long)bi * p.s + kv_row) * p.width +
                               (is_v ? p.v_col + 16 * cc : p.k_col + 16 * cc - D) + (long long)g * D;
          store_row16(dst, reinterpret_cast<const uint32_t*>(acc), is_v ? 1.f : p.scale);
        }
      }
    }
    __syncwarp();
    cluster_sync_all();  // the others have read this CTA's sums
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
}

// ===========================================================================
// dQ
// ===========================================================================
// Shared memory of the dQ kernel: dQ on its way out, a ring of pairs of tiles
// ((Q, dO), (K_0, V_0), (K_1, V_1), ... of one item after the other), barriers.
// (Each wait of an issuing warp costs a hundred cycles, and its loop bounds the
// kernel as much as the products do: one barrier for two tiles.)
template <int D>
struct ModDqCfg {
  using T = TileGeom<D>;
  static constexpr int CTL = 640;
  static constexpr int FIT = (232448 - T::TILE - CTL) / (2 * T::TILE);
  static constexpr int NP = FIT > 5 ? 5 : FIT;
  static constexpr int SMEM = (1 + 2 * NP) * T::TILE + CTL;
};

// One work item per 128-row query tile of one head, over the key tiles that
// some row of it sees, in 64-key sub-tiles: sub-tile u is the half u % 2 of
// tile u / 2.  Q and dO sit in TMEM as the A operands of S = Q K^T and dP = dO
// V^T; dS goes over the first 32 columns of its dP buffer as the A operand of
// dQ += dS K.  Compute warps 2..5 take the even sub-tiles, 6..9 the odd ones,
// with issuing warps 1 and 10: S(u), dP(u), S(u+2) (once S(u) is read), dQ(u)
// (after dS(u)), dP(u+2).  A row's window, LSE and D are scalars of its thread.
// Persistent like the forward: warp 11 takes the items, warp 0 loads the next
// one's Q and dO and its first keys during the current one.  (A CTA of its own
// per item spent 11,000 cycles outside its loop, of 25,000 with documents of
// 1500: start and TMEM 3,300, the first loads 2,500, the stores 900, the next
// CTA's launch 1,400.)
// TMEM: S [0, 128), dP [128, 256) as two 64-column buffers each, dQ at 256,
// Q at 256 + D, dO at 256 + 1.5 D.
template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(384, 1) attn_mod_dq_kernel(const __grid_constant__ ModBwdParams p) {
  using T = TileGeom<D>;
  using C = ModDqCfg<D>;
  constexpr int NP = C::NP;
  static_assert(NP >= 3, "Q, dO, K and V of two tiles");
  static_assert(256 + 2 * D <= 512, "TMEM columns");
  static_assert((2 * NP + 17) * 8 + WORK_BYTES + 8 <= C::CTL, "control block");
  constexpr uint32_t ID_S = idesc_bf16(128, 64, false, false);
  constexpr uint32_t ID_DQ = idesc_bf16(128, D, false, true);
  constexpr uint32_t COL_DQ = 256, COL_Q = 256 + D, COL_DO = 256 + D + D / 2;

  // the tiles' swizzle needs 1024-byte alignment, which the declaration gives
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sOut = smem;                 // dQ
  uint8_t* sRing = smem + T::TILE;
  uint8_t* control = sRing + 2 * NP * T::TILE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(control + WORK_BYTES);
  // (read by 8 compute warps, 2 issuers, the loads)
  const WorkQueue queue{control, bars, bars + 2, bars + 4};
  uint64_t* qo_ready = bars + 5;   // Q, dO copied to TMEM, dQ zeroed (8 compute warps)
  uint64_t* s_full = bars + 6;     // [2] S(u) in buffer u % 2
  uint64_t* s_free = bars + 8;     // [2] S(u) read (4 warps of the group)
  uint64_t* dp_full = bars + 10;   // [2]
  uint64_t* ds_full = bars + 12;   // [2] dS(u) written (4 warps)
  uint64_t* all_done = bars + 14;  // both issuers' last products of an item done
  uint64_t* drain = bars + 15;     // [2], one per issuer
  uint64_t* t_full = bars + 17;    // [NP]
  uint64_t* t_empty = t_full + NP; // [NP], once per issuer (both sub-tiles' products of K and V)
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(t_empty + NP);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = warp_id();
  const int lane = lane_id();
  if (threadIdx.x == 0) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(&queue.full[b], 1);
      mbar_init(&queue.empty[b], 11);
      mbar_init(&s_full[b], 1);
      mbar_init(&s_free[b], 4);
      mbar_init(&dp_full[b], 1);
      mbar_init(&ds_full[b], 4);
      mbar_init(&drain[b], 1);
    }
    mbar_init(queue.answered, 1);
    mbar_init(qo_ready, 8);
    mbar_init(all_done, 2);
    for (int k = 0; k < NP; ++k) {
      mbar_init(&t_full[k], 1);
      mbar_init(&t_empty[k], 2);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch(&p.map_qkv);
    tma_prefetch(&p.map_do);
    tma_prefetch(&p.map_out);
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const uint32_t tS = tmem;         // + 64 b
  const uint32_t tdP = tmem + 128;  // + 64 b
  const uint32_t tdQ = tmem + COL_DQ;
  const uint32_t tQA = tmem + COL_Q;
  const uint32_t tOA = tmem + COL_DO;
  bool took_last = false;

  if (warp == 11) {
    // ------------------------------------------------ items (the whole warp)
    took_last = publish_items(queue, blockIdx.x, gridDim.x - 1, true, abort_flag, p.err, [&](int block) {
      // the last (with a causal mask heaviest) query tiles first; the query
      // heads of one key/value head are adjacent
      const Item w = item_of(p.order_q, block);
      const int i = p.n_t - 1 - w.tile, bi = w.kv / p.Hkv;
      // key tiles [j0, j0 + nkv) hold every key that some row sees
      const int2 span = p.span[(long long)bi * p.n_t + i];
      const int j0 = span.x < span.y ? span.x / 128 : 0;
      return WorkItem{w.kv % p.Hkv * p.G + w.sub, bi, i * 128, j0, span.x < span.y ? (span.y + 127) / 128 - j0 : 0};
    }, [](int, const WorkItem&) { return true; });
  } else if (warp == 0) {
    // ------------------------------------------------ loads (the whole warp
    // runs the loop, one lane issues)
    int c = 0;  // pairs loaded
    // columns x of `first` and y of `second`, from the same row
    auto load_pair = [&](const CUtensorMap* first, int x, const CUtensorMap* second, int y, int row, int bi) -> bool {
      const int st = c % NP;
      if (c >= NP && !bounded_wait_w(&t_empty[st], ((c / NP) & 1) ^ 1, abort_flag, 731, p.err)) return false;
      if (lane == 0) {
        uint8_t* to = sRing + 2 * st * T::TILE;
        mbar_expect_tx(&t_full[st], 2 * T::TILE);
#pragma unroll
        for (int k = 0; k < T::NCH; ++k) tma_load_3d(to + k * T::CHUNK, first, &t_full[st], x + k * T::CW, row, bi);
#pragma unroll
        for (int k = 0; k < T::NCH; ++k)
          tma_load_3d(to + T::TILE + k * T::CHUNK, second, &t_full[st], y + k * T::CW, row, bi);
      }
      ++c;
      return true;
    };
    bool ok = true;
    for (int it = 0; ok; ++it) {
      WorkItem w;
      if (!next_item<true>(queue, it, &w, abort_flag, p.err) || w.n < 0) break;
      if (w.nkv == 0) {
        release_item(queue, it);
        continue;
      }
      ok = load_pair(&p.map_qkv, w.n * D, &p.map_do, w.n * D, w.q0, w.bi);
      const int k_col = p.k_col + w.n / p.G * D, v_col = p.v_col + w.n / p.G * D;
      for (int j = w.j0; ok && j < w.j0 + w.nkv; ++j)
        ok = load_pair(&p.map_qkv, k_col, &p.map_qkv, v_col, j * 128, w.bi);
      release_item(queue, it);
    }
    // every copy lands before the shared memory goes, also when a wait elsewhere
    // in the block gives up later
    for (int k = (c > NP ? c - NP : 0); k < c; ++k) drain_wait(&t_full[k % NP], (k / NP) & 1);
  } else if (warp == 1 || warp == 10) {
    // ------------------------------------------------ MMA issuers (the whole
    // warp runs the loop, one elected lane issues).  One issuer (fixed-order
    // mode): warp 1 issues every sub-tile's products in sub-tile order, so dQ
    // takes its products in a fixed order, and warp 10 only reads the items.
    const bool issues = !(p.one_issuer && warp == 10);
    const int b0 = warp == 1 ? 0 : 1;  // this issuer's first sub-tile
    const int ustep = p.one_issuer ? 1 : 2;
    const uint32_t ring = smem_u32(sRing);
    // the 64 key rows of half b start 64 b rows into every chunk of K's and
    // V's tiles (whole swizzle atoms); sub-tile u uses buffer b = u % 2.  tg,
    // qi: key tiles, items with keys before this one
    int tg = 0, qi = 0;
    RingPos<NP> c;  // the pair of K and V (before an item's first, of Q and dO)
    const bool leader = elected();
    auto k_tile = [&](RingPos<NP> c) { return ring + 2 * c.at * T::TILE; };
    auto landed = [&](RingPos<NP> c) { return bounded_wait_w(&t_full[c.at], c.round, abort_flag, 741, p.err); };
    auto issue_s = [&](int b, RingPos<NP> c) {
      const uint32_t tSb = tS + 64 * b;
      const uint64_t k = T::kmajor(k_tile(c) + 64 * T::SWB * b, 0);
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) umma_bf16_tmem_a_1(tSb, tQA + kk * 8, k + T::kmajor_step(kk), ID_S, kk > 0);
        umma_commit_1(&s_full[b]);
      }
      __syncwarp();
    };
    auto issue_dp = [&](int b, RingPos<NP> c) {
      const uint32_t tdPb = tdP + 64 * b;
      const uint64_t v = T::kmajor(k_tile(c) + T::TILE + 64 * T::SWB * b, 0);
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) umma_bf16_tmem_a_1(tdPb, tOA + kk * 8, v + T::kmajor_step(kk), ID_S, kk > 0);
        umma_commit_1(&dp_full[b]);
      }
      __syncwarp();
    };
    bool ok = true;
    for (int it = 0; ok; ++it) {
      WorkItem w;
      if (!next_item(queue, it, &w, abort_flag, p.err)) { ok = false; break; }
      if (w.n < 0) break;
      if (w.nkv == 0 || !issues) continue;
      const int U = 2 * w.nkv;
      ok = bounded_wait_w(qo_ready, qi & 1, abort_flag, 742, p.err);
      if (!ok) break;
      if (lane == 0) {
        // the tiles of Q and dO are free
        uint64_t* bar = &t_empty[c.at];
        mbar_arrive(bar);
        if (p.one_issuer) mbar_arrive(bar);
      }
      c = c.next();
      ok = landed(c);
      if (!ok) break;
      tc_fence_after();
      // sub-tiles 0 and 1 share the first tiles (U is even)
      for (int u = b0; u < 2; u += ustep) {
        issue_s(u, c);
        issue_dp(u, c);
      }
      for (int u = b0; u < U; u += ustep) {
        const int b = u & 1;
        const uint32_t phase = (tg + (u >> 1)) & 1;
        const bool more = u + 2 < U;
        const RingPos<NP> ahead = c.next();
        if (more) {
          // S(u+2) once the group has read S(u)
          ok = bounded_wait_w(&s_free[b], phase, abort_flag, 743, p.err) && landed(ahead);
          if (!ok) break;
          tc_fence_after();
          issue_s(b, ahead);
        }
        // dQ += dS(u) K_u: key rows 64b.. are K blocks 4b..4b+3 of the tile
        ok = bounded_wait_w(&ds_full[b], phase, abort_flag, 744, p.err);
        if (!ok) break;
        tc_fence_after();
        const uint64_t k = T::mnmajor(k_tile(c), 4 * b);
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16_tmem_a_1(tdQ, tdP + 64 * b + kk * 8, k + T::mnmajor_step(kk), ID_DQ, 1);
          umma_commit_1(&t_empty[c.at]);
        }
        __syncwarp();
        if (more) issue_dp(b, ahead);  // over dS(u), after dQ(u) in issue order
        if (ustep == 2 || b == 1) c = ahead;
      }
      if (!ok) break;
      // all_done counts two commits: one per issuer, or both from one
      if (leader) {
        umma_commit_1(all_done);
        if (p.one_issuer) umma_commit_1(all_done);
      }
      __syncwarp();
      tg += w.nkv;
      ++qi;
    }
    if (!ok) {
      if (leader) umma_commit_1(&drain[b0]);
      drain_wait(&drain[b0], 0);
    }
  } else {
    // ------------------------------------------------ compute (warps 2..9)
    const int quarter = warp & 3;
    const int b = (warp - 2) >> 2;  // group = buffer = sub-tile parity
    const int r = quarter * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t tSb = tS + 64 * b, tdPb = tdP + 64 * b;
    constexpr int CC = T::CW / 16, CH0 = (T::NCH + 1) / 2;
    const int cbeg = b == 0 ? 0 : CH0, cend = b == 0 ? CH0 : T::NCH;  // dQ's chunks of this group
    uint32_t zero[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) zero[k] = 0u;
    for (int cc = cbeg * CC; cc < cend * CC; ++cc) tmem_st16_nw(tdQ + lane_off + cc * 16, zero);
    int tg = 0, qi = 0;  // key tiles of the items before, items with keys
    bool ok = true;
    for (int it = 0; ok; ++it) {
      WorkItem w;
      if (!next_item(queue, it, &w, abort_flag, p.err) || w.n < 0) break;
      const int qpos = w.q0 + r;
      if (w.nkv == 0) {
        // no row of the tile sees a key
        if (b == 0 && qpos < p.s) {
          uint4* row = reinterpret_cast<uint4*>(p.dqkv + ((long long)w.bi * p.s + qpos) * p.width + (long long)w.n * D);
#pragma unroll
          for (int cc = 0; cc < D / 8; ++cc) row[cc] = make_uint4(0u, 0u, 0u, 0u);
        }
        continue;
      }
      const int2 win = key_window(p.row_begin, p.row_end, p.causal, p.s, w.bi, qpos);
      const float slope2 = BIAS ? p.slopes[w.n] * 1.4426950408889634f : 0.f;
      // this row's -LSE*log2(e) and dO.O sum (finite filler past the sequence)
      const float nl = p.nl2[((long long)w.bi * p.H + w.n) * p.s_pad + qpos];
      const float dsum = p.dsum[((long long)w.bi * p.H + w.n) * p.s_pad + qpos];
      {
        // Q (group 0) or dO (group 1) row of this thread into TMEM (zeros past
        // the sequence)
        uint32_t row[D / 2];
        const int c = tg + qi;
        ok = __all_sync(0xffffffffu, bounded_wait(&t_full[c % NP], (c / NP) & 1, abort_flag, 754, p.err));
        if (!ok) break;
        load_tile_row<D>(sRing + (2 * (c % NP) + b) * T::TILE, r, row);
        tmem_store_row<D / 2>((b == 0 ? tQA : tOA) + lane_off, row);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(qo_ready);
      }
      const int U = 2 * w.nkv;
      for (int u = b; u < U; u += 2) {
        const uint32_t phase = (tg + (u >> 1)) & 1;
        ok = bounded_wait(&s_full[b], phase, abort_flag, 751, p.err);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        tc_fence_after();
        // ---- phase 1: P (1 - u^2) of the 64 keys; [klo, khi) are visible
        const int kv0 = (w.j0 + (u >> 1)) * 128 + 64 * b;
        const int klo = max(win.x - kv0, 0), khi = min(win.y - kv0, 64);
        uint32_t sv[64];
        const float am = load_scores<true>(tSb + lane_off, sv);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[b]);
        const bool all = klo == 0 && khi == 64;
        auto on = [&](int x) { return x >= klo && x < khi; };
        auto seen = [&](const uint32_t (&sv)[64]) { return largest_within(sv, klo, khi); };
        float pe[64];
        {
          uint32_t pk[32];
          const uint64_t nl2 = f2(nl, nl);
          if constexpr (!BIAS) {
            auto add = [&](int) { return nl2; };
            probabilities<CAP, false>(p, sv, am, pe, pk, all, add, on, seen);
          } else {
            const BiasLine bl = bias_line(slope2, qpos, kv0, 64, p.causal != 0, false);
            if (!__any_sync(0xffffffffu, bl.mixed)) {
              const uint64_t step2 = both(bl.step), base2 = both(bl.base + nl);
              auto add = [&](int x) { return on_line(x, step2, base2); };
              probabilities<CAP, false>(p, sv, am, pe, pk, all, add, on, seen);
            } else {
              const float dist = (float)(qpos - kv0);
              auto add = [&](int x) {
                return add2(nl2, f2(-slope2 * fabsf(dist - (float)x), -slope2 * fabsf(dist - (float)(x + 1))));
              };
              probabilities<CAP, false>(p, sv, am, pe, pk, all, add, on, seen);
            }
          }
        }
        // ---- phase 2: dx = P (1 - u^2) (dP - D), over the first 32 columns of buffer b
        ok = bounded_wait(&dp_full[b], phase, abort_flag, 752, p.err);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        tc_fence_after();
        uint32_t dr[64];
        tmem_ld32_nw(tdPb + lane_off, dr);
        tmem_ld32_nw(tdPb + lane_off + 32, dr + 32);
        tmem_wait_ld(dr);
        if (!all) mask_gradient(dr, pe);
        uint32_t o[32];
        const uint64_t ds2 = f2(dsum, dsum);
#pragma unroll
        for (int k = 0; k < 64; k += 2) {
          const float2 v = f2split(
              mul2(f2(pe[k], pe[k + 1]), sub2(f2(__uint_as_float(dr[k]), __uint_as_float(dr[k + 1])), ds2)));
          o[k / 2] = pack_bf16(v.x, v.y);
        }
        tmem_st32(tdPb + lane_off, o);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ds_full[b]);
      }
      tg += w.nkv;
      // both issuers' products of the item are done
      if (ok) ok = __all_sync(0xffffffffu, bounded_wait(all_done, qi & 1, abort_flag, 753, p.err));
      if (!ok) break;
      ++qi;
      tc_fence_after();
      // each group's half of dQ out by TMA, and zeroed for the next item
      if (lane == 0) bulk_wait_read0();  // this warp's part of the tile is free
      __syncwarp();
      for (int cc = cbeg * CC; cc < cend * CC; ++cc) {
        uint32_t v[16];
        tmem_ld16_nw(tdQ + lane_off + cc * 16, v);
        tmem_wait_ld(v);
        tmem_st16_nw(tdQ + lane_off + cc * 16, zero);
        store_tile16<D>(sOut, r, cc, v, p.scale);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && qpos < p.s) {
        for (int c = cbeg; c < cend; ++c)
          tma_store_3d(&p.map_out, sOut + c * T::CHUNK + quarter * 32 * T::SWB, w.n * D + c * T::CW, qpos, w.bi);
        bulk_commit();
      }
    }
    if (lane == 0) bulk_wait0();  // before the shared memory goes
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // dK/dV started after the preparation had ended and let this kernel start,
  // so nothing above waited for it; but the call ends when both have
  if (took_last) wait_for_previous();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
}

// ===========================================================================
// What both need of the rows
// ===========================================================================
// The first b * n_t blocks write the windows of one query tile each; the
// others take 16 rows of one head per half-warp (whole lines in, and whole
// lines of the [head][row] outputs): D = dO . O in fp32, and from it and the
// log-sum-exp the per-row inputs of the two kernels.  A value as three bf16
// terms keeps 24 bits of it.
__device__ __forceinline__ void three_terms(float v, uint32_t (&t)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const __nv_bfloat16 h = __float2bfloat16(v);
    t[i] = (uint32_t)__bfloat16_as_ushort(h);
    v -= __bfloat162float(h);
  }
}

__global__ void __launch_bounds__(256) attn_mod_prep_kernel(int b, int s, int n_t, int H, int d, int causal, int cap,
                                                            float inv_scale, const int32_t* row_begin,
                                                            const int32_t* row_end, const __nv_bfloat16* o,
                                                            const __nv_bfloat16* dout, const float* lse,
                                                            WinRecord* rec, int2* span, float* dsum, float* nl2,
                                                            uint4* aux) {
  const int s_pad = n_t * 128;
  if ((int)blockIdx.x < b * n_t) {
    __shared__ int part[4][4];
    const int bi = blockIdx.x / n_t, t = blockIdx.x % n_t;
    const int r = threadIdx.x;
    WinRecord* out = rec + blockIdx.x;
    if (r < 128) {
      const int2 w = key_window(row_begin, row_end, causal, s, bi, t * 128 + r);
      out->row[r] = make_int2(w.x, w.y - w.x);
      const int lo = __reduce_min_sync(0xffffffffu, w.x < w.y ? w.x : INT32_MAX);
      const int hi = __reduce_max_sync(0xffffffffu, w.y);
      const int lo_cut = __reduce_max_sync(0xffffffffu, w.x), hi_cut = __reduce_min_sync(0xffffffffu, w.y);
      if ((r & 31) == 0) {
        part[r >> 5][0] = lo;
        part[r >> 5][1] = hi;
        part[r >> 5][2] = lo_cut;
        part[r >> 5][3] = hi_cut;
      }
    }
    __syncthreads();
    if (r == 0) {
      span[blockIdx.x] = make_int2(min(min(part[0][0], part[1][0]), min(part[2][0], part[3][0])),
                                   max(max(part[0][1], part[1][1]), max(part[2][1], part[3][1])));
      for (int h = 0; h < 2; ++h)
        out->cut[h] = make_int2(max(part[2 * h][2], part[2 * h + 1][2]), min(part[2 * h][3], part[2 * h + 1][3]));
      out->unused = make_int4(0, 0, 0, 0);
    }
    return;
  }
  const int sub = threadIdx.x & 15;
  const int groups = s_pad / 16;
  const int total = b * groups * H;
  const int stride = (int)(gridDim.x - b * n_t) * 16;
  const unsigned mask = 0xffffu << (threadIdx.x & 16);
  // whole half-warps step together: the shuffles below stay within one
  for (int it = (int)(blockIdx.x - b * n_t) * 16 + (threadIdx.x >> 4); it < total; it += stride) {
    const int hn = it % H, rg = it / H;
    const int bi = rg / groups, q0 = rg % groups * 16;
    float mine = 0.f;  // row q0 + sub
#pragma unroll 4
    for (int k = 0; k < 16; ++k) {
      float acc = 0.f;
      if (q0 + k < s && sub * 8 < d) {
        const int64_t at = (((int64_t)bi * s + q0 + k) * H + hn) * d + sub * 8;
        const uint4 x = *reinterpret_cast<const uint4*>(o + at), y = *reinterpret_cast<const uint4*>(dout + at);
        const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int m = 0; m < 4; ++m)
          acc = fmaf(bf16_lo(xw[m]), bf16_lo(yw[m]), fmaf(bf16_hi(xw[m]), bf16_hi(yw[m]), acc));
      }
#pragma unroll
      for (int m = 8; m > 0; m >>= 1) acc += __shfl_xor_sync(mask, acc, m);
      if (sub == k) mine = acc;
    }
    const int q = q0 + sub;
    const int64_t row = ((int64_t)bi * H + hn) * s_pad + q;
    float l = q < s ? lse[row] : 0.f;
    if (l == -INFINITY) l = 0.f;  // a row that sees nothing: every P is masked
    uint32_t a[3] = {0u, 0u, 0u}, c[3];
    if (!cap) three_terms(-l * inv_scale, a);
    three_terms(-mine, c);
    dsum[row] = mine;
    nl2[row] = -1.4426950408889634f * l;
    aux[row] = make_uint4(a[0] | (a[1] << 16), a[2] | (c[0] << 16), c[1] | (c[2] << 16), 0u);
  }
}

// CTAs that share one dK/dV item (a key tile's stream of up to `stream` query
// tiles): whichever of 1, 2, 4, 8 an estimate in query tiles makes shortest.  A CTA
// takes its part of the longest stream, and sharing costs it the sum over the
// cluster, a start and the persistence, some 3 + s tiles.  Clusters that do not fit
// at once (of four and eight, not every SM finds partners in its GPC) take a second
// round; with a causal mask it has the lighter items.  And no split beats the work
// of all SMs, dQ's 0.8 of dK/dV's with it, which fills what one leaves idle: that
// is why full rows share later than causal ones.  Windows, which live on the device,
// are taken to leave half of the pairs, unevenly, as a causal mask does.
// Measured, the whole backward in us at d = 128 by 1 / 2 / 4 / 8 (chosen: *):
//   108 items of up to 27 tiles   causal 61* / 73 / 88 / 161, all 91* / 102 / 107 / 182
//   108 items of up to 54 tiles   causal 105 / 86* / 105 / 183, all 136* / 149 / 168 / 236
//   108 items of up to 216 tiles  causal 377 / 259* / 283 / 372, all 477* / 497 / 528 / 625
//   36 items of up to 72 tiles    causal 130 / 79 / 52* / 82, all 136 / 83 / 75* / 107
//   9 items of up to 72 tiles     causal 130 / 78 / 50 / 38*, all 138 / 81 / 52 / 40*
// Over 1,335 such calls (4 to 152 items, d = 80, 96 and 128; causal, full, prefixes,
// documents seen both ways, a quarter padded; plain or capped and biased) the choice
// is 2% behind the best on average, at worst 46%; windows taken for full rows 3%, at
// worst 82%; up to three CTAs for two SMs and a dozen tiles each, whatever the mask,
// 9%, at worst twice.  (3 x 1111 rows of 12 + 4 + 4 heads of 96 behind prefixes of a
// quarter, 108 items of up to 27 tiles: 89 us, 78 by two; 3456 rows of 8 + 4 + 4 of
// 128, all keys of the first three quarters: 105 by two, 88 unshared.)
int split_for(int items, int stream, int n_t, bool uneven) {
  const double nsm = sm_count();
  const double mean = uneven ? stream * (n_t + 1) / (2.0 * n_t) : stream;
  double least = 0;
  int best = 1;
  for (int s = 1; s <= 8 && (s == 1 || stream >= 2 * s); s *= 2) {
    const double ctas = (double)items * s, part = (double)stream / s, cost = s == 1 ? 0 : 3 + s;
    const double room = nsm * (s <= 2 ? 1.0 : s == 4 ? 18.0 / 19 : 16.0 / 19);
    double t = part + cost;
    if (s > 1 && ctas > room) {
      if (ctas > 2 * room) break;
      t += (uneven ? 1 - room / ctas : 1.0) * part + cost;
    }
    t = std::max(t, (1.8 * items * mean + ctas * cost) / nsm);
    if (s == 1 || t < least) {
      least = t;
      best = s;
    }
  }
  return best;
}

template <int D, bool CAP, bool BIAS>
int launch_both(const ModBwdParams& p, int b, double pairs, cudaStream_t st) {
  constexpr int SMEM_KV = ModDkdvCfg<D>::SMEM, SMEM_Q = ModDqCfg<D>::SMEM;
  static_assert(SMEM_KV <= 232448 && SMEM_Q <= 232448, "tile sets exceed shared memory");
  static std::atomic<uint64_t> attr_kv{0}, attr_q{0};  // devices whose limit is set
  if (smem_limit_once(reinterpret_cast<const void*>(attn_mod_dkdv_kernel<D, CAP, BIAS>), SMEM_KV, &attr_kv) ||
      smem_limit_once(reinterpret_cast<const void*>(attn_mod_dq_kernel<D, CAP, BIAS>), SMEM_Q, &attr_q))
    return BPT_ECUDA;
  {
    ProfScope prof(PROF_ATTN_BWD, 8.0 * D * pairs * p.H * b, 0.0, st);
    // CTAs per item: see split_for
    const int items = p.n_t * p.Hkv * b;
    const int split = split_for(items, p.G * p.n_t, p.n_t, p.causal || p.row_begin || p.row_end);
    if (launch_dependent(attn_mod_dkdv_kernel<D, CAP, BIAS>, items * split, split, dim3(384), SMEM_KV, st, p) != cudaSuccess)
      return BPT_ECUDA;
  }
  ProfScope prof(PROF_ATTN_BWD, 2.0 * D * pairs * p.H * b, 0.0, st);
  return launch_dependent(attn_mod_dq_kernel<D, CAP, BIAS>, p.n_t * p.H * b, 1, dim3(384), SMEM_Q, st, p) == cudaSuccess
             ? BPT_OK
             : BPT_ECUDA;
}

template <int D>
int launch_for(const ModBwdParams& p, bool cap, int b, double pairs, cudaStream_t st) {
  if (p.slopes)
    return cap ? launch_both<D, true, true>(p, b, pairs, st) : launch_both<D, false, true>(p, b, pairs, st);
  return cap ? launch_both<D, true, false>(p, b, pairs, st) : launch_both<D, false, false>(p, b, pairs, st);
}

struct ModBwdWs {
  float *dsum, *nl2;
  uint4* aux;
  WinRecord* rec;
  int2* span;
};
size_t plan(const PackedDims& D, void* base, ModBwdWs* w) {
  size_t off = 0;
  auto take = [&](size_t bytes) {
    uint8_t* p = base ? reinterpret_cast<uint8_t*>(base) + off : nullptr;
    off += (bytes + 255) / 256 * 256;
    return p;
  };
  const size_t rows = (size_t)D.b * D.H * D.s_pad, tiles = (size_t)D.b * (D.s_pad / 128);
  w->dsum = reinterpret_cast<float*>(take(rows * 4));
  w->nl2 = reinterpret_cast<float*>(take(rows * 4));
  w->aux = reinterpret_cast<uint4*>(take(rows * 16));
  w->rec = reinterpret_cast<WinRecord*>(take(tiles * sizeof(WinRecord)));
  w->span = reinterpret_cast<int2*>(take(tiles * sizeof(int2)));
  return off;
}

}  // namespace

size_t attention_mod_bwd_ws_bytes(const PackedDims& D) {
  ModBwdWs w;
  return plan(D, nullptr, &w);
}

int attention_mod_bwd(const PackedDims& D, int causal, const bpt_score_mod& mod, const void* qkv, const void* o,
                      const float* lse, const void* dout, void* dqkv, void* ws, cudaStream_t st) {
  ModBwdWs w;
  plan(D, ws, &w);
  const bool cap = mod.softcap > 0.f;
  ModBwdParams p;
  memset(&p, 0, sizeof(p));
  const uint64_t rows = (uint64_t)D.b * D.H * D.s_pad;
  if (make_attn_map(&p.map_qkv, qkv, (int)D.b, (int)D.s, D.width, (int)D.d, 128) ||
      make_attn_map(&p.map_do, dout, (int)D.b, (int)D.s, D.H * D.d, (int)D.d, 128) ||
      make_attn_map(&p.map_out, dqkv, (int)D.b, (int)D.s, D.width, (int)D.d, 32) ||
      make_map_2d(&p.map_aux, w.aux, rows, 8, 8, 8, 128, 0))
    return BPT_EINVAL;
  p.s = (int)D.s;
  p.s_pad = (int)D.s_pad;
  p.H = (int)D.H;
  p.Hkv = (int)D.Hkv;
  p.G = (int)D.G;
  p.causal = causal;
  p.n_t = (int)(D.s_pad / 128);
  p.order_kv = item_order(p.n_t, 1, D.b * D.Hkv, 4 * D.G * D.s * D.d);
  p.order_q = item_order(p.n_t, D.G, D.b * D.Hkv, 4 * D.s * D.d);
  p.k_col = (int)(D.H * D.d);
  p.v_col = (int)((D.H + D.Hkv) * D.d);
  p.dsum = w.dsum;
  p.nl2 = w.nl2;
  p.rec = w.rec;
  p.span = w.span;
  p.qkv = reinterpret_cast<const __nv_bfloat16*>(qkv);
  p.dout = reinterpret_cast<const __nv_bfloat16*>(dout);
  p.dqkv = reinterpret_cast<__nv_bfloat16*>(dqkv);
  p.width = D.width;
  p.row_begin = mod.row_begin;
  p.row_end = mod.row_end;
  p.slopes = mod.slopes;
  p.scale = 1.f / sqrtf((float)D.d);
  p.scale_log2 = p.scale * 1.4426950408889634f;
  if (cap) {
    p.cap = cap_coef(mod.softcap, 1.0 / (mod.softcap * sqrt((double)D.d)), 1.0);
    p.cap_log2 = mod.softcap * 1.4426950408889634f;
  }
  p.one_issuer = D.det ? 1 : 0;
  p.err = device_error_word();
  if (!p.err) return BPT_ECUDA;
  const int nsm = sm_count();
  if (nsm <= 0) return BPT_ECUDA;
  const int tiles = (int)(D.b * p.n_t);
  {
    ProfScope prof(PROF_MISC, 0.0, 4.0 * D.rows * D.H * D.d + 28.0 * rows, st);
    const int64_t items = (int64_t)rows / 16;  // 16 per block and round
    const int blocks = (int)std::min<int64_t>((items + 15) / 16, (int64_t)nsm * 16);
    attn_mod_prep_kernel<<<tiles + blocks, 256, 0, st>>>(
        (int)D.b, p.s, p.n_t, p.H, (int)D.d, causal, cap, sqrtf((float)D.d), p.row_begin, p.row_end,
        reinterpret_cast<const __nv_bfloat16*>(o), p.dout, lse, w.rec, w.span, w.dsum, w.nl2, w.aux);
    if (cudaGetLastError() != cudaSuccess) return BPT_ECUDA;
  }
  // credited as without windows, which live on the device
  const double pairs = causal ? (double)D.s * (D.s + 1) / 2 : (double)D.s * D.s;
  const int b = (int)D.b;
  switch (D.d) {
    case 64: return launch_for<64>(p, cap, b, pairs, st);
    case 80: return launch_for<80>(p, cap, b, pairs, st);
    case 96: return launch_for<96>(p, cap, b, pairs, st);
    case 112: return launch_for<112>(p, cap, b, pairs, st);
    case 128: return launch_for<128>(p, cap, b, pairs, st);
    default: return BPT_EUNSUPPORTED;
  }
}

}  // namespace bpt
