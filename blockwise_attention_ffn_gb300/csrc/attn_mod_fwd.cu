// attn_mod_fwd.cu -- attention forward with a key window per query row, capped
// scores and a distance bias, on tcgen05 (bpt_attention_mod_fwd).
//
// The recurrence is that of the plain forward: for the key tiles j of a query
// tile, S = Q K_j^T, y = modified scores, m' = max(m, rowmax y),
// l = l 2^(m - m') + rowsum 2^(y - m'), O = O 2^(m - m') + 2^(y - m') V_j; at
// the end O / l and the log-sum-exp.  What differs:
//  * A tile's first and last key tile come from its rows' windows, so packed
//    documents, prefixes and padding cost only the tiles that some row sees.
//  * Scores are modified between the tensor core and the softmax.  With a cap
//    of at most 61, scores within 0.6 C (where a polynomial does for the tanh)
//    have exponentials between 2^-47 and 2^47: no maximum is looked for in such
//    a tile, m is at least 0 (with a bias the largest bias seen, less up to 8).
//    That leaves fp32 sums 2^72 for values times keys.  Tiles with a score beyond
//    0.6 C take their maximum: with m = 0 there too, P reached 2^88 and values of
//    2^39 over the keys overflowed.  Biased scores without a cap take the load's
//    own maximum and the nearest key's bias for an upper bound of theirs.
//  * Row sums are fp32 sums of the fp32 exponentials, so the log-sum-exp is an
//    fp32-exact output; the tensor core's row sums of bf16 P would be off by
//    up to 2^-9.
//  * P is rounded to bf16, V's type, to be an operand of the second product: by at
//    most 2^-8 of its value, with signs that do not build up.  Two terms of it would
//    double that product.  o is off by 1.7e-3 to 2.4e-3 (relative norm, its own bf16
//    rounding of 1.6e-3 included).
//
// Work item = one 128-row query tile of one head, the last (with a causal mask
// heaviest) tiles first.  The 128 keys of a tile are split in two halves, each with its own
// softmax warps (2..5, 6..9), MMA-issuing warp (1, 10), running maximum and O
// accumulator, merged at the end by the log-sum-exp rule: the modified softmax
// bounds the loop, and two warps per SM sub-partition hide each other's
// latency.
//
// A CTA is persistent: it takes further items by cluster launch control (the
// hardware's own queue of unstarted blocks, so no counter in memory and the
// order of the grid).  With windows an item is often a handful of key tiles,
// and a CTA of its own spent about 12,000 cycles on starting, TMEM, barriers,
// the first loads and its end, as much as ten key tiles.  Here warp 11 looks up
// the next item's windows and warp 0 loads its Q and K/V while the softmax is
// still in the current one, and its first S is made during the current item's
// merge.
//
// Measured at 8192 rows of 32 + 8 + 8 heads of 128, causal: 371 us plain scores
// (1,482 TFLOP/s of unmasked pairs), 430 capped (1,279; 812 where most scores are
// beyond the cap), 403 biased, 490 capped and biased; documents of 1500: 119 us, 139
// capped.  What bounds it: at d = 128 a step's products take
// 1,280 of 1,620 cycles (S reads both operands from shared memory, 48 cycles for
// 16 of depth and 64 columns), with a cap the chain S, modified softmax, P, PV of
// each half.  The issuing warps' loops are part of that chain: with a barrier per
// tile instead of per pair of K and V the plain scores took 434 us.
#include <math.h>
#include <string.h>

#include "../../include/bpt.h"
#include "attn_mod.cuh"
#include "internal.h"

namespace bpt {
int make_attn_map(CUtensorMap* map, const void* qkv, int b, int s, int64_t ld, int d, int box_rows);

namespace {

struct ModFwdParams {
  CUtensorMap map_qkv;  // 3-D {width, s, b}, box {CW, 128, 1}
  CUtensorMap map_o;    // 3-D {H d, s, b}, box {CW, 32, 1}
  int s, s_pad, H, G, causal;
  int k_col, v_col;
  ItemOrder order;
  __nv_bfloat16* o;
  float* lse;
  const int32_t *row_begin, *row_end;
  const float* slopes;
  float scale_log2;  // log2(e)/sqrt(d)
  CapCoef cap;       // capped scores in log2 units
  float bounded;  // largest |z| of capped scores that need no maximum (negative: none)
  unsigned int* err;
};

// TMEM: S of half b as two 64-column buffers at 128 b, O_b at 256 + b D.
// Shared memory: two Q tiles, a ring of pairs of K and V tiles as a step takes
// them ((K_0, -), (K_1, V_0), (K_2, V_1), ..., (-, V_last), then the next item's),
// the merge's maxima and sums, barriers.
template <int D>
struct ModFwdCfg {
  using T = TileGeom<D>;
  static constexpr int RED = 4 * 128 * 4;
  static constexpr int CTL = 640;  // barriers, work items, answers
  static constexpr int FIT = (232448 - 2 * T::TILE - RED - CTL) / (2 * T::TILE);
  static constexpr int NP = FIT > 5 ? 5 : FIT;
  static constexpr int SMEM = (2 + 2 * NP) * T::TILE + RED + CTL;
  static constexpr uint32_t COL_O = 256;
};

template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(384, 1) attn_mod_fwd_kernel(const __grid_constant__ ModFwdParams p) {
  using T = TileGeom<D>;
  using C = ModFwdCfg<D>;
  constexpr int NP = C::NP;
  static_assert(NP >= 2, "K and V of two steps");
  static_assert(C::COL_O + 2 * D <= 512, "TMEM columns");
  static_assert((2 * NP + 30) * 8 + WORK_BYTES + 8 <= C::CTL, "control block");
  constexpr uint32_t IDESC_S = idesc_bf16(128, 64, false, false);
  constexpr uint32_t IDESC_PV = idesc_bf16(128, D, false, true);
  constexpr float NEG_INF = -INFINITY;
  constexpr float LN2 = 0.6931471805599453f;

  // the tiles' swizzle needs 1024-byte alignment, which the declaration gives
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + 2 * T::TILE;
  float* red_m = reinterpret_cast<float*>(sKV + 2 * NP * T::TILE);  // [half][row]
  float* red_l = red_m + 256;
  uint8_t* control = reinterpret_cast<uint8_t*>(red_l + 256);
  uint64_t* bars = reinterpret_cast<uint64_t*>(control + WORK_BYTES);
  // (read by 8 softmax warps, 2 issuers, the loads)
  const WorkQueue queue{control, bars, bars + 2, bars + 19};
  uint64_t* q_full = bars + 4;          // [2]
  uint64_t* q_empty = bars + 6;         // [2] both issuers' last S, 8 warps' O stored from it
  uint64_t* s_full = bars + 8;          // [half][buffer]
  uint64_t* p_full = bars + 12;         // [half][buffer] 4 warps
  uint64_t* pv_done = bars + 16;        // [half]
  uint64_t* o_free = bars + 18;         // both O's read (8 warps)
  uint64_t* drain = bars + 20;          // [half]
  uint64_t* merged = bars + 22;         // [half][quarter] its maxima and sums are written
  uint64_t* t_full = bars + 30;         // [NP]
  uint64_t* t_empty = t_full + NP;      // [NP] both issuers
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(t_empty + NP);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  // Step j's key tile.  With a bias the last comes first: the keys nearest to a
  // row set its maximum, and the rest never move it (32 heads of 80, causal:
  // 423 us, 475 in ascending order, where a steep head's O is rescaled at
  // every step).  Else ascending: then the CTAs of a head begin with the same
  // keys (32 + 8 + 8 heads of 128: 422 us, 436 descending).
  auto key_tile = [](int j, int j0, int nkv) { return BIAS ? j0 + nkv - 1 - j : j0 + j; };

  const int warp = warp_id();
  const int lane = lane_id();
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&queue.full[i], 1);
      mbar_init(&queue.empty[i], 11);
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 2 + 8);
      mbar_init(&pv_done[i], 1);
      mbar_init(&drain[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
    }
    for (int i = 0; i < 8; ++i) mbar_init(&merged[i], 1);
    mbar_init(o_free, 8);
    mbar_init(queue.answered, 1);
    for (int i = 0; i < NP; ++i) {
      mbar_init(&t_full[i], 1);
      mbar_init(&t_empty[i], 2);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch(&p.map_qkv);
    tma_prefetch(&p.map_o);
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  if (warp == 11) {
    // ------------------------------------------------ items (the whole warp)
    publish_items(queue, blockIdx.x, -1, true, abort_flag, p.err, [&](int block) {
      const Item w = item_of(p.order, block);
      const int bi = w.kv / (p.H / p.G), n = w.kv % (p.H / p.G) * p.G + w.sub;
      const int q0 = (p.order.tiles - 1 - w.tile) * 128;
      // key tiles [j0, j0 + nkv) hold every key that some row sees
      int lo = INT32_MAX, hi = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int2 win = key_window(p.row_begin, p.row_end, p.causal, p.s, bi, q0 + 32 * k + lane);
        if (win.x < win.y) lo = min(lo, win.x);
        hi = max(hi, win.y);
      }
      lo = __reduce_min_sync(0xffffffffu, lo);
      hi = __reduce_max_sync(0xffffffffu, hi);
      const int j0 = lo < hi ? lo / 128 : 0;
      return WorkItem{n, bi, q0, j0, lo < hi ? (hi + 127) / 128 - j0 : 0};
    }, [](int, const WorkItem&) { return true; });
  } else if (warp == 0) {
    // ------------------------------------------------ loads (the whole warp
    // runs the loop, one lane issues).  The next item is asked for three key
    // tiles before the last load.  At the last load is too late for its tiles
    // to be there (documents of 1500, 32 heads of 80: 132 us against 122), at
    // the item's start too early to balance the CTAs (324 items of prefix rows,
    // heads of 96: 38 us against 32)
    constexpr int LEAD = 3;
    int qi = 0, c = 0;  // items with keys, pairs loaded
    bool ok = true;
    // K's row k_row and V's row v_row (negative: none)
    auto load_pair = [&](int k_col, int k_row, int v_col, int v_row, int bi) -> bool {
      const int st = c % NP;
      if (c >= NP && !bounded_wait_w(&t_empty[st], ((c / NP) & 1) ^ 1, abort_flag, 251, p.err)) return false;
      if (lane == 0) {
        uint8_t* to = sKV + 2 * st * T::TILE;
        mbar_expect_tx(&t_full[st], (k_row >= 0 && v_row >= 0 ? 2 : 1) * T::TILE);
        if (k_row >= 0) {
#pragma unroll
          for (int k = 0; k < T::NCH; ++k)
            tma_load_3d(to + k * T::CHUNK, &p.map_qkv, &t_full[st], k_col + k * T::CW, k_row, bi);
        }
        if (v_row >= 0) {
#pragma unroll
          for (int k = 0; k < T::NCH; ++k)
            tma_load_3d(to + T::TILE + k * T::CHUNK, &p.map_qkv, &t_full[st], v_col + k * T::CW, v_row, bi);
        }
      }
      ++c;
      return true;
    };
    for (int it = 0; ok; ++it) {
      WorkItem w;
      if (!next_item<true>(queue, it, &w, abort_flag, p.err)) break;
      const int n = w.n, bi = w.bi, q0 = w.q0, j0 = w.j0, nkv = w.nkv;
      if (n < 0) break;
      if (nkv < LEAD) release_item(queue, it);
      if (nkv == 0) continue;
      const int sl = qi & 1;
      if (qi >= 2 && !bounded_wait_w(&q_empty[sl], ((qi >> 1) & 1) ^ 1, abort_flag, 256, p.err)) break;
      if (lane == 0) {
        mbar_expect_tx(&q_full[sl], T::TILE);
#pragma unroll
        for (int k = 0; k < T::NCH; ++k)
          tma_load_3d(sQ + sl * T::TILE + k * T::CHUNK, &p.map_qkv, &q_full[sl], n * D + k * T::CW, q0, bi);
      }
      ++qi;
      const int k_col = p.k_col + n / p.G * D, v_col = p.v_col + n / p.G * D;
      for (int j = 0; ok && j <= nkv; ++j) {
        ok = load_pair(k_col, j < nkv ? key_tile(j, j0, nkv) * 128 : -1, v_col,
                       j > 0 ? key_tile(j - 1, j0, nkv) * 128 : -1, bi);
        if (j == nkv - LEAD) release_item(queue, it);
      }
    }
    // every copy lands before the shared memory goes, also when a wait elsewhere
    // in the block gives up later
    for (int k = (qi > 2 ? qi - 2 : 0); k < qi; ++k) drain_wait(&q_full[k & 1], (k >> 1) & 1);
    for (int k = (c > NP ? c - NP : 0); k < c; ++k) drain_wait(&t_full[k % NP], (k / NP) & 1);
  } else if (warp == 1 || warp == 10) {
    // ------------------------------------------------ MMA issuers (the
    // whole warp runs the loop, one elected lane issues).  Steps are counted
    // through all items: S_b(t) into buffer t % 2, then PV_b(t-1) of the same
    // item; an item's last PV comes before the next item's first S, which
    // waits for loads that need not have come.  S_b(t) overwrites P_b(t-2)
    // after PV_b(t-2) from the same thread.  The first PV of an item
    // overwrites both O's once the item before has been read.
    const int b = warp == 1 ? 0 : 1;
    const uint32_t uKV = smem_u32(sKV), uQ = smem_u32(sQ);
    const uint32_t tSb = tmem + 128 * b;
    const uint32_t tOb = tmem + C::COL_O + b * D;
    int t = 0, qi = 0;  // steps through all items, items with keys
    RingPos<NP> c;      // pair
    const bool leader = elected();
    auto landed = [&]() { return bounded_wait_w(&t_full[c.at], c.round, abort_flag, 253, p.err); };
    auto pv = [&](int tp, bool first) -> bool {  // PV of step tp, its item's first
      const int sb = tp & 1;
      const uint64_t v = T::mnmajor(uKV + (2 * c.at + 1) * T::TILE, 4 * b);
      if (!bounded_wait_w(&p_full[2 * b + sb], (tp >> 1) & 1, abort_flag, 255, p.err)) return false;
      if (first && qi > 0 && !bounded_wait_w(o_free, (qi - 1) & 1, abort_flag, 258, p.err)) return false;
      tc_fence_after();
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_bf16_tmem_a_1(tOb, tSb + sb * 64 + kk * 8, v + T::mnmajor_step(kk), IDESC_PV, !first || kk > 0);
        umma_commit_1(&pv_done[b]);
        umma_commit_1(&t_empty[c.at]);
      }
      __syncwarp();
      return true;
    };
    bool ok = true;
    for (int it = 0; ok; ++it) {
      WorkItem w;
      if (!next_item(queue, it, &w, abort_flag, p.err)) { ok = false; break; }
      const int nkv = w.nkv;
      if (w.n < 0) break;
      if (nkv == 0) continue;
      if (!bounded_wait_w(&q_full[qi & 1], (qi >> 1) & 1, abort_flag, 259, p.err)) { ok = false; break; }
      const uint64_t q = T::kmajor(uQ + (qi & 1) * T::TILE, 0);
      for (int j = 0; j < nkv; ++j, ++t) {
        if (!landed()) { ok = false; break; }
        tc_fence_after();
        const uint64_t k = T::kmajor(uKV + 2 * c.at * T::TILE + 64 * T::SWB * b, 0);
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            umma_bf16_1(tSb + (t & 1) * 64, q + T::kmajor_step(kk), k + T::kmajor_step(kk), IDESC_S, kk > 0);
          umma_commit_1(&s_full[2 * b + (t & 1)]);
          if (j == nkv - 1) umma_commit_1(&q_empty[qi & 1]);
          if (j == 0) umma_commit_1(&t_empty[c.at]);
        }
        __syncwarp();
        if (j > 0 && !pv(t - 1, j == 1)) { ok = false; break; }
        c = c.next();
      }
      ok = ok && landed() && pv(t - 1, nkv == 1);
      if (!ok) break;
      c = c.next();
      ++qi;
    }
    if (!ok) {
      if (leader) umma_commit_1(&drain[b]);
      drain_wait(&drain[b], 0);
    }
  } else {
    // ------------------------------------------------ softmax (warps 2..9)
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const int b = (warp - 2) >> 2;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t tSb = tmem + 128 * b;
    const uint32_t tOb = tmem + C::COL_O + b * D;
    // the units of m and of the scores when exponentiated: raw scores times
    // log2(e)/sqrt(d) without a modifier, else already log2
    const float ce = (CAP || BIAS) ? 1.f : p.scale_log2;
    int t = 0, items = 0;  // steps, through all items, and items with keys
    auto stored = [&]() {  // the last item's O has left its Q buffer
      if (lane == 0 && items > 0) {
        bulk_wait_read0();
        mbar_arrive(&q_empty[(items - 1) & 1]);
      }
    };
    // an item and its row's window; the next one's are read during the merge
    WorkItem w{-1, 0, 0, 0, 0};
    int2 raw;
    auto take = [&](int it) -> bool {
      if (!next_item(queue, it, &w, abort_flag, p.err)) return false;
      raw = w.n < 0 ? make_int2(0, 0) : raw_window(p.row_begin, p.row_end, p.s, w.bi, w.q0 + r);
      return true;
    };
    bool ok = take(0);
    for (int it = 0; ok; ++it) {
      const int n = w.n, bi = w.bi, qpos = w.q0 + r, j0 = w.j0, nkv = w.nkv;
      if (n < 0) break;
      // (an item without keys leaves it to the next one with some)
      if (nkv > 0) stored();
      const int2 win = clamped_window(raw, p.causal, p.s, qpos);
      const bool valid = qpos < p.s;
      __nv_bfloat16* orow = p.o + (((long long)bi * p.s + qpos) * p.H + n) * D;
      float* lse = p.lse ? p.lse + ((long long)bi * p.H + n) * p.s_pad + qpos : nullptr;
      if (nkv == 0) {
        // no row of the tile sees a key
        if (b == 0) {
          if (valid) {
#pragma unroll
            for (int cc = 0; cc < D / 8; ++cc) reinterpret_cast<uint4*>(orow)[cc] = make_uint4(0u, 0u, 0u, 0u);
          }
          if (lse) *lse = valid ? NEG_INF : 0.f;
        }
        ok = take(it + 1);
        continue;
      }
      const float slope2 = BIAS ? p.slopes[n] * 1.4426950408889634f : 0.f;
      // capped without a bias: 0 until the warp meets a tile beyond 0.6 C, so that
      // the ordinary ones need not look at it
      bool zero = CAP && !BIAS && p.bounded > 0.f;
      float m_run = zero ? 0.f : NEG_INF, l_run = 0.f;
      // a maximum taken from the raw scores and the nearest key's bias is too
      // large by what the bias falls within the 64 columns: 2^-40 at most of P
      const bool gentle = fabsf(slope2) <= 0.6f;
      for (int j = 0; j < nkv; ++j, ++t) {
        const int sb = t & 1;
        const uint32_t tb = tSb + sb * 64 + lane_off;
        // this half's key columns [klo, khi) of the 64 are visible
        const int kv0 = key_tile(j, j0, nkv) * 128 + 64 * b;
        const int klo = max(win.x - kv0, 0), khi = min(win.y - kv0, 64);
        const bool full = klo == 0 && khi == 64;
        float top = NEG_INF;
        if (BIAS) {
          // the nearest visible key's bias is the tile's largest (with a
          // negative slope the farthest one's)
          const int first = kv0 + klo, last = kv0 + khi - 1;
          const int dist = slope2 >= 0.f ? abs(qpos - min(max(qpos, first), last))
                                         : max(abs(qpos - first), abs(qpos - last));
          if (klo < khi) top = -slope2 * (float)dist;
        }
        ok = bounded_wait(&s_full[2 * b + sb], (t >> 1) & 1, abort_flag, 261, p.err);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        tc_fence_after();
        uint32_t pk[32];
        bool rescale = false;
        float alpha = 1.f;
        if (!__any_sync(0xffffffffu, klo < khi)) {
          // nothing of this half is visible to the warp's rows
#pragma unroll
          for (int i = 0; i < 32; ++i) pk[i] = 0u;
        } else {
          uint32_t sv[64];
          const float largest = load_scores<CAP>(tb, sv);  // CAP: in magnitude
          auto z2 = [&](int i) { return f2(__uint_as_float(sv[i]), __uint_as_float(sv[i + 1])); };
          uint64_t rs[2] = {0ull, 0ull};
          // the exponentials of e(i) = the pair (i, i+1) in log2 units
          auto exps = [&](auto e) {
#pragma unroll
            for (int i = 0; i < 64; i += 2) {
              const float2 x = f2split(e(i));
              const float e0 = ex2(x.x), e1 = ex2(x.y);
              rs[(i >> 1) & 1] = add2(rs[(i >> 1) & 1], f2(e0, e1));
              pk[i / 2] = pack_bf16(e0, e1);
            }
          };
          // m: the row's reference, in the units of the scores
          auto refer = [&](float mx) {
            const float m_new = fmaxf(m_run, mx);
            // the maximum is left stale while it moves by less than 2^8 (O
            // and l are scaled alike, so the result does not change)
            rescale = __any_sync(0xffffffffu, (m_new - m_run) * ce > 8.f);
            if (rescale) {
              alpha = (m_run == NEG_INF) ? 0.f : ex2((m_run - m_new) * ce);
              m_run = m_new;
            }
          };
          const bool all = __all_sync(0xffffffffu, full);
          bool near1 = false, bounded = false, done = false;
          if constexpr (CAP) {
            near1 = __all_sync(0xffffffffu, largest <= p.cap.near1);
            // scores so far within the cap that a reference of 0, or the largest
            // bias, serves for their maximum
            bounded = __all_sync(0xffffffffu, largest <= p.bounded);
          }
          BiasLine line{0.f, 0.f, false};
          if (BIAS) line = bias_line(slope2, qpos, kv0, 64, p.causal != 0, false);
          auto refer_bounded = [&]() {
            if (BIAS) refer(top);
            if (!BIAS && !zero) {
              refer(0.f);
              zero = __all_sync(0xffffffffu, m_run == 0.f);
            }
          };
          if (CAP && bounded && all) refer_bounded();
          if (BIAS && !CAP && gentle && all) refer(fmaf(largest, p.scale_log2, top));
          // nothing masked and no maximum to look for: straight to the
          // exponentials, of (score) + (bias - m) on the line
          if (all && (!BIAS || !__any_sync(0xffffffffu, line.mixed))) {
            const uint64_t step2 = both(line.step), base2 = both(line.base - m_run);
            if constexpr (CAP) {
              if (bounded && (BIAS || zero)) {
                done = true;
                if (!BIAS) {
                  if (near1) exps([&](int i) { return cap_near1(p.cap, z2(i)); });
                  else exps([&](int i) { return cap_near2(p.cap, z2(i)); });
                } else if (near1) {
                  exps([&](int i) { return fma2(z2(i), near1_factor(p.cap, z2(i)), on_line(i, step2, base2)); });
                } else {
                  exps([&](int i) { return fma2(z2(i), near2_factor(p.cap, z2(i)), on_line(i, step2, base2)); });
                }
              }
            } else if (!BIAS) {
              done = true;
              refer(largest);
              const uint64_t c2 = both(p.scale_log2), nmc2 = both(-m_run * p.scale_log2);
              exps([&](int i) { return fma2(z2(i), c2, nmc2); });
            } else if (gentle) {
              done = true;
              const uint64_t c2 = both(p.scale_log2);
              exps([&](int i) { return fma2(z2(i), c2, on_line(i, step2, base2)); });
            }
          }
          if (!done) {
            auto put = [&](int i, uint64_t v) {
              const float2 x = f2split(v);
              sv[i] = __float_as_uint(x.x);
              sv[i + 1] = __float_as_uint(x.y);
            };
            bool quick = bounded;  // needs no maximum
            if constexpr (CAP) {
              // masked scores have no say in the form that the others take: what
              // lies in padding changes no bit of the result (8192 rows in documents
              // of 1500, cap 50: 134 us without, 139 so; each element of such a tile in
              // its own form: 134, but 285 against 267 for 16384 rows in documents of
              // 4000, cap 30, whose scores pass C/4 often)
              bool n1 = near1;
              float seen = largest;
              if (!all && !near1) {
                seen = largest_within(sv, klo, khi);
                n1 = __all_sync(0xffffffffu, seen <= p.cap.near1);
                quick = __all_sync(0xffffffffu, seen <= p.bounded);
              }
              if (quick && !all) refer_bounded();
              if (n1) {
#pragma unroll
                for (int i = 0; i < 64; i += 2) put(i, cap_near1(p.cap, z2(i)));
              } else if (__all_sync(0xffffffffu, seen <= p.cap.near2)) {
#pragma unroll
                for (int i = 0; i < 64; i += 2) put(i, cap_near2(p.cap, z2(i)));
              } else if (!p.cap.large) {
#pragma unroll
                for (int i = 0; i < 64; i += 2) put(i, cap_far(p.cap, z2(i)));
              } else {
#pragma unroll
                for (int i = 0; i < 64; i += 2) put(i, cap_far_large(p.cap, z2(i)));
              }
            }
            if (BIAS) {
              const uint64_t cs2 = both(CAP ? 1.f : p.scale_log2);
              if (!__any_sync(0xffffffffu, line.mixed)) {
                const uint64_t step2 = both(line.step), base2 = both(line.base);
#pragma unroll
                for (int i = 0; i < 64; i += 2) put(i, fma2(z2(i), cs2, on_line(i, step2, base2)));
              } else {
                const float dist = (float)(qpos - kv0);
#pragma unroll
                for (int i = 0; i < 64; i += 2)
                  put(i, fma2(z2(i), cs2,
                              f2(-slope2 * fabsf(dist - (float)i), -slope2 * fabsf(dist - (float)(i + 1)))));
              }
            }
            // masked scores to -inf; a window cuts a half on one side mostly
            if (__any_sync(0xffffffffu, khi < 64)) {
#pragma unroll
              for (int i = 0; i < 64; ++i)
                if (i >= khi) sv[i] = 0xFF800000u;
            }
            if (__any_sync(0xffffffffu, klo > 0)) {
#pragma unroll
              for (int i = 0; i < 64; ++i)
                if (i < klo) sv[i] = 0xFF800000u;
            }
            if (!quick && !(BIAS && !CAP && gentle && all)) {
              float m4[4] = {NEG_INF, NEG_INF, NEG_INF, NEG_INF};
#pragma unroll
              for (int i = 0; i < 64; i += 2)
                m4[(i >> 1) & 3] = max3f(m4[(i >> 1) & 3], __uint_as_float(sv[i]), __uint_as_float(sv[i + 1]));
              if (CAP && !BIAS && l_run == 0.f) m_run = NEG_INF;  // nothing seen yet
              refer(fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])));
              zero = false;
            }
            // a row that has seen no key keeps m = -inf: offset 0, P = 2^-inf
            const float mc = (m_run == NEG_INF) ? 0.f : m_run * ce;
            const uint64_t c2 = both(ce), nmc2 = both(-mc);
            exps([&](int i) { return fma2(z2(i), c2, nmc2); });
          }
          const float2 rsum = f2split(add2(rs[0], rs[1]));
          l_run = fmaf(l_run, alpha, rsum.x + rsum.y);
        }
        // P over the first 32 columns of its own S buffer (all read above)
        tmem_st32(tb, pk);
        // PV(t-1) must be done before O is rescaled.  Having seen S(t), which
        // was issued after PV(t-2), these warps know pv_done is in phase t-1
        // or t, so a wait on the parity of t - 1 is exact however many phases
        // went by unwaited; an item's last step always waits, so the wait
        // after the loop is exact too.
        if (j > 0 && (rescale || j == nkv - 1)) {
          ok = bounded_wait(&pv_done[b], (t - 1) & 1, abort_flag, 262, p.err);
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
      if (ok) ok = take(it + 1);
      if (ok) ok = __all_sync(0xffffffffu, bounded_wait(&pv_done[b], (t - 1) & 1, abort_flag, 263, p.err));
      if (!ok) break;
      // merge: each half leaves its maxima and row sums for the other
      red_m[b * 128 + r] = m_run;
      red_l[b * 128 + r] = l_run;
      __syncwarp();
      if (lane == 0) mbar_arrive(&merged[4 * b + quarter]);
      ok = bounded_wait(&merged[4 * (b ^ 1) + quarter], items & 1, abort_flag, 265, p.err) &&
           bounded_wait(&pv_done[b ^ 1], (t - 1) & 1, abort_flag, 264, p.err);
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      tc_fence_after();
      const float m_o = red_m[(b ^ 1) * 128 + r], l_o = red_l[(b ^ 1) * 128 + r];
      const float m = fmaxf(m_run, m_o);
      const float a_self = (m_run == NEG_INF) ? 0.f : ex2((m_run - m) * ce);
      const float a_o = (m_o == NEG_INF) ? 0.f : ex2((m_o - m) * ce);
      const float l = l_run * a_self + l_o * a_o;
      const float inv_l = l == 0.f ? 0.f : 1.f / l;  // nothing visible: O = 0
      const float w_self = a_self * inv_l, w_o = a_o * inv_l;
      const uint32_t tOo = tmem + C::COL_O + (b ^ 1) * D;
      // Each half's warp merges its columns of its 32 rows and stores them by
      // TMA (whole lines, and rows past the sequence are left out), staged in
      // the item's Q tile, which every S product has read: O has Q's tile
      // layout.  Direct stores of 32 bytes per row cost 3,000 cycles an item.
      // Half a tile per half where it has an even number of chunks' columns,
      // else the first half takes the odd one.
      constexpr int NC = D / 16, CC = T::CW / 16;  // 16-column groups, per chunk
      constexpr int NC0 = (T::NCH + 1) / 2 * CC;
      const int cbeg = b == 0 ? 0 : NC0, ncc = b == 0 ? NC0 : NC - NC0;
      uint8_t* stage = sQ + (items & 1) * T::TILE;
#pragma unroll
      for (int cc = 0; cc < NC0; cc += 2) {
        uint32_t vs[32], vo[32];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (cc + h < ncc) {
            tmem_ld16_nw(tOb + lane_off + (cbeg + cc + h) * 16, vs + 16 * h);
            tmem_ld16_nw(tOo + lane_off + (cbeg + cc + h) * 16, vo + 16 * h);
          }
        tmem_wait_ld(vs);
        tmem_wait_ld(vo);
        if (cc + 2 >= NC0) {
          // this warp's reads of both O's and of the other half's maxima are
          // done: nothing overwrites either before all eight warps say so
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(o_free);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (cc + h < ncc) {
            const int col = cbeg + cc + h;  // group of 16 columns
#pragma unroll
            for (int k = 16 * h; k < 16 * h + 16; ++k)
              vs[k] = __float_as_uint(__uint_as_float(vs[k]) * w_self + __uint_as_float(vo[k]) * w_o);
            store_tile16<D>(stage, r, col, vs + 16 * h, 1.f);
          }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        for (int ch = cbeg / CC; valid && ch < (cbeg + ncc) / CC; ++ch)  // not a box past the end
          tma_store_3d(&p.map_o, stage + ch * T::CHUNK + quarter * 32 * T::SWB, n * D + ch * T::CW, qpos, bi);
        bulk_commit();
      }
      ++items;
      if (b == 0 && lse) *lse = !valid ? 0.f : l == 0.f ? NEG_INF : fmaf(m * ce, LN2, logf(l));
    }
    if (lane == 0) bulk_wait0();  // before the shared memory goes
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool CAP, bool BIAS>
int launch_mod_fwd(const ModFwdParams& prm, int grid, cudaStream_t st) {
  constexpr int SMEM = ModFwdCfg<D>::SMEM;
  static_assert(SMEM <= 232448, "attention forward tile set exceeds shared memory");
  static std::atomic<uint64_t> attr{0};  // devices whose limit is set
  if (smem_limit_once(reinterpret_cast<const void*>(attn_mod_fwd_kernel<D, CAP, BIAS>), SMEM, &attr)) return BPT_ECUDA;
  attn_mod_fwd_kernel<D, CAP, BIAS><<<grid, 384, SMEM, st>>>(prm);
  return cudaGetLastError() == cudaSuccess ? BPT_OK : BPT_ECUDA;
}

template <int D>
int launch_for(const ModFwdParams& p, bool cap, int grid, cudaStream_t st) {
  if (p.slopes) return cap ? launch_mod_fwd<D, true, true>(p, grid, st) : launch_mod_fwd<D, false, true>(p, grid, st);
  return cap ? launch_mod_fwd<D, true, false>(p, grid, st) : launch_mod_fwd<D, false, false>(p, grid, st);
}

}  // namespace

int attention_mod_fwd(const PackedDims& D, int causal, const bpt_score_mod& mod, const void* qkv, void* o, float* lse,
                      cudaStream_t st) {
  ModFwdParams p;
  memset(&p, 0, sizeof(p));
  if (make_attn_map(&p.map_qkv, qkv, (int)D.b, (int)D.s, D.width, (int)D.d, 128) ||
      make_attn_map(&p.map_o, o, (int)D.b, (int)D.s, D.H * D.d, (int)D.d, 32))
    return BPT_EINVAL;
  p.s = (int)D.s;
  p.s_pad = (int)D.s_pad;
  p.H = (int)D.H;
  p.G = (int)D.G;
  p.causal = causal;
  p.k_col = (int)(D.H * D.d);
  p.v_col = (int)((D.H + D.Hkv) * D.d);
  p.order = item_order(D.s_pad / 128, D.G, D.b * D.Hkv, 4 * D.s * D.d);
  p.o = reinterpret_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.row_begin = mod.row_begin;
  p.row_end = mod.row_end;
  p.slopes = mod.slopes;
  p.scale_log2 = (float)(1.4426950408889634 / sqrt((double)D.d));
  const bool cap = mod.softcap > 0.f;
  if (cap) {
    const double out = mod.softcap * 1.4426950408889634;
    p.cap = cap_coef(mod.softcap, 1.0 / (mod.softcap * sqrt((double)D.d)), out);
    p.bounded = out <= 88.0 ? p.cap.near2 : -1.f;
  }
  p.err = device_error_word();
  if (!p.err) return BPT_ECUDA;
  const int grid = (int)(D.s_pad / 128 * D.H * D.b);
  // credited as without windows, which live on the device
  const double pairs = causal ? (double)D.s * (D.s + 1) / 2 : (double)D.s * D.s;
  ProfScope prof(PROF_ATTN_FWD, 4.0 * D.d * pairs * D.H * D.b, 0.0, st);
  switch (D.d) {
    case 64: return launch_for<64>(p, cap, grid, st);
    case 80: return launch_for<80>(p, cap, grid, st);
    case 96: return launch_for<96>(p, cap, grid, st);
    case 112: return launch_for<112>(p, cap, grid, st);
    case 128: return launch_for<128>(p, cap, grid, st);
    default: return BPT_EUNSUPPORTED;
  }
}

}  // namespace bpt
