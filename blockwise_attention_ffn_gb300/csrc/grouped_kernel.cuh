// grouped_kernel.cuh -- matrix products over ragged groups of rows, each
// group against its own matrix: the experts' products of a mixture-of-experts
// feed-forward network and their gradients.
//
//   NT  out[r, :] = A[r, :] W_e^T      W [G, N, K]: the forward
//   NN  out[r, :] = A[r, :] W_e        W [G, K, N]: the gradient of the rows
//   TN  out_e     = A_e^T B_e          the gradient of the matrices
//
// for the rows r in [offsets[e], offsets[e + 1]).  The offsets live on the
// device: every CTA reads them once and lays out the same list of work units
// (tiles of each group, in the groups' order) in its shared memory, so
// nothing has to come back to the host and no tile holds rows of two groups.
//
// Warp roles, ring and accumulators are those of gemm_kernel.cuh (a producer
// warp, an issuing warp, eight epilogue warps; two accumulators; one SM or a
// pair of SMs per tile).  What is different:
//   - Rows are gathered on the way in: the 32 lanes of the producer warp hold
//     the four row indices of a quad each and issue one 4-row TMA gather a
//     stage, so the 128 rows of a CTA's A tile come from where the router left
//     them and no copy in the groups' order is ever made.  Quads behind the
//     group's last row are not loaded: what their shared memory holds reaches
//     only accumulator rows that are never stored.
//   - TN runs over a group's rows as K.  The last, partial block of 64 rows
//     is loaded by gathers too, with an index outside the tensor (a row of
//     zeros) behind the group's end: what lies there, a NaN even, stays out.
//   - Weights are 3-D maps [G, rows, cols]: a tile that runs over a matrix's
//     edge reads zeros, not the next group's matrix.
#pragma once

#include "gemm_kernel.cuh"
#include "grouped.h"

namespace bpt {
namespace gg {

using gk::A_BYTES;
using gk::BK;
using gk::BM;
using gk::NUM_EPI_WARPS;
using gk::NUM_THREADS;

struct Params {
  CUtensorMap map_a[2];   // A tiles (TN: {64, 64} boxes)
  CUtensorMap map_ag[2];  // A gathers (one-row boxes)
  CUtensorMap map_b[2];   // weights, or TN: B tiles
  CUtensorMap map_bg;     // TN: B gathers
  const int* offsets;
  int groups, rows;
  int M, N, nkt, segs;    // TN: M; NT, NN: k-tiles of one segment and the number of segments (TN: segments of M)
  int mt, nt;             // TN: tile rows per segment; tile columns
  int band;               // tile rows walked before the next tile column (m fastest)
  int a_rows, b_rows;     // rows of the gathered tensors (the index of a row of zeros)
  const int* order;       // pair at each sorted row, or NULL: row r is row r
  int top_k, pairs;
  void *out, *out2, *out3;
  int out_f32;
  float beta;
  int act;
  const __nv_bfloat16 *aux, *aux2;
  const void* row_weight;
  int row_weight_f32;
  float* part;
  int vec32;
  unsigned int* err;
};

// Units before each group (s_unit[0 .. G]) and the groups' first row and row
// count, by one warp.  A group whose offsets fall, leave [0, rows] or start
// before the end of an earlier group is empty and recorded: nothing outside
// the tensors is ever touched and no row is written twice.
template <bool TN, int TM>
__device__ __forceinline__ void lay_out(const Params& p, int* s_unit, int* s_lo, int* s_cnt) {
  const int lane = lane_id();
  int base = 0, end = 0;  // units and the largest end of the groups before
  for (int e0 = 0; e0 < p.groups; e0 += 32) {
    const int e = e0 + lane;
    const bool in = e < p.groups;
    int lo = in ? p.offsets[e] : 0;
    const int hi = in ? p.offsets[e + 1] : 0;
    const bool inside = lo >= 0 && lo <= hi && hi <= p.rows;
    int top = inside ? hi : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, top, d);
      if (lane >= d) top = max(top, v);
    }
    int before = __shfl_up_sync(0xffffffffu, top, 1);
    before = max(end, lane ? before : 0);
    end = max(end, __shfl_sync(0xffffffffu, top, 31));
    const bool ok = inside && lo >= before;
    if (in && !ok && blockIdx.x == 0) report_bad_data(p.err, BPT_GROUPED_BAD_OFFSET_SITE);
    const int cnt = ok ? hi - lo : 0;
    lo = ok ? lo : 0;
    if (in) {
      s_lo[e] = lo;
      s_cnt[e] = cnt;
    }
    int u = !in ? 0 : TN ? p.segs * p.mt * p.nt : (cnt + TM - 1) / TM * p.nt;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, u, d);
      if (lane >= d) u += v;
    }
    if (in) s_unit[e + 1] = base + u;
    base += __shfl_sync(0xffffffffu, u, 31);
  }
  if (lane == 0) s_unit[0] = 0;
}

// A work unit's place: group, first row of the tile in the group (TN: of the
// matrix), first column, segment of M (TN).
struct Place {
  int e, lo, cnt, m0, n0, seg;
};
template <bool TN, int TM, int BN>
__device__ __forceinline__ void place(const Params& p, int unit, const int* s_unit, const int* s_lo, const int* s_cnt, Place& at) {
  int e = at.e;  // units come in rising order
  while (unit >= s_unit[e + 1]) ++e;
  at.e = e;
  at.lo = s_lo[e];
  at.cnt = s_cnt[e];
  const int local = unit - s_unit[e];
  const int mt = TN ? p.segs * p.mt : (at.cnt + TM - 1) / TM;
  const int per = p.band * p.nt;
  const int g = local / per, r = local - g * per;
  const int gs = min(p.band, mt - g * p.band);
  const int nb = r / gs;
  int mb = g * p.band + (r - nb * gs);
  at.seg = TN && mb >= p.mt ? 1 : 0;
  if (TN) mb -= at.seg * p.mt;
  at.m0 = mb * TM;
  at.n0 = nb * BN;
}

// four rows of 64 columns, by index
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int4 r) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w)
      : "memory");
}
__device__ __forceinline__ void tma_gather4_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int4 r) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// sigmoid with an error of a few units of fp32's last place: what it enters
// is rounded to bf16
__device__ __forceinline__ float fast_sigmoid(float z) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.4426950408889634f * z));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
}

// W consecutive columns n .. of output row `row` (in the groups' order; TN:
// of all the groups' matrices), the accumulators a (and b: the up product)
template <int EPI, bool DUAL, int W>
__device__ __forceinline__ void epi_cols(const Params& p, void* out, long long row, int n, const float (&a)[W], const float (&b)[W],
                                         float w, float& dot) {
  const long long i = row * p.N + n;
  if constexpr (EPI == GROUPED_STORE) {
    if (p.out_f32) {
      float* o = reinterpret_cast<float*>(out) + i;
      float v[W];
      if (p.beta != 0.f) {
        gk::loadw_f32<W>(o, v);
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] = fmaf(p.beta, v[j], a[j]);
        gk::storew_f32<W>(o, v);
      } else {
        gk::storew_f32<W>(o, a);
      }
    } else {
      gk::storew_bf16<W>(reinterpret_cast<__nv_bfloat16*>(out) + i, a);
    }
  } else if constexpr (EPI == GROUPED_ACT) {
    float v[W];
    if constexpr (DUAL) {
#pragma unroll
      for (int j = 0; j < W; ++j) v[j] = a[j] * fast_sigmoid(a[j]) * b[j];
      if (p.out2) {
        gk::storew_bf16<W>(reinterpret_cast<__nv_bfloat16*>(p.out2) + i, a);
        gk::storew_bf16<W>(reinterpret_cast<__nv_bfloat16*>(p.out3) + i, b);
      }
    } else if (p.out2) {
      float d[W];
#pragma unroll
      for (int j = 0; j < W; ++j) gk::gelu_and_grad_f(a[j], p.act, v[j], d[j]);
      gk::storew_bf16<W>(reinterpret_cast<__nv_bfloat16*>(p.out2) + i, d);
    } else {
#pragma unroll
      for (int j = 0; j < W; ++j) v[j] = gk::gelu_f(a[j], p.act);
    }
    gk::storew_bf16<W>(reinterpret_cast<__nv_bfloat16*>(out) + i, v);
  } else {
    // The saved pair is bf16 (2^-9 of its size each): the activation and its
    // slopes are taken again from it in fp32 and rounded once.
    float s0[W], s1[W], v[W], aw[W];
    gk::loadw_bf16<W>(p.aux + i, s0);
    gk::loadw_bf16<W>(p.aux2 + i, s1);
    if (p.act == BPT_ACT_SWIGLU) {
      float dv[W];
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const float sg = fast_sigmoid(s0[j]);
        const float si = s0[j] * sg;  // silu(g)
        const float act = si * s1[j];
        const float wa = w * a[j];
        dot = fmaf(a[j], act, dot);
        aw[j] = w * act;
        v[j] = wa * s1[j] * (sg + si * (1.f - sg));
        dv[j] = wa * si;
      }
      gk::storew_bf16<W>(reinterpret_cast<__nv_bfloat16*>(p.out2) + i, dv);
    } else {
#pragma unroll
      for (int j = 0; j < W; ++j) {
        dot = fmaf(a[j], s0[j], dot);
        aw[j] = w * s0[j];
        v[j] = w * a[j] * s1[j];
      }
    }
    gk::storew_bf16<W>(reinterpret_cast<__nv_bfloat16*>(out) + i, v);
    gk::storew_bf16<W>(reinterpret_cast<__nv_bfloat16*>(p.out3) + i, aw);
  }
}

// ring stages that fit beside the group lists
template <int STAGE_BYTES>
constexpr int ring_stages() {
  return 200 * 1024 / STAGE_BYTES > 8 ? 8 : 200 * 1024 / STAGE_BYTES;
}
template <int BN, bool DUAL, bool PAIR>
constexpr int stage_bytes() {
  return A_BYTES + (DUAL ? 2 : 1) * (PAIR ? BN / 2 : BN) * BK * 2;
}
template <int BN, bool DUAL, bool PAIR>
constexpr int smem_bytes() {
  return ring_stages<stage_bytes<BN, DUAL, PAIR>()>() * stage_bytes<BN, DUAL, PAIR>() + 1024 + 256 +
         (3 * GROUPED_MAX_GROUPS + 4) * 4;
}

// BN: tile width.  AG, BG: rows of A (TN: of A, of B) gathered.  DUAL: two
// weight tiles against one A tile (gate and up).  PAIR: a 256-row tile per
// cluster of two CTAs.
template <int FORM, int EPI, int BN, bool AG, bool BG, bool DUAL, bool PAIR>
__global__ void __launch_bounds__(NUM_THREADS, 1) grouped_kernel(const __grid_constant__ Params p) {
  constexpr bool TN = FORM == GROUPED_TN;
  constexpr bool B_MN = FORM != GROUPED_NT;
  constexpr int BNS = PAIR ? BN / 2 : BN;  // rows (columns) of each B this CTA stages
  constexpr int STAGE_BYTES = stage_bytes<BN, DUAL, PAIR>();
  constexpr int STAGES = ring_stages<STAGE_BYTES>();
  constexpr int ACC_COLS = (DUAL ? 2 : 1) * BN;
  constexpr uint32_t TMEM_COLS = 2 * ACC_COLS;
  static_assert(TMEM_COLS <= 512 && TMEM_COLS >= 32 && (TMEM_COLS & (TMEM_COLS - 1)) == 0, "two accumulators");
  static_assert(BN % 64 == 0 && (!DUAL || FORM == GROUPED_NT), "tile width");
  constexpr int TM = PAIR ? 2 * BM : BM;
  constexpr uint32_t IDESC = idesc_bf16(TM, BN, TN, B_MN);

  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * STAGE_BYTES);
  uint64_t* empty = full + STAGES;
  uint64_t* acc_full = empty + STAGES;  // [2]
  uint64_t* acc_empty = acc_full + 2;   // [2]
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* s_unit = reinterpret_cast<int*>(smem + STAGES * STAGE_BYTES + 256);  // [groups + 1]
  int* s_lo = s_unit + GROUPED_MAX_GROUPS + 4;
  int* s_cnt = s_lo + GROUPED_MAX_GROUPS;
  static_assert((2 * STAGES + 5) * 8 + 8 <= 256, "barriers");

  const int warp = warp_id();
  const int lane = lane_id();
  const uint32_t rank = PAIR ? cluster_rank() : 0u;
  const int unit0 = PAIR ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
  const int units_in_flight = PAIR ? (int)(gridDim.x >> 1) : (int)gridDim.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], (PAIR ? 2 : 1) * NUM_EPI_WARPS);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(tmem_holder, TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_holder, TMEM_COLS);
      tmem_relinquish();
    }
  }
  // everything above touches this CTA's own memory alone
  wait_for_previous();
  let_next_start();
  if (warp == 0) lay_out<TN, TM>(p, s_unit, s_lo, s_cnt);
  tc_fence_before();
  if constexpr (PAIR) cluster_sync_all();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const int nunits = s_unit[p.groups];
  // k-tiles of a unit
  auto k_tiles = [&](const Place& at) { return TN ? (at.cnt + BK - 1) / BK : p.segs * p.nkt; };

  if (warp == 0) {
    // -------------------------------------------------- producer (the warp)
    const uint32_t full0 = PAIR ? cluster_addr(smem_u32(full), 0) : smem_u32(full);
    const uint32_t smem_base = smem_u32(smem);
    uint32_t it = 0;
    bool ok = true;
    Place at;
    at.e = 0;
    auto gather = [&](uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int4 r) {
      if constexpr (PAIR) tma_gather4_pair(dst, map, bar, x, r);
      else tma_gather4(dst, map, bar, x, r);
    };
    auto load2 = [&](uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
      if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
            : "memory");
      else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
            : "memory");
    };
    auto load3 = [&](uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
      if constexpr (PAIR) tma_load_3d_pair(dst, map, bar, x, y, z);
      else tma_load_3d(dst, map, bar, x, y, z);
    };
    // row of the rows operand at sorted row r (in range), by the router's order
    auto row_of = [&](int r) {
      const int q = p.order[r];
      return q < 0 || q >= p.pairs ? p.a_rows + p.b_rows : q / p.top_k;
    };
    auto claim = [&](int s) {  // the stage is free, by one verdict of the warp
      return it < (uint32_t)STAGES || bounded_wait_w(&empty[s], ((it / STAGES) & 1) ^ 1, abort_flag, 101, p.err);
    };
    for (int unit = unit0; ok && unit < nunits; unit += units_in_flight) {
      place<TN, TM, BN>(p, unit, s_unit, s_lo, s_cnt, at);
      const int nbs = at.n0 + (int)rank * BNS;
      if constexpr (!TN) {
        const int mine = at.m0 + (int)rank * BM;  // this CTA's first row in the group
        int4 q = make_int4(0, 0, 0, 0);           // this lane's quad
        bool live = false;
        uint32_t bytes = STAGE_BYTES * (PAIR ? 2 : 1);
        if constexpr (AG) {
          const int r0 = mine + 4 * lane;
          live = r0 < at.cnt;
          auto one = [&](int r) { return r >= at.cnt ? p.a_rows : p.order ? row_of(at.lo + r) : at.lo + r; };
          if (live) q = make_int4(one(r0), one(r0 + 1), one(r0 + 2), one(r0 + 3));
          // bytes of both CTAs' live quads and weights
          bytes = (PAIR ? 2 : 1) * (STAGE_BYTES - A_BYTES);
          const int left = at.cnt - at.m0;
          bytes += (uint32_t)((min(left, TM) + 3) / 4) * 512u;
        }
        const int nk = p.segs * p.nkt;
        for (int kt = 0; kt < nk; ++kt) {
          const int s = it % STAGES;
          if (!claim(s)) {
            ok = false;
            break;
          }
          const uint32_t sa = smem_base + s * STAGE_BYTES;
          const uint32_t sb = sa + A_BYTES;
          const uint32_t fb = full0 + 8u * (uint32_t)s;
          const int seg = FORM == GROUPED_NN && kt >= p.nkt ? 1 : 0;
          const int kx = (kt - seg * p.nkt) * BK;
          if (lane == 0) {
            if (rank == 0) mbar_expect_tx(&full[s], bytes);
            if constexpr (!AG) load2(sa, &p.map_a[seg], fb, kx, at.lo + mine);
            if constexpr (FORM == GROUPED_NT) {
              load3(sb, &p.map_b[0], fb, kx, nbs, at.e);
              if constexpr (DUAL) load3(sb + BNS * BK * 2, &p.map_b[1], fb, kx, nbs, at.e);
            } else {
#pragma unroll
              for (int c = 0; c < BNS / 64; ++c) load3(sb + c * 8192, &p.map_b[seg], fb, nbs + c * 64, kx, at.e);
            }
          }
          __syncwarp();
          if constexpr (AG) {
            if (live) gather(sa + lane * 512, &p.map_ag[seg], fb, kx, q);
          }
          ++it;
        }
      } else {
        const int ma = at.m0 + (int)rank * BM;
        const int nk = (at.cnt + BK - 1) / BK;
        const int quad = lane & 15, c0 = lane >> 4;
        // rows of this lane's quad in block kt: by the router's order
        // (gathered operands), or as they lie (the last, partial block)
        auto rows_of = [&](int kt) {
          const int r0 = kt * BK + 4 * quad;
          auto one = [&](int r) { return r < at.cnt ? row_of(at.lo + r) : p.a_rows + p.b_rows; };
          return make_int4(one(r0), one(r0 + 1), one(r0 + 2), one(r0 + 3));
        };
        constexpr int AHEAD = 4;  // blocks whose indices are on their way
        int4 ring[AHEAD];
        if constexpr (AG || BG) {
#pragma unroll
          for (int u = 0; u < AHEAD; ++u) ring[u] = rows_of(u);
        }
        for (int k4 = 0; ok && k4 < nk; k4 += AHEAD) {
#pragma unroll
          for (int u = 0; u < AHEAD; ++u) {
            const int kt = k4 + u;
            if (kt >= nk) break;
            const int s = it % STAGES;
            if (!claim(s)) {
              ok = false;
              break;
            }
            int4 by_order = make_int4(0, 0, 0, 0);
            if constexpr (AG || BG) {
              by_order = ring[u];
              ring[u] = rows_of(kt + AHEAD);
            }
            const uint32_t sa = smem_base + s * STAGE_BYTES;
            const uint32_t sb = sa + A_BYTES;
            const uint32_t fb = full0 + 8u * (uint32_t)s;
            const bool whole = (kt + 1) * BK <= at.cnt;
            const int y = at.lo + kt * BK;
            int4 as_is = make_int4(0, 0, 0, 0);
            if (!whole) {
              const int r0 = kt * BK + 4 * quad;
              auto one = [&](int r) { return r < at.cnt ? at.lo + r : p.a_rows + p.b_rows; };
              as_is = make_int4(one(r0), one(r0 + 1), one(r0 + 2), one(r0 + 3));
            }
            if (lane == 0) {
              if (rank == 0) mbar_expect_tx(&full[s], (PAIR ? 2 : 1) * STAGE_BYTES);
              if (!AG && whole) {
                load2(sa, &p.map_a[at.seg], fb, ma, y);
                load2(sa + 8192, &p.map_a[at.seg], fb, ma + 64, y);
              }
              if (!BG && whole) {
#pragma unroll
                for (int c = 0; c < BNS / 64; ++c) load2(sb + c * 8192, &p.map_b[0], fb, nbs + c * 64, y);
              }
            }
            __syncwarp();
            if (AG || !whole) gather(sa + c0 * 8192 + quad * 512, &p.map_ag[at.seg], fb, ma + c0 * 64, AG ? by_order : as_is);
            if (BG || !whole) {
#pragma unroll
              for (int c = 0; c < BNS / 64; c += 2)
                if (c + c0 < BNS / 64)
                  gather(sb + (c + c0) * 8192 + quad * 512, &p.map_bg, fb, nbs + (c + c0) * 64, BG ? by_order : as_is);
            }
            ++it;
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0 && *abort_flag) {
      // let every load issued land before the CTA goes away; a pair's ranks
      // cannot wait for one another's stragglers and give them a fixed time
      if (rank == 0)
        for (uint32_t j = (it > (uint32_t)STAGES ? it - STAGES : 0); j < it; ++j) drain_wait(&full[j % STAGES], (j / STAGES) & 1);
      if (PAIR) {
        const long long t0 = clock64();
        while (clock64() - t0 < 1000000) {
        }
      }
    }
  } else if (warp == 1) {
    // -------------------------------------------------- MMA issuer
    if (rank == 0) {
      const uint32_t smem_base = smem_u32(smem);
      uint32_t it = 0;
      int tc = 0;
      bool ok = true;
      Place at;
      at.e = 0;
      for (int unit = unit0; ok && unit < nunits; unit += units_in_flight) {
        place<TN, TM, BN>(p, unit, s_unit, s_lo, s_cnt, at);
        const int nk = k_tiles(at);
        if (nk == 0) continue;  // an empty group's matrix: the epilogue writes zeros
        const int acc = tc & 1;
        if (tc >= 2) {
          const uint32_t par = ((tc >> 1) - 1) & 1;
          const bool w = PAIR ? bounded_wait_cluster_w(&acc_empty[acc], par, abort_flag, 106, p.err)
                              : bounded_wait_w(&acc_empty[acc], par, abort_flag, 106, p.err);
          if (!w) {
            ok = false;
            break;
          }
        }
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(acc * ACC_COLS);
        for (int kt = 0; kt < nk; ++kt) {
          const int s = it % STAGES;
          if (!bounded_wait_w(&full[s], (it / STAGES) & 1, abort_flag, 103, p.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_base + s * STAGE_BYTES;
          const uint32_t sb = sa + A_BYTES;
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk) {
            const uint64_t ad = TN ? sdesc(sa + kk * 2048, 8192, 1024, 2) : sdesc(sa + kk * 32, 16, 1024, 2);
            const uint64_t bd = B_MN ? sdesc(sb + kk * 2048, 8192, 1024, 2) : sdesc(sb + kk * 32, 16, 1024, 2);
            const bool accum = kt != 0 || kk != 0;
            if constexpr (PAIR) umma_bf16_pair_w(d, ad, bd, IDESC, accum);
            else umma_bf16_w(d, ad, bd, IDESC, accum);
            if (DUAL) {
              const uint64_t bd2 = sdesc(sb + BNS * BK * 2 + kk * 32, 16, 1024, 2);
              if constexpr (PAIR) umma_bf16_pair_w(d + BN, ad, bd2, IDESC, accum);
              else umma_bf16_w(d + BN, ad, bd2, IDESC, accum);
            }
          }
          if constexpr (PAIR) umma_commit_pair_w(&empty[s], 3);
          else umma_commit_w(&empty[s]);
          ++it;
        }
        if (!ok) break;
        if constexpr (PAIR) umma_commit_pair_w(&acc_full[acc], 3);
        else umma_commit_w(&acc_full[acc]);
        ++tc;
      }
      if (!ok) {
        if constexpr (PAIR) umma_commit_pair_w(drain, 1);
        else umma_commit_w(drain);
        drain_wait(drain, 0);
      }
    }
  } else {
    // -------------------------------------------------- epilogue (warps 2..9)
    constexpr int EPI_COLS = BN / 2;
    constexpr int CH = EPI_COLS < 32 ? EPI_COLS : 32;
    static_assert(CH == 32, "32 columns a chunk");
    const int q = warp & 3;
    const int half = (warp - 2) >> 2;
    const uint32_t acc_empty0 = PAIR ? cluster_addr(smem_u32(acc_empty), 0) : 0u;
    int tc = 0;
    Place at;
    at.e = 0;
    for (int unit = unit0; unit < nunits; unit += units_in_flight) {
      place<TN, TM, BN>(p, unit, s_unit, s_lo, s_cnt, at);
      const bool none = k_tiles(at) == 0;
      const int acc = tc & 1;
      if (!none) {
        // the TMEM loads below are warp-collective, so the decision is too
        const bool ok = __all_sync(0xffffffffu, bounded_wait(&acc_full[acc], (tc >> 1) & 1, abort_flag, 105, p.err));
        if (!ok) break;
        tc_fence_after();
      } else if (p.beta != 0.f) {
        continue;  // nothing to add
      }
      const int m = at.m0 + (int)rank * BM + q * 32 + lane;
      const bool mine = m < (TN ? p.M : at.cnt);
      const long long row = TN ? (long long)at.e * p.M + m : (long long)at.lo + m;
      void* out = TN && at.seg ? p.out2 : p.out;
      float w = 0.f, dot = 0.f;
      if constexpr (EPI == GROUPED_ACT_BWD) {
        if (mine) {
          const int pair = p.order[row];
          if (pair >= 0 && pair < p.pairs)
            w = p.row_weight_f32 ? reinterpret_cast<const float*>(p.row_weight)[pair]
                                 : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.row_weight)[pair]);
        }
      }
      const uint32_t tbase = tmem + (uint32_t)(acc * ACC_COLS) + ((uint32_t)(q * 32) << 16);
#pragma unroll 1
      for (int c = 0; c < EPI_COLS / 32; ++c) {
        const int col = half * EPI_COLS + c * 32;
        const int nb = at.n0 + col;
        if (nb >= p.N) break;  // warp-uniform
        uint32_t ra[32], rb[32];
        if (!none) {
          tmem_ld32(tbase + col, ra);
          if (DUAL) tmem_ld32(tbase + BN + col, rb);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) ra[j] = rb[j] = 0u;
        }
        if (mine) {
          if (nb + 32 <= p.N && p.vec32) {
            float a32[32], b32[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              a32[j] = __uint_as_float(ra[j]);
              b32[j] = DUAL ? __uint_as_float(rb[j]) : 0.f;
            }
            epi_cols<EPI, DUAL, 32>(p, out, row, nb, a32, b32, w, dot);
          } else {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              if (nb + g * 8 < p.N) {  // N is a multiple of 8
                float a8[8], b8[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  a8[j] = __uint_as_float(ra[g * 8 + j]);
                  b8[j] = DUAL ? __uint_as_float(rb[g * 8 + j]) : 0.f;
                }
                epi_cols<EPI, DUAL, 8>(p, out, row, nb + g * 8, a8, b8, w, dot);
              }
            }
          }
        }
        __syncwarp();
      }
      if constexpr (EPI == GROUPED_ACT_BWD) {
        // one sum per row and half tile, added in this order later
        if (mine) p.part[(long long)(2 * (at.n0 / BN) + half) * p.rows + row] = dot;
      }
      if (!none) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (PAIR) mbar_arrive_cluster(acc_empty0 + 8u * (uint32_t)acc);
          else mbar_arrive(&acc_empty[acc]);
        }
        ++tc;
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  if constexpr (PAIR) cluster_sync_all();
  else __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    if constexpr (PAIR) tmem_dealloc_pair(tmem, TMEM_COLS);
    else tmem_dealloc(tmem, TMEM_COLS);
  }
}

template <int FORM, int EPI, int BN, bool AG, bool BG, bool DUAL, bool PAIR>
int launch(Params& p, int64_t units, cudaStream_t st) {
  constexpr int SMEM = smem_bytes<BN, DUAL, PAIR>();
  auto kern = grouped_kernel<FORM, EPI, BN, AG, BG, DUAL, PAIR>;
  static std::atomic<uint64_t> attr{0};
  if (smem_limit_once(reinterpret_cast<const void*>(kern), SMEM, &attr)) return 3;
  int slots;
  if constexpr (PAIR) {
    static std::atomic<int> fit[64];
    slots = gk::pair_slots(reinterpret_cast<const void*>(kern), SMEM, fit);
  } else {
    slots = sm_count();
  }
  if (slots <= 0) return 3;
  const int n = (int)std::min<int64_t>(units, slots);
  return launch_dependent(kern, PAIR ? 2 * n : n, PAIR ? 2 : 1, dim3(NUM_THREADS), (size_t)SMEM, st, p) == cudaSuccess ? 0 : 3;
}

// One translation unit per form (they compile in parallel); `small`: 64
// columns a tile, `pair`: a pair of SMs a tile.
int launch_nt(Params& p, int epi, bool gather, bool dual, bool pair, bool small, int64_t units, cudaStream_t st);
int launch_nn(Params& p, int epi, bool pair, int64_t units, cudaStream_t st);
int launch_tn(Params& p, bool a_gather, bool b_gather, bool pair, int64_t units, cudaStream_t st);

}  // namespace gg
}  // namespace bpt
