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
//   - Rows are gathered on the way in: two more warps copy them, 16 bytes a
//     lane, from where the router left them into the ring (cp.async, eight
//     lanes a 128-byte line, the swizzle applied by hand), so no copy in the
//     groups' order is ever made.  Lines behind the group's last row are not
//     copied: what their shared memory holds reaches only accumulator rows
//     that are never stored.  (TMA's own four-row gathers were taken first:
//     an instruction each, they fed a stage in about 1000 cycles where the
//     products take 256: 458 TFLOP/s on the gate and up products of 8 experts
//     of 4096 x 14336, 4096 positions.)
//   - TN runs over a group's rows as K.  The last, partial block of 64 rows
//     is copied by those warps too, with zeros behind the group's end: what
//     lies there, a NaN even, stays out.
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
constexpr int COPY_WARP = 2 + NUM_EPI_WARPS;  // the first of those that copy rows
// TN reads the rows' places anew for every block, about 1190 cycles a stage
// with two warps (8 experts of 4096 x 14336) where the products take 512
template <int FORM>
constexpr int copy_warps() {
  return FORM == GROUPED_TN ? 4 : 2;
}

struct Params {
  CUtensorMap map_a[2];  // A tiles (TN: {64, 64} boxes)
  CUtensorMap map_b[2];  // weights, or TN: B tiles
  // A and TN's B for the copying warps: row-major, a_rows and b_rows rows of
  // a_cols and b_cols columns
  const __nv_bfloat16 *a[2], *b;
  int a_cols, b_cols;
  const int* offsets;
  int groups, rows;
  int M, N, nkt, segs;    // TN: M; NT, NN: k-tiles of one segment and the number of segments (TN: segments of M)
  int mt, nt;             // TN: tile rows per segment; tile columns
  int band;               // tile rows walked before the next tile column (m fastest)
  const int* order;       // pair at each sorted row, or NULL: row r is row r
  unsigned long long by_k;  // ceil(2^37 / top_k): pair / top_k = pair * by_k >> 37, exact below 2^29 pairs and 32 choices
  int pairs;
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

// 16 bytes into shared memory, or zeros
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool some) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(some ? 16 : 0) : "memory");
}
// arrives once for this thread on `bar` (whose count has this thread in it)
// when its copies so far have landed
__device__ __forceinline__ void copy_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void copy_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// arrive on another CTA's mbarrier (shared::cluster address), ordering this
// CTA's memory alone: the products that wait for it read this CTA's copies
// from this CTA's shared memory
__device__ __forceinline__ void mbar_arrive_other(uint32_t cl_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cl_addr) : "memory");
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
__device__ __forceinline__ void epi_cols(const Params& p, void* out, long long row, int n, const float (&a)[W], const float (&b)[W]) {
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
  }  // GROUPED_ACT_BWD: act_bwd_cols
}

// The saved pair of W columns, as loaded
template <int W>
struct SavedPair {
  uint32_t s0[W / 2], s1[W / 2];
};
template <int W>
__device__ __forceinline__ void load_pair(const Params& p, long long i, SavedPair<W>& r) {
  if constexpr (W == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p.aux + i), v = *reinterpret_cast<const uint4*>(p.aux2 + i);
    r.s0[0] = u.x, r.s0[1] = u.y, r.s0[2] = u.z, r.s0[3] = u.w;
    r.s1[0] = v.x, r.s1[1] = v.y, r.s1[2] = v.z, r.s1[3] = v.w;
  } else {
#pragma unroll
    for (int h = 0; h < W / 16; ++h) {
      gk::ld32B(p.aux + i + 16 * h, *reinterpret_cast<uint32_t(*)[8]>(&r.s0[8 * h]));
      gk::ld32B(p.aux2 + i + 16 * h, *reinterpret_cast<uint32_t(*)[8]>(&r.s1[8 * h]));
    }
  }
}
// GROUPED_ACT_BWD of W columns at element i from their saved pair.  The pair is
// bf16 (off by up to 2^-8 of its size): the activation and its slopes are taken
// again from it in fp32 and rounded once.
template <int W>
__device__ __forceinline__ void act_bwd_cols(const Params& p, void* out, long long i, const uint32_t* acc, const SavedPair<W>& r, float w,
                                             float& dot) {
  constexpr int S = W < 16 ? W : 16;  // columns at a time
#pragma unroll
  for (int h = 0; h < W / S; ++h) {
    float v[S], aw[S], dv[S];
#pragma unroll
    for (int j = 0; j < S; ++j) {
      const int c = h * S + j;
      const float a = __uint_as_float(acc[c]);
      const float s0 = c & 1 ? bf16_hi(r.s0[c / 2]) : bf16_lo(r.s0[c / 2]);
      const float s1 = c & 1 ? bf16_hi(r.s1[c / 2]) : bf16_lo(r.s1[c / 2]);
      const float wa = w * a;
      if (p.act == BPT_ACT_SWIGLU) {
        const float sg = fast_sigmoid(s0);
        const float si = s0 * sg;  // silu(g)
        const float act = si * s1;
        dot = fmaf(a, act, dot);
        aw[j] = w * act;
        v[j] = wa * s1 * (sg + si * (1.f - sg));
        dv[j] = wa * si;
      } else {
        dot = fmaf(a, s0, dot);
        aw[j] = w * s0;
        v[j] = wa * s1;
        dv[j] = 0.f;
      }
    }
    gk::storew_bf16<S>(reinterpret_cast<__nv_bfloat16*>(out) + i + h * S, v);
    if (p.act == BPT_ACT_SWIGLU) gk::storew_bf16<S>(reinterpret_cast<__nv_bfloat16*>(p.out2) + i + h * S, dv);
    gk::storew_bf16<S>(reinterpret_cast<__nv_bfloat16*>(p.out3) + i + h * S, aw);
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
template <int FORM, bool AG>
constexpr bool copies() {  // whether the kernel has the copying warps
  return AG || FORM == GROUPED_TN;
}
template <int FORM, bool AG>
constexpr int threads() {
  return 32 * (2 + NUM_EPI_WARPS + (copies<FORM, AG>() ? copy_warps<FORM>() : 0));
}

template <int FORM, int EPI, int BN, bool AG, bool BG, bool DUAL, bool PAIR>
__global__ void __launch_bounds__(threads<FORM, AG>(), 1) grouped_kernel(const __grid_constant__ Params p) {
  constexpr bool TN = FORM == GROUPED_TN;
  constexpr bool B_MN = FORM != GROUPED_NT;
  constexpr bool COPY = copies<FORM, AG>();
  constexpr int COPY_WARPS = copy_warps<FORM>();
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
  uint64_t* copied = drain + 1;  // [STAGES], this CTA's copying warps
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(copied + STAGES);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* s_unit = reinterpret_cast<int*>(smem + STAGES * STAGE_BYTES + 256);  // [groups + 1]
  int* s_lo = s_unit + GROUPED_MAX_GROUPS + 4;
  int* s_cnt = s_lo + GROUPED_MAX_GROUPS;
  static_assert((3 * STAGES + 5) * 8 + 8 <= 256, "barriers");

  const int warp = warp_id();
  const int lane = lane_id();
  const uint32_t rank = PAIR ? cluster_rank() : 0u;
  const int unit0 = PAIR ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
  const int units_in_flight = PAIR ? (int)(gridDim.x >> 1) : (int)gridDim.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      // the loads' bytes, and word of the other CTA's copies
      mbar_init(&full[s], 1 + (COPY && PAIR ? 1 : 0));
      mbar_init(&empty[s], 1);
      mbar_init(&copied[s], 32 * COPY_WARPS);
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
    if (lane == 0) {
      // ------------------------------------------------ producer
      const uint32_t full0 = PAIR ? cluster_addr(smem_u32(full), 0) : smem_u32(full);
      const uint32_t smem_base = smem_u32(smem);
      uint32_t it = 0;
      bool ok = true;
      Place at;
      at.e = 0;
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
      for (int unit = unit0; ok && unit < nunits; unit += units_in_flight) {
        place<TN, TM, BN>(p, unit, s_unit, s_lo, s_cnt, at);
        const int nbs = at.n0 + (int)rank * BNS;
        const int ma = at.m0 + (int)rank * BM;
        const int nk = k_tiles(at);
        for (int kt = 0; kt < nk; ++kt) {
          const int s = it % STAGES;
          if (it >= (uint32_t)STAGES && !bounded_wait(&empty[s], ((it / STAGES) & 1) ^ 1, abort_flag, 101, p.err)) {
            ok = false;
            break;
          }
          const uint32_t sa = smem_base + s * STAGE_BYTES;
          const uint32_t sb = sa + A_BYTES;
          const uint32_t fb = full0 + 8u * (uint32_t)s;
          if constexpr (!TN) {
            const int seg = FORM == GROUPED_NN && kt >= p.nkt ? 1 : 0;
            const int kx = (kt - seg * p.nkt) * BK;
            if (rank == 0) mbar_expect_tx(&full[s], (PAIR ? 2 : 1) * (STAGE_BYTES - (AG ? A_BYTES : 0)));
            if constexpr (!AG) load2(sa, &p.map_a[seg], fb, kx, at.lo + ma);
            if constexpr (FORM == GROUPED_NT) {
              load3(sb, &p.map_b[0], fb, kx, nbs, at.e);
              if constexpr (DUAL) load3(sb + BNS * BK * 2, &p.map_b[1], fb, kx, nbs, at.e);
            } else {
#pragma unroll
              for (int c = 0; c < BNS / 64; ++c) load3(sb + c * 8192, &p.map_b[seg], fb, nbs + c * 64, kx, at.e);
            }
          } else {
            const bool whole = (kt + 1) * BK <= at.cnt;
            const int y = at.lo + kt * BK;
            const uint32_t bytes = whole ? (AG ? 0 : A_BYTES) + (BG ? 0 : STAGE_BYTES - A_BYTES) : 0;
            if (rank == 0) mbar_expect_tx(&full[s], (PAIR ? 2 : 1) * bytes);
            if (!AG && whole) {
              load2(sa, &p.map_a[at.seg], fb, ma, y);
              load2(sa + 8192, &p.map_a[at.seg], fb, ma + 64, y);
            }
            if (!BG && whole) {
#pragma unroll
              for (int c = 0; c < BNS / 64; ++c) load2(sb + c * 8192, &p.map_b[0], fb, nbs + c * 64, y);
            }
          }
          ++it;
        }
      }
      if (*abort_flag) {
        // let every load issued land before the CTA goes away; a pair's ranks
        // cannot wait for one another's stragglers and give them a fixed time
        if (rank == 0 && !COPY)
          for (uint32_t j = (it > (uint32_t)STAGES ? it - STAGES : 0); j < it; ++j) drain_wait(&full[j % STAGES], (j / STAGES) & 1);
        if (PAIR || COPY) {
          const long long t0 = clock64();
          while (clock64() - t0 < 1000000) {
          }
        }
      }
    }
  } else if (COPY && warp >= COPY_WARP) {
    // -------------------------------------------------- copying warps
    // A stage's operand is 128 lines of 128 bytes for the CTA's 128 rows (TN:
    // 64 rows of each 64-column chunk).  A lane holds 16 bytes of a line at
    // their swizzled place: chunk (lane % 8) ^ (line % 8).
    const int w = warp - COPY_WARP;
    const uint32_t smem_base = smem_u32(smem);
    const int col = (lane & 7) * 8;  // this lane's columns of a line
    uint32_t it = 0;
    bool ok = true;
    Place at;
    at.e = 0;
    auto row_of = [&](int r) {  // row of the gathered tensor at row r of the order; -1: none
      const int q = p.order[r];
      return q < 0 || q >= p.pairs ? -1 : (int)(((unsigned long long)(unsigned)q * p.by_k) >> 37);
    };
    auto claim = [&]() {
      const int s = it % STAGES;
      return it < (uint32_t)STAGES || bounded_wait_w(&empty[s], ((it / STAGES) & 1) ^ 1, abort_flag, 102, p.err);
    };
    auto next = [&]() {
      copy_arrive(&copied[it % STAGES]);
      ++it;
    };
    for (int unit = unit0; ok && unit < nunits; unit += units_in_flight) {
      place<TN, TM, BN>(p, unit, s_unit, s_lo, s_cnt, at);
      const int nk = k_tiles(at);
      if constexpr (!TN) {
        // lines w * PER + 4 i + lane / 8 of the CTA's rows
        constexpr int PER = BM / COPY_WARPS;
        const int r0 = at.m0 + (int)rank * BM + w * PER + (lane >> 3);
        int idx[PER / 4];
#pragma unroll
        for (int i = 0; i < PER / 4; ++i) {
          const int r = r0 + 4 * i;
          idx[i] = r >= at.cnt ? -2 : p.order ? row_of(at.lo + r) : at.lo + r;
        }
        const int live = (at.cnt - r0 + 3) / 4;  // lines of this lane with a row
        const uint32_t line0 = (uint32_t)(w * PER + (lane >> 3));
        for (int kt = 0; kt < nk; ++kt) {
          if (!claim()) {
            ok = false;
            break;
          }
          const int seg = FORM == GROUPED_NN && kt >= p.nkt ? 1 : 0;
          const int x = (kt - seg * p.nkt) * BK + col;
          const bool in = x < p.a_cols;
          const __nv_bfloat16* src = p.a[seg] + (in ? x : 0);
          const uint32_t sa = smem_base + (it % STAGES) * STAGE_BYTES;
#pragma unroll
          for (int i = 0; i < PER / 4; ++i) {
            if (i < live) {
              const uint32_t line = line0 + 4 * i;
              copy16(sa + line * 128 + ((((lane & 7) ^ line) & 7) << 4), src + (long long)max(idx[i], 0) * p.a_cols, in && idx[i] >= 0);
            }
          }
          next();
        }
      } else {
        // rows w * PER + 4 i + lane / 8 of a block, in every chunk of 64 columns
        constexpr int PER = BK / COPY_WARPS, LINES = PER / 4;
        const int ma = at.m0 + (int)rank * BM, nbs = at.n0 + (int)rank * BNS;
        constexpr int AHEAD = 4;  // blocks whose rows of the order are on their way
        int ring[AG || BG ? AHEAD : 1][LINES];
        auto fetch = [&](int kt, int (&v)[LINES]) {
#pragma unroll
          for (int i = 0; i < LINES; ++i) {
            const int r = kt * BK + w * PER + 4 * i + (lane >> 3);
            v[i] = r < at.cnt ? p.order[at.lo + r] : -1;
          }
        };
        const uint32_t line0 = (uint32_t)(w * PER + (lane >> 3));
        auto lines = [&](uint32_t dst, const __nv_bfloat16* src, int cols, int x0, int chunks, const int (&rows)[LINES]) {
          const __nv_bfloat16* from[LINES];
#pragma unroll
          for (int i = 0; i < LINES; ++i) from[i] = src + (long long)max(rows[i], 0) * cols + x0 + col;
#pragma unroll
          for (int c = 0; c < chunks; ++c) {
            const bool in = x0 + c * 64 + col < cols;
#pragma unroll
            for (int i = 0; i < LINES; ++i) {
              const uint32_t line = line0 + 4 * i;
              const bool some = in && rows[i] >= 0;
              copy16(dst + c * 8192 + line * 128 + ((((lane & 7) ^ line) & 7) << 4), some ? from[i] + c * 64 : src, some);
            }
          }
        };
        constexpr int A_CHUNKS = 2, B_CHUNKS = BNS / 64;
        if constexpr (AG || BG) {
#pragma unroll
          for (int u = 0; u < AHEAD; ++u) fetch(u, ring[u]);
        }
        for (int k4 = 0; ok && k4 < nk; k4 += AHEAD) {
#pragma unroll
          for (int u = 0; u < AHEAD; ++u) {
            const int kt = k4 + u;
            if (kt >= nk) break;
            if (!claim()) {
              ok = false;
              break;
            }
            const uint32_t sa = smem_base + (it % STAGES) * STAGE_BYTES;
            const uint32_t sb = sa + A_BYTES;
            const bool whole = (kt + 1) * BK <= at.cnt;
            if constexpr (AG || BG) {
              int rows[LINES];
#pragma unroll
              for (int i = 0; i < LINES; ++i) {
                const int q = ring[u][i];
                rows[i] = q < 0 || q >= p.pairs ? -1 : (int)(((unsigned long long)(unsigned)q * p.by_k) >> 37);
              }
              fetch(kt + AHEAD, ring[u]);
              if constexpr (AG) lines(sa, p.a[0], p.a_cols, ma, A_CHUNKS, rows);
              else lines(sb, p.b, p.b_cols, nbs, B_CHUNKS, rows);
            }
            if (!whole) {
              int rows[LINES];
#pragma unroll
              for (int i = 0; i < LINES; ++i) {
                const int r = kt * BK + w * PER + 4 * i + (lane >> 3);
                rows[i] = r < at.cnt ? at.lo + r : -1;
              }
              if constexpr (!AG) lines(sa, at.seg ? p.a[1] : p.a[0], p.a_cols, ma, A_CHUNKS, rows);
              if constexpr (!BG) lines(sb, p.b, p.b_cols, nbs, B_CHUNKS, rows);
            }
            next();
          }
        }
      }
    }
    copy_wait_all();
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
          if (!bounded_wait_w(&full[s], (it / STAGES) & 1, abort_flag, 103, p.err) ||
              (COPY && !bounded_wait_w(&copied[s], (it / STAGES) & 1, abort_flag, 104, p.err))) {
            ok = false;
            break;
          }
          if constexpr (COPY) fence_proxy_async_smem();  // the copies are read by the tensor core
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
    } else if (COPY) {
      // the pair's other CTA: word of every stage's copies to the one that issues
      const uint32_t full0 = cluster_addr(smem_u32(full), 0);
      uint32_t it = 0;
      bool ok = true;
      Place at;
      at.e = 0;
      for (int unit = unit0; ok && unit < nunits; unit += units_in_flight) {
        place<TN, TM, BN>(p, unit, s_unit, s_lo, s_cnt, at);
        const int nk = k_tiles(at);
        for (int kt = 0; kt < nk; ++kt, ++it) {
          const int s = it % STAGES;
          if (!bounded_wait_w(&copied[s], (it / STAGES) & 1, abort_flag, 104, p.err)) {
            ok = false;
            break;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive_other(full0 + 8u * (uint32_t)s);
        }
      }
    }
  } else if (warp < COPY_WARP) {
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
      const int m = at.m0 + (int)rank * BM + q * 32 + lane;
      const bool mine = m < (TN ? p.M : at.cnt);
      const long long row = TN ? (long long)at.e * p.M + m : (long long)at.lo + m;
      void* out = TN && at.seg ? p.out2 : p.out;
      float w = 0.f, dot = 0.f;
      SavedPair<EPI == GROUPED_ACT_BWD ? 32 : 8> pair;
      // the saved pair of a chunk of 32 columns is on its way while the chunk
      // before is worked on, the first while the products are
      auto fetch = [&](int c) {
        const int nb = at.n0 + half * EPI_COLS + c * 32;
        if (mine && p.vec32 && nb + 32 <= p.N) load_pair(p, row * p.N + nb, pair);
      };
      if constexpr (EPI == GROUPED_ACT_BWD) {
        if (mine) {
          const int q1 = p.order[row];
          if (q1 >= 0 && q1 < p.pairs)
            w = p.row_weight_f32 ? reinterpret_cast<const float*>(p.row_weight)[q1]
                                 : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.row_weight)[q1]);
        }
        fetch(0);
      }
      if (!none) {
        // the TMEM loads below are warp-collective, so the decision is too
        const bool ok = __all_sync(0xffffffffu, bounded_wait(&acc_full[acc], (tc >> 1) & 1, abort_flag, 105, p.err));
        if (!ok) break;
        tc_fence_after();
      } else if (p.beta != 0.f) {
        continue;  // nothing to add
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
        if constexpr (EPI == GROUPED_ACT_BWD) {
          if (nb + 32 <= p.N && p.vec32) {
            const SavedPair<32> now = pair;
            if (c + 1 < EPI_COLS / 32) fetch(c + 1);
            if (mine) act_bwd_cols<32>(p, out, row * p.N + nb, ra, now, w, dot);
          } else if (mine) {
#pragma unroll
            for (int g = 0; g < 4; ++g)
              if (nb + g * 8 < p.N) {  // N is a multiple of 8
                SavedPair<8> now;
                load_pair(p, row * p.N + nb + g * 8, now);
                act_bwd_cols<8>(p, out, row * p.N + nb + g * 8, ra + g * 8, now, w, dot);
              }
          }
        } else if (mine) {
          if (nb + 32 <= p.N && p.vec32) {
            float a32[32], b32[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              a32[j] = __uint_as_float(ra[j]);
              b32[j] = DUAL ? __uint_as_float(rb[j]) : 0.f;
            }
            epi_cols<EPI, DUAL, 32>(p, out, row, nb, a32, b32);
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
                epi_cols<EPI, DUAL, 8>(p, out, row, nb + g * 8, a8, b8);
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
  return launch_dependent(kern, PAIR ? 2 * n : n, PAIR ? 2 : 1, dim3(threads<FORM, AG>()), (size_t)SMEM, st, p) == cudaSuccess ? 0 : 3;
}

// One translation unit per form (they compile in parallel); `small`: 64
// columns a tile, `pair`: a pair of SMs a tile.
int launch_nt(Params& p, int epi, bool gather, bool dual, bool pair, bool small, int64_t units, cudaStream_t st);
int launch_nn(Params& p, int epi, bool pair, int64_t units, cudaStream_t st);
int launch_tn(Params& p, bool a_gather, bool b_gather, bool pair, int64_t units, cudaStream_t st);

}  // namespace gg
}  // namespace bpt
