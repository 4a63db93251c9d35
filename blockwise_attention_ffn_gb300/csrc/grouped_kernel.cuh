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
//   - Rows are gathered on the way in: two or four more warps copy them, 16 bytes a
//     lane, from where the router left them into the ring (cp.async, eight
//     lanes a 128-byte line, the swizzle applied by hand), so no copy in the
//     groups' order is ever made.  Lines behind the group's last row are not
//     copied: what their shared memory holds reaches only accumulator rows
//     that are never stored.  The copies complete a barrier of their CTA; a
//     pair's second CTA passes word of it on.  (TMA's own four-row gathers, an
//     instruction for each quad of rows, reached 458 TFLOP/s on the gate and up
//     products of 8 experts of 4096 x 14336, 4096 positions; the copies 1570.)
//   - TN runs over a group's rows as K.  The last, partial block of 64 rows
//     is copied by those warps too, with zeros behind the group's end: what
//     lies there, a NaN even, stays out.
//   - Weights are 3-D maps [G, rows, cols]: a tile that runs over a matrix's
//     edge reads zeros, not the next group's matrix.
#pragma once

#include "attn_common.cuh"
#include "gemm_kernel.cuh"
#include "grouped.h"

namespace bpt {
namespace gg {

using gk::BK;
using gk::BM;
using gk::NUM_EPI_WARPS;
constexpr int COPY_WARP = 2 + NUM_EPI_WARPS;  // the first of those that copy rows
// TN reads the rows' places anew for every block: about 1190 cycles a stage with
// two warps (8 experts of 4096 x 14336), 860 with four, where the products take
// 512; eight cost the epilogue its registers and gain nothing.  Of the others NN
// (the backward's first product: 772 us with two, 720 with four) takes four, NT
// two (1227 and 1355 us: its epilogue keeps two accumulators' columns).
template <int FORM>
constexpr int copy_warps() {
  return FORM == GROUPED_NT ? 2 : 4;
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
  unsigned long long by_k;  // ceil(2^37 / top_k): pair / top_k = pair * by_k >> 37, exact up to 2^26 pairs and 32 choices
  int pairs;
  void *out, *out2, *out3;
  int out_f32;
  float beta;
  const __nv_bfloat16 *aux, *aux2;
  const void* row_weight;
  int row_weight_f32;
  float* part;
  int2* span;  // for the rows that the groups hold (grouped.h), or NULL
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
  bool odd = false;
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
    odd |= in && !ok;
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
  odd = __any_sync(0xffffffffu, odd);
  if (lane == 0) {
    s_unit[0] = 0;
    if (p.span && blockIdx.x == 0) *p.span = make_int2(odd ? -1 : p.offsets[0], p.offsets[p.groups]);
  }
}

// TN: the groups by falling row count, equal ones in their order, by all
// threads of the block after lay_out (whose lists they reorder; s_id: the
// group at each place).  A unit's work is its group's rows, and the units go
// round the CTAs in snakes (unit_of below), so heavy and light ones even out.
constexpr int SORT_MOST = (GROUPED_MAX_GROUPS + 319) / 320;  // groups a thread, of at least 320
__device__ __forceinline__ void sort_groups(const Params& p, int* s_lo, int* s_cnt, int* s_id) {
  int lo[SORT_MOST], cnt[SORT_MOST], rank[SORT_MOST];
#pragma unroll
  for (int i = 0; i < SORT_MOST; ++i) {
    const int e = (int)threadIdx.x + i * (int)blockDim.x;
    rank[i] = 0;
    if (e < p.groups) {
      lo[i] = s_lo[e];
      cnt[i] = s_cnt[e];
      for (int o = 0; o < p.groups; ++o) rank[i] += s_cnt[o] > cnt[i] || (s_cnt[o] == cnt[i] && o < e);
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < SORT_MOST; ++i) {
    const int e = (int)threadIdx.x + i * (int)blockDim.x;
    if (e < p.groups) {
      s_lo[rank[i]] = lo[i];
      s_cnt[rank[i]] = cnt[i];
      s_id[rank[i]] = e;
    }
  }
}

// A work unit's place: group, first row of the tile in the group (TN: of the
// matrix), first column, segment of M (TN).
struct Place {
  int e, lo, cnt, m0, n0, seg;
};
template <bool TN, int TM, int BN>
__device__ __forceinline__ void place(const Params& p, int unit, const int* s_unit, const int* s_lo, const int* s_cnt, const int* s_id,
                                      Place& at) {
  int local, mt;
  if constexpr (TN) {
    // every group has the same units; the groups with the most rows first
    mt = p.segs * p.mt;
    const int g = unit / (mt * p.nt);
    at.e = s_id[g];
    at.lo = s_lo[g];
    at.cnt = s_cnt[g];
    local = unit - g * (mt * p.nt);
  } else {
    int e = at.e;  // units come in rising order
    while (unit >= s_unit[e + 1]) ++e;
    at.e = e;
    at.lo = s_lo[e];
    at.cnt = s_cnt[e];
    local = unit - s_unit[e];
    mt = (at.cnt + TM - 1) / TM;
  }
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

// The activations' arithmetic on two columns at a time (attn_common.cuh's
// packed forms): the epilogues are bound by issue slots, two warps a scheduler
// with some 34 scalar instructions a column (the tanh GeLU's gradient of a
// 32-column chunk took 2300 cycles).
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint64_t rcp2(uint64_t v) {
  const float2 x = f2split(v);
  return f2(rcp(x.x), rcp(x.y));
}
__device__ __forceinline__ uint64_t exp2_2(uint64_t v) {
  const float2 x = f2split(v);
  return f2(ex2(x.x), ex2(x.y));
}
// 1 / (1 + 2^x), with an error of a few units of fp32's last place: what it
// enters is rounded to bf16.  sigmoid(z) at x = -z log2(e)
__device__ __forceinline__ uint64_t sigmoid_of(uint64_t x) { return rcp2(add2(exp2_2(x), f2(1.f, 1.f))); }

// GeLU and its slope: z cdf(z), cdf + z pdf(z) with the cdf as in
// gemm_kernel.cuh (gelu_erf_parts), or the tanh form as z s with
// s = sigmoid(2 c (z + 0.044715 z^3)), c = sqrt(2 / pi).
template <int ACT>
__device__ __forceinline__ void gelu2(uint64_t z, uint64_t& g, uint64_t& d) {
  auto c2 = [](float v) { return f2(v, v); };
  if constexpr (ACT == BPT_ACT_GELU_ERF) {
    const uint64_t zz = mul2(z, z);
    const float2 v = f2split(z);
    const uint64_t t = rcp2(fma2(f2(fabsf(v.x), fabsf(v.y)), c2(0.3275911f * 0.70710678118654752f), c2(1.f)));
    uint64_t poly = fma2(c2(1.061405429f), t, c2(-1.453152027f));
    poly = fma2(poly, t, c2(1.421413741f));
    poly = fma2(poly, t, c2(-0.284496736f));
    poly = fma2(poly, t, c2(0.254829592f));
    const uint64_t e = exp2_2(mul2(zz, c2(-0.72134752044448170f)));  // exp(-z^2 / 2)
    const uint64_t tail = mul2(mul2(poly, t), mul2(e, c2(0.5f)));     // 0.5 (1 - erf(|z| / sqrt 2))
    const float2 lo = f2split(tail), hi = f2split(sub2(c2(1.f), tail));
    const uint64_t cdf = f2(v.x >= 0.f ? hi.x : lo.x, v.y >= 0.f ? hi.y : lo.y);
    g = mul2(z, cdf);
    d = fma2(mul2(z, e), c2(0.3989422804014327f), cdf);
  } else {
    const float c = 1.5957691216057308f, l2e = 1.4426950408889634f;
    const uint64_t kz = mul2(z, c2(-l2e * c * 0.044715f));
    const uint64_t s = sigmoid_of(mul2(z, fma2(kz, z, c2(-l2e * c))));
    g = mul2(z, s);
    const uint64_t rest = mul2(g, sub2(c2(1.f), s));
    // s + rest c (1 + 3 * 0.044715 z^2), z by z: far out rest is 0 where z^2 is infinite
    d = fma2(mul2(rest, z), mul2(kz, c2(-3.f / l2e)), fma2(rest, c2(c), s));
  }
}

// A warp's 32 output rows, one a lane in registers, to global memory by whole
// 64- or 128-byte pieces of a row, through the warp's 2 KB of shared memory.
// (Stored straight from the registers, 32 bytes of 32 rows at a time, the fp32
// gradient of 16 matrices of 2048 x 2560 over 14336 rows took 155 us, this way
// 141, and the GeLU product of 12 experts of 1000 x 2744 116 and 84.)  P 16-byte words a row: 4, all rows at once, or 8, 16 rows at a
// time.  The words' places are swapped so that neither the rows' writes nor
// the lines' reads meet in a bank.  to: the first row's first byte; ld: bytes
// from row to row; rows, words: how many of them there are.
template <int P, bool ADD>
__device__ __forceinline__ void put_rows(const uint32_t* v, uint4* stage, char* to, long long ld, int rows, int words, float beta) {
  const int lane = lane_id();
  constexpr int STEPS = P == 8 ? 2 : 1, AT_ONCE = 32 / P;  // rows a store covers
#pragma unroll
  for (int h = 0; h < STEPS; ++h) {
    if (STEPS == 1 || (lane >> 4) == h) {
      const int r = STEPS == 1 ? lane : lane & 15;
      const int mix = P == 8 ? r & 7 : (r >> 1) & 3;
#pragma unroll
      for (int j = 0; j < P; ++j) stage[r * P + (j ^ mix)] = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    }
    __syncwarp();
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int r = t * AT_ONCE + lane / P, j = lane % P;
      const int mix = P == 8 ? r & 7 : (r >> 1) & 3;
      uint4 w = stage[r * P + (j ^ mix)];
      const int row = h * 16 + r;
      if (row < rows && j < words) {
        uint4* o = reinterpret_cast<uint4*>(to + row * ld) + j;
        if constexpr (ADD) {
          const float4 old = *reinterpret_cast<const float4*>(o);
          w.x = __float_as_uint(fmaf(beta, old.x, __uint_as_float(w.x)));
          w.y = __float_as_uint(fmaf(beta, old.y, __uint_as_float(w.y)));
          w.z = __float_as_uint(fmaf(beta, old.z, __uint_as_float(w.z)));
          w.w = __float_as_uint(fmaf(beta, old.w, __uint_as_float(w.w)));
        }
        *o = w;
      }
    }
    __syncwarp();
  }
}

// What the forward leaves for the backward (SwiGLU: the gate and the up
// product; GeLU: the product) is read by these kernels alone, so it lies as a
// warp holds it: blocks of 32 rows of a group (the last one of fewer), in them
// chunks of 32 columns, in them the 16-byte words of 8 columns, each for all
// rows of the block.  A warp's words are then whole lines.  Element of word 0
// of chunk c for the row at `lane` of the block of `rows` rows that begins
// `first` rows into the order; a word further is 8 * rows.
__device__ __forceinline__ long long kept_at(const Params& p, long long first, int rows, int c, int lane) {
  return first * p.N + ((long long)c * 4 * rows + lane) * 8;
}
__device__ __forceinline__ void keep(void* t, long long at, int rows, int words, const uint32_t* v) {
  uint4* o = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(t) + at);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < words) o[j * rows] = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
}
__device__ __forceinline__ void kept(const __nv_bfloat16* t, long long at, int rows, int words, uint32_t* v) {
  const uint4* o = reinterpret_cast<const uint4*>(t + at);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint4 u = j < words ? __ldg(o + j * rows) : make_uint4(0, 0, 0, 0);
    v[4 * j] = u.x, v[4 * j + 1] = u.y, v[4 * j + 2] = u.z, v[4 * j + 3] = u.w;
  }
}

constexpr int PUT_BYTES = 2048;  // shared memory of put_rows, a warp
// Few rows a group (64-column tiles): the weights' bytes bound the product and a
// stage's hand-overs, some 600 cycles, its rate.  So a stage holds two blocks of
// 64 K, and 32 rows of A at most: the product's other 96 rows are whatever lies
// behind them in the ring (in bounds; accumulator rows that are never stored).
template <int BN>
constexpr int k_blocks() {  // of a stage
  return BN == 64 ? 2 : 1;
}
template <int BN>
constexpr int a_rows() {  // staged by a CTA
  return BN == 64 ? 32 : BM;
}
template <int BN, bool DUAL, bool PAIR>
constexpr int stage_bytes() {
  return k_blocks<BN>() * (a_rows<BN>() + (DUAL ? 2 : 1) * (PAIR ? BN / 2 : BN)) * BK * 2;
}
// ring stages that fit beside put_rows' memory and the group lists
template <int STAGE_BYTES>
constexpr int ring_stages() {
  return 198 * 1024 / STAGE_BYTES > 8 ? 8 : 198 * 1024 / STAGE_BYTES;
}
template <int BN, bool DUAL, bool PAIR>
constexpr int smem_bytes() {
  return ring_stages<stage_bytes<BN, DUAL, PAIR>()>() * stage_bytes<BN, DUAL, PAIR>() + NUM_EPI_WARPS * PUT_BYTES + 1024 + 256 +
         (4 * GROUPED_MAX_GROUPS + 4) * 4;
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

// ACT: the activation of GROUPED_ACT and GROUPED_ACT_BWD (a branch for each
// value otherwise; 0 elsewhere).
template <int FORM, int EPI, int ACT, int BN, bool AG, bool BG, bool DUAL, bool PAIR>
__global__ void __launch_bounds__(threads<FORM, AG>(), 1) grouped_kernel(const __grid_constant__ Params p) {
  constexpr bool GATED = ACT == BPT_ACT_SWIGLU;
  static_assert(EPI != GROUPED_ACT || GATED == DUAL, "gate and up");
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
  constexpr int KB = k_blocks<BN>(), A_ROWS = a_rows<BN>();
  constexpr int A_STAGE = KB * A_ROWS * BK * 2, B_BLOCK = (DUAL ? 2 : 1) * BNS * BK * 2;
  static_assert(BN != 64 || (FORM == GROUPED_NT && AG && !PAIR), "few rows");
  constexpr int TM = PAIR ? 2 * BM : A_ROWS;
  constexpr uint32_t IDESC = idesc_bf16(PAIR ? 2 * BM : BM, BN, TN, B_MN);

  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* put = smem + STAGES * STAGE_BYTES;  // the epilogue warps'
  uint64_t* full = reinterpret_cast<uint64_t*>(put + NUM_EPI_WARPS * PUT_BYTES);
  uint64_t* empty = full + STAGES;
  uint64_t* acc_full = empty + STAGES;  // [2]
  uint64_t* acc_empty = acc_full + 2;   // [2]
  uint64_t* drain = acc_empty + 2;
  uint64_t* copied = drain + 1;  // [STAGES], this CTA's copying warps
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(copied + STAGES);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* s_unit = reinterpret_cast<int*>(put + NUM_EPI_WARPS * PUT_BYTES + 256);  // [groups + 1]
  int* s_lo = s_unit + GROUPED_MAX_GROUPS + 4;
  int* s_cnt = s_lo + GROUPED_MAX_GROUPS;
  int* s_id = s_cnt + GROUPED_MAX_GROUPS;
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
  if constexpr (TN) {
    __syncthreads();
    sort_groups(p, s_lo, s_cnt, s_id);
  }
  tc_fence_before();
  if constexpr (PAIR) cluster_sync_all();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const int nunits = s_unit[p.groups];
  // this CTA's (or pair's) unit in a round over all of them: TN's rounds run to
  // and fro
  auto unit_of = [&](int round) { return round * units_in_flight + (TN && (round & 1) ? units_in_flight - 1 - unit0 : unit0); };
  // k-tiles of a unit
  auto k_tiles = [&](const Place& at) { return TN ? (at.cnt + BK - 1) / BK : p.segs * ((p.nkt + KB - 1) / KB); };

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
      for (int round = 0; ok; ++round) {
        const int unit = unit_of(round);
        if (unit >= nunits) break;  // the last round's
        place<TN, TM, BN>(p, unit, s_unit, s_lo, s_cnt, s_id, at);
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
          const uint32_t sb = sa + A_STAGE;
          const uint32_t fb = full0 + 8u * (uint32_t)s;
          if constexpr (!TN) {
            const int seg = FORM == GROUPED_NN && kt >= p.nkt ? 1 : 0;
            const int kx = (kt - seg * p.nkt) * (KB * BK);
            if (rank == 0) mbar_expect_tx(&full[s], (PAIR ? 2 : 1) * (STAGE_BYTES - (AG ? A_STAGE : 0)));
            if constexpr (!AG) load2(sa, &p.map_a[seg], fb, kx, at.lo + ma);
            if constexpr (FORM == GROUPED_NT) {
#pragma unroll
              for (int i = 0; i < KB; ++i) {
                load3(sb + i * B_BLOCK, &p.map_b[0], fb, kx + i * BK, nbs, at.e);
                if constexpr (DUAL) load3(sb + i * B_BLOCK + BNS * BK * 2, &p.map_b[1], fb, kx + i * BK, nbs, at.e);
              }
            } else {
#pragma unroll
              for (int c = 0; c < BNS / 64; ++c) load3(sb + c * 8192, &p.map_b[seg], fb, nbs + c * 64, kx, at.e);
            }
          } else {
            const bool whole = (kt + 1) * BK <= at.cnt;
            const int y = at.lo + kt * BK;
            const uint32_t bytes = whole ? (AG ? 0 : A_STAGE) + (BG ? 0 : STAGE_BYTES - A_STAGE) : 0;
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
    for (int round = 0; ok; ++round) {
      const int unit = unit_of(round);
      if (unit >= nunits) break;  // the last round's
      place<TN, TM, BN>(p, unit, s_unit, s_lo, s_cnt, s_id, at);
      const int nk = k_tiles(at);
      if constexpr (!TN) {
        // lines w * PER + 4 i + lane / 8 of the CTA's rows
        constexpr int PER = A_ROWS / COPY_WARPS;
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
#pragma unroll
          for (int kb = 0; kb < KB; ++kb) {
            const int x = ((kt - seg * p.nkt) * KB + kb) * BK + col;
            const bool in = x < p.a_cols;
            const __nv_bfloat16* src = p.a[seg] + (in ? x : 0);
            const uint32_t sa = smem_base + (it % STAGES) * STAGE_BYTES + kb * (A_ROWS * BK * 2);
#pragma unroll
            for (int i = 0; i < PER / 4; ++i) {
              if (i < live) {
                const uint32_t line = line0 + 4 * i;
                copy16(sa + line * 128 + ((((lane & 7) ^ line) & 7) << 4), src + (long long)max(idx[i], 0) * p.a_cols, in && idx[i] >= 0);
              }
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
            const uint32_t sb = sa + A_STAGE;
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
      for (int round = 0; ok; ++round) {
        const int unit = unit_of(round);
        if (unit >= nunits) break;  // the last round's
        place<TN, TM, BN>(p, unit, s_unit, s_lo, s_cnt, s_id, at);
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
          // with copies in the pair's other CTA, its word of them is on `full` too
          const bool landed = COPY && PAIR ? bounded_wait_cluster_w(&full[s], (it / STAGES) & 1, abort_flag, 103, p.err)
                                           : bounded_wait_w(&full[s], (it / STAGES) & 1, abort_flag, 103, p.err);
          if (!landed || (COPY && !bounded_wait_w(&copied[s], (it / STAGES) & 1, abort_flag, 104, p.err))) {
            ok = false;
            break;
          }
          if constexpr (COPY) fence_proxy_async_smem();  // the copies are read by the tensor core
          tc_fence_after();
          const uint32_t sa = smem_base + s * STAGE_BYTES;
          const uint32_t sb = sa + A_STAGE;
#pragma unroll
          for (int kk = 0; kk < KB * BK / 16; ++kk) {
            const uint32_t ka = sa + (kk / 4) * (A_ROWS * BK * 2), kb = sb + (kk / 4) * B_BLOCK;  // the block of 64
            const int in = kk % 4;
            const uint64_t ad = TN ? sdesc(ka + in * 2048, 8192, 1024, 2) : sdesc(ka + in * 32, 16, 1024, 2);
            const uint64_t bd = B_MN ? sdesc(kb + in * 2048, 8192, 1024, 2) : sdesc(kb + in * 32, 16, 1024, 2);
            const bool accum = kt != 0 || kk != 0;
            if constexpr (PAIR) umma_bf16_pair_w(d, ad, bd, IDESC, accum);
            else umma_bf16_w(d, ad, bd, IDESC, accum);
            if (DUAL) {
              const uint64_t bd2 = sdesc(kb + BNS * BK * 2 + in * 32, 16, 1024, 2);
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
      // The pair's other CTA: word of every stage's copies to the one that issues.
      // The products there read this CTA's shared memory, so the arrival releases
      // that at the cluster's scope and the issuing warp's wait acquires at it.
      const uint32_t full0 = cluster_addr(smem_u32(full), 0);
      uint32_t it = 0;
      bool ok = true;
      Place at;
      at.e = 0;
      for (int round = 0; ok; ++round) {
        const int unit = unit_of(round);
        if (unit >= nunits) break;  // the last round's
        place<TN, TM, BN>(p, unit, s_unit, s_lo, s_cnt, s_id, at);
        const int nk = k_tiles(at);
        for (int kt = 0; kt < nk; ++kt, ++it) {
          const int s = it % STAGES;
          if (!bounded_wait_w(&copied[s], (it / STAGES) & 1, abort_flag, 104, p.err)) {
            ok = false;
            break;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_smem(full0 + 8u * (uint32_t)s);
        }
      }
    }
  } else if (warp < COPY_WARP) {
    // -------------------------------------------------- epilogue (warps 2..9)
    constexpr int EPI_COLS = BN / 2;
    const int q = warp & 3;
    const int half = (warp - 2) >> 2;
    const uint32_t acc_empty0 = PAIR ? cluster_addr(smem_u32(acc_empty), 0) : 0u;
    uint4* stage = reinterpret_cast<uint4*>(put + (warp - 2) * PUT_BYTES);
    int tc = 0;
    Place at;
    at.e = 0;
    for (int round = 0;; ++round) {
      const int unit = unit_of(round);
      if (unit >= nunits) break;  // the last round's
      place<TN, TM, BN>(p, unit, s_unit, s_lo, s_cnt, s_id, at);
      const bool none = k_tiles(at) == 0;
      const int acc = tc & 1;
      const int m0 = at.m0 + (int)rank * BM + q * 32;  // the warp's first row in the group (TN: of the matrix)
      const int rows = TM == 32 && q ? 0 : max(0, min(32, (TN ? p.M : at.cnt) - m0));
      const long long first = TN ? (long long)at.e * p.M + m0 : (long long)at.lo + m0;
      void* out = TN && at.seg ? p.out2 : p.out;
      const bool mine = lane < rows;
      const int n0 = at.n0 + half * EPI_COLS;  // the warp's first column
      float w = 0.f;
      uint32_t s0[EPI == GROUPED_ACT_BWD ? 16 : 1], s1[EPI == GROUPED_ACT_BWD && GATED ? 16 : 1];
      auto fetch = [&](int c) {
        const int words = (p.N - n0 - c * 32) / 8;
        if (mine && words > 0) {
          const long long k = kept_at(p, first, rows, n0 / 32 + c, lane);
          kept(p.aux, k, rows, words, s0);
          if constexpr (GATED) kept(p.aux2, k, rows, words, s1);
        }
      };
      if constexpr (EPI == GROUPED_ACT_BWD) {
        // on their way while the products are; a chunk's while the one before is worked on
        if (mine) {
          const int q1 = p.order[first + lane];
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
      const uint32_t tbase = tmem + (uint32_t)(acc * ACC_COLS) + ((uint32_t)(q * 32) << 16) + (uint32_t)(half * EPI_COLS);
      auto read = [&](int col, uint32_t (&r)[32]) {
        if (!none) {
          tmem_ld32(tbase + col, r);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) r[j] = 0u;
        }
      };
      char* to = reinterpret_cast<char*>(out) + (first * p.N + n0) * (EPI == GROUPED_STORE && p.out_f32 ? 4 : 2);
      const int left = rows ? p.N - n0 : 0;  // columns to store
      if constexpr (EPI == GROUPED_STORE) {
        if (p.out_f32) {
#pragma unroll 1
          for (int c = 0; c < EPI_COLS && c < left; c += 32) {
            uint32_t r[32];
            read(c, r);
            const int words = min(8, (left - c) / 4);
            if (p.beta != 0.f) put_rows<8, true>(r, stage, to + c * 4, p.N * 4ll, rows, words, p.beta);
            else put_rows<8, false>(r, stage, to + c * 4, p.N * 4ll, rows, words, 0.f);
          }
        } else {
          constexpr int W = EPI_COLS < 64 ? EPI_COLS : 64;
#pragma unroll 1
          for (int c = 0; c < EPI_COLS && c < left; c += W) {
            uint32_t v[W / 2];
#pragma unroll
            for (int h = 0; h < W / 32; ++h) {
              uint32_t r[32];
              read(c + 32 * h, r);
#pragma unroll
              for (int j = 0; j < 16; ++j) v[16 * h + j] = pack_bf16(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
            }
            put_rows<W / 8, false>(v, stage, to + c * 2, p.N * 2ll, rows, min(W / 8, (left - c) / 8), 0.f);
          }
        }
      } else if constexpr (EPI == GROUPED_ACT) {
        constexpr int W = EPI_COLS < 64 ? EPI_COLS : 64;
#pragma unroll 1
        for (int c = 0; c < EPI_COLS && c < left; c += W) {
          uint32_t v[W / 2];
#pragma unroll
          for (int h = 0; h < W / 32; ++h) {
            uint32_t r[32], u[DUAL ? 32 : 1];
            read(c + 32 * h, r);
            if constexpr (DUAL) read(BN + c + 32 * h, u);
            const int words = (left - c) / 8 - 4 * h;
            if (p.out2 && mine && words > 0) {
              const long long k = kept_at(p, first, rows, (n0 + c) / 32 + h, lane);
              uint32_t t[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) t[j] = pack_bf16(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
              keep(p.out2, k, rows, words, t);
              if constexpr (DUAL) {
#pragma unroll
                for (int j = 0; j < 16; ++j) t[j] = pack_bf16(__uint_as_float(u[2 * j]), __uint_as_float(u[2 * j + 1]));
                keep(p.out3, k, rows, words, t);
              }
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const uint64_t z = f2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
              uint64_t y;
              if constexpr (DUAL) {
                const uint64_t up = f2(__uint_as_float(u[2 * j]), __uint_as_float(u[2 * j + 1]));
                // the gate first: a closed one is 0 whatever z up would be
                y = mul2(mul2(z, sigmoid_of(mul2(z, f2(-1.4426950408889634f, -1.4426950408889634f)))), up);
              } else {
                uint64_t slope;
                gelu2<ACT>(z, y, slope);
              }
              const float2 o = f2split(y);
              v[16 * h + j] = pack_bf16(o.x, o.y);
            }
          }
          put_rows<W / 8, false>(v, stage, to + c * 2, p.N * 2ll, rows, min(W / 8, (left - c) / 8), 0.f);
        }
      } else {
        // what was kept is bf16 (off by up to 2^-8 of its size): the activation
        // and its slopes are taken again from it in fp32 and rounded once
        const uint64_t w2 = f2(w, w);
        uint64_t dot2 = f2(0.f, 0.f);
#pragma unroll 1
        for (int c = 0; c < EPI_COLS && c < left; c += 32) {
          uint32_t r[32], v[16], dv[GATED ? 16 : 1], aw[16];
          read(c, r);
          const int words = min(4, (left - c) / 8);
          // columns past N are zeros in r and in what was kept; rows past the
          // group's end hold anything and are not stored
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const uint64_t a = f2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
            const uint64_t g = f2(bf16_lo(s0[j]), bf16_hi(s0[j]));
            const uint64_t wa = mul2(w2, a);
            uint64_t act, x;
            if constexpr (GATED) {
              const uint64_t u = f2(bf16_lo(s1[j]), bf16_hi(s1[j]));
              const uint64_t sg = sigmoid_of(mul2(g, f2(-1.4426950408889634f, -1.4426950408889634f)));
              const uint64_t si = mul2(g, sg);  // silu(g)
              act = mul2(si, u);
              x = mul2(wa, mul2(u, fma2(si, sub2(f2(1.f, 1.f), sg), sg)));  // the slope first, as above
              const float2 y = f2split(mul2(wa, si));
              dv[j] = pack_bf16(y.x, y.y);
            } else {
              uint64_t slope;
              gelu2<ACT>(g, act, slope);
              x = mul2(wa, slope);
            }
            dot2 = fma2(a, act, dot2);
            const float2 xs = f2split(x), zs = f2split(mul2(w2, act));
            v[j] = pack_bf16(xs.x, xs.y);
            aw[j] = pack_bf16(zs.x, zs.y);
          }
          if (c + 32 < EPI_COLS) fetch(c / 32 + 1);
          const long long ld = p.N * 2ll;
          put_rows<4, false>(v, stage, to + c * 2, ld, rows, words, 0.f);
          if constexpr (GATED)
            put_rows<4, false>(dv, stage, reinterpret_cast<char*>(p.out2) + (first * p.N + n0 + c) * 2, ld, rows, words, 0.f);
          put_rows<4, false>(aw, stage, reinterpret_cast<char*>(p.out3) + (first * p.N + n0 + c) * 2, ld, rows, words, 0.f);
        }
        // one sum per row and half tile, added in this order later
        const float2 dot = f2split(dot2);
        if (mine) p.part[(long long)(2 * (at.n0 / BN) + half) * p.rows + first + lane] = dot.x + dot.y;
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

template <int FORM, int EPI, int ACT, int BN, bool AG, bool BG, bool DUAL, bool PAIR>
int launch(Params& p, int64_t units, cudaStream_t st) {
  constexpr int SMEM = smem_bytes<BN, DUAL, PAIR>();
  auto kern = grouped_kernel<FORM, EPI, ACT, BN, AG, BG, DUAL, PAIR>;
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

// One translation unit per form (they compile in parallel); bn: columns a tile,
// pair: a pair of SMs a tile.
int launch_nt(Params& p, int epi, int act, bool gather, bool pair, int bn, int64_t units, cudaStream_t st);
int launch_nn(Params& p, int epi, int act, bool pair, int bn, int64_t units, cudaStream_t st);
int launch_tn(Params& p, bool a_gather, bool b_gather, bool pair, int64_t units, cudaStream_t st);

}  // namespace gg
}  // namespace bpt
