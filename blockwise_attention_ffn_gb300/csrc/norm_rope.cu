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
// statistics, angles' sines and sums are fp32, in packed pairs (the count of
// instructions, not memory, held back an unpacked version); each output is
// rounded once.
//
// Two forms.  With rows for every SM several times over, blocks stream tiles
// of whole rows through shared memory by bulk copies (32768 rows of 32 + 32 + 32
// heads of 64: 137 us, 87% of a copy's bandwidth; of 80: 155 us, 97%, backward 235 us,
// 85%; 65536 rows of 32 + 8 + 8 heads of 128: 258 us, 93%, backward 411 us, 83%; the
// rotation alone, in place, 215 us either way, 93%).  Fewer rows are read straight into registers, their
// heads spread over all warps (40 heads of 8 rows: one step of 80 warps).
//
// Angles: p * theta in turns, as a 64-bit fraction of a turn.  The product of
// the integer position with the frequency's fraction, modulo 2^64, is the
// angle reduced exactly, whatever the position; its upper 32 bits give the
// argument of one sincospi.  A row's d/2 angles are the same for all its
// heads: a block takes a few rows at a time and keeps their sines and cosines
// in shared memory.
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
#include "attn_common.cuh"
#include "internal.h"

namespace bpt {
namespace {

constexpr int NR_THREADS = 256;
constexpr int NR_WARPS = NR_THREADS / 32;
constexpr int NR_MAX_BLOCKS = 152 * 4;  // partials of the weight gradients
constexpr int NR_STAGED_TILES = 3;      // tiles per block from which the staged form is taken

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

// eight bf16 as four packed pairs of fp32, and back (times sc)
__device__ __forceinline__ void unpack8(uint4 v, uint64_t* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = f2(bf16_lo(w[i]), bf16_hi(w[i]));
}
__device__ __forceinline__ uint4 pack8(const uint64_t* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = f2split(f[i]);
    w[i] = pack_bf16(v.x, v.y);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ float sum2(uint64_t v) {
  const float2 s = f2split(v);
  return s.x + s.y;
}
constexpr uint64_t MINUS2 = 0x8000000080000000ull;  // sign bits of a packed pair

// One lane's 16 elements of one head: x (va, vb: halves) and, backward, dy
// (ya, yb); acc: the weight gradient's sums.  All lanes of the warp together.
template <int L, bool BWD>
__device__ __forceinline__ void head_math(uint4 va, uint4 vb, uint4 ya, uint4 yb, bool norm, float eps,
                                          const uint64_t (&cs)[4], const uint64_t (&sn)[4], const uint64_t (&wa)[4],
                                          const uint64_t (&wb)[4], uint64_t (&acc)[8], int base, int idx,
                                          uint64_t (&oa)[4], uint64_t (&ob)[4]) {
  constexpr int D = 16 * L;
  uint64_t a[4], b[4];
  unpack8(va, a);
  unpack8(vb, b);
  float r = 1.f;
  if (norm) {
    uint64_t s = 0ull;
#pragma unroll
    for (int i = 0; i < 4; ++i) s = fma2(a[i], a[i], fma2(b[i], b[i], s));
    r = rsqrtf(head_sum<L>(sum2(s), base, idx) * (1.f / D) + eps);
  }
  const uint64_t r2 = f2(r, r);
  if constexpr (!BWD) {
    if (norm) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = mul2(mul2(a[i], r2), wa[i]);
        b[i] = mul2(mul2(b[i], r2), wb[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      oa[i] = fma2(a[i], cs[i], mul2(b[i] ^ MINUS2, sn[i]));
      ob[i] = fma2(a[i], sn[i], mul2(b[i], cs[i]));
    }
  } else {
    uint64_t da[4], db[4];
    unpack8(ya, da);
    unpack8(yb, db);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      oa[i] = fma2(da[i], cs[i], mul2(db[i], sn[i]));
      ob[i] = fma2(db[i], cs[i], mul2(da[i] ^ MINUS2, sn[i]));
    }
    if (norm) {
      uint64_t s = 0ull;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = mul2(a[i], r2);  // n
        b[i] = mul2(b[i], r2);
        acc[i] = fma2(oa[i], a[i], acc[i]);
        acc[4 + i] = fma2(ob[i], b[i], acc[4 + i]);
        oa[i] = mul2(oa[i], wa[i]);  // g
        ob[i] = mul2(ob[i], wb[i]);
        s = fma2(oa[i], a[i], fma2(ob[i], b[i], s));
      }
      const float m = -head_sum<L>(sum2(s), base, idx) * (1.f / D);
      const uint64_t m2 = f2(m, m);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        oa[i] = mul2(r2, fma2(a[i], m2, oa[i]));
        ob[i] = mul2(r2, fma2(b[i], m2, ob[i]));
      }
    }
  }
}
// sines and cosines of `rows` rows from row0, the first one's index in its
// sequence being index0
__device__ __forceinline__ void angle_table(const NormRopeParams& p, int64_t row0, int index0, int rows, int half,
                                            float* cosines, float* sines) {
  for (int u = threadIdx.x; u < rows * half; u += blockDim.x) {
    const int r = u / half;
    const uint32_t index = (uint32_t)index0 + r;
    const int64_t pos = p.pos ? (int64_t)p.pos[row0 + r] : index < (uint32_t)p.s ? index : index % (uint32_t)p.s;
    const uint64_t turn = (uint64_t)pos * p.turn[u % half];
    sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &sines[u], &cosines[u]);
  }
}
// a row's eight angles of lane idx
__device__ __forceinline__ void load_angles(const float* cosines, const float* sines, int at, uint64_t (&cs)[4],
                                            uint64_t (&sn)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const ulonglong2 c = reinterpret_cast<const ulonglong2*>(cosines + at)[i];
    const ulonglong2 s = reinterpret_cast<const ulonglong2*>(sines + at)[i];
    cs[2 * i] = c.x;
    cs[2 * i + 1] = c.y;
    sn[2 * i] = s.x;
    sn[2 * i + 1] = s.y;
  }
}
// a block's sums of one weight's gradient, added over its slots in order
template <int L>
__device__ __forceinline__ void block_dw(const uint64_t (&acc)[8], float* red, float* part) {
  constexpr int HPW = 32 / L, D = 16 * L;
  const int lane = lane_id(), slot = lane / L, idx = lane % L;
  if (slot < HPW) {
    float* dst = red + (warp_id() * HPW + slot) * D;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      *reinterpret_cast<uint64_t*>(dst + 8 * idx + 2 * i) = acc[i];
      *reinterpret_cast<uint64_t*>(dst + D / 2 + 8 * idx + 2 * i) = acc[4 + i];
    }
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float s = 0.f;
    for (int k = 0; k < (int)blockDim.x / 32 * HPW; ++k) s += red[k * D + threadIdx.x];
    part[threadIdx.x] = s;
  }
  __syncthreads();
}

constexpr int NR_ROWS = 32;  // rows of a tile at most

// One section of the columns (the query heads, or the key heads): n heads
// from column col0.  A block takes tiles of `tile_rows` rows; the tile's
// (row, head) pairs in memory order go to its warps' slots in turn.
template <int L, bool BWD>
__device__ __forceinline__ void section(const NormRopeParams& p, int n, int col0, const __nv_bfloat16* w, int tile_rows,
                                        float* cosines, float* sines, uint64_t (&acc)[8]) {
  constexpr int HPW = 32 / L, D = 16 * L, HALF = 8 * L;
  constexpr int STEP = NR_WARPS * HPW;  // pairs of a block's step
  const int lane = lane_id();
  const int slot = lane / L, idx = lane % L, base = slot * L;
  const bool lane_on = slot < HPW;
  const int step_rows = STEP / n, step_heads = STEP % n;
  uint64_t wa[4], wb[4];
  if (w && lane_on) {
    unpack8(*reinterpret_cast<const uint4*>(w + 8 * idx), wa);
    unpack8(*reinterpret_cast<const uint4*>(w + HALF + 8 * idx), wb);
  }
  uint64_t cs[4], sn[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    cs[i] = f2(1.f, 1.f);
    sn[i] = 0ull;
  }
  for (int64_t row0 = (int64_t)blockIdx.x * tile_rows; row0 < p.rows; row0 += (int64_t)gridDim.x * tile_rows) {
    const int rows = (int)min((int64_t)tile_rows, p.rows - row0);
    const int pairs = rows * n;
    int f = warp_id() * HPW + slot;
    int row = f / n, head = f % n, angles_of = -1;
    // a step's loads are in flight while the one before is computed, the
    // first one's while the angles are
    bool on = lane_on && f < pairs;
    int64_t at = (row0 + row) * p.width + col0 + head * D + 8 * idx;
    uint4 xa, xb, ya, yb;
    auto fetch = [&]() {
      xa = xb = ya = yb = make_uint4(0u, 0u, 0u, 0u);  // a slot without a pair adds nothing
      if (on && (!BWD || w)) {
        xa = *reinterpret_cast<const uint4*>(p.x + at);
        xb = *reinterpret_cast<const uint4*>(p.x + at + HALF);
      }
      if (BWD && on) {
        ya = *reinterpret_cast<const uint4*>(p.dy + at);
        yb = *reinterpret_cast<const uint4*>(p.dy + at + HALF);
      }
    };
    fetch();
    if (p.rope) {
      __syncthreads();  // the tile before has been read
      angle_table(p, row0, (int)(row0 % p.s), rows, HALF, cosines, sines);
      __syncthreads();
    }
    // a warp's slots step together: the shuffles take all its lanes
    for (int f0 = warp_id() * HPW; f0 < pairs; f0 += STEP) {
      if (p.rope && on && row != angles_of) {
        angles_of = row;
        load_angles(cosines, sines, row * HALF + 8 * idx, cs, sn);
      }
      const uint4 va = xa, vb = xb, da = ya, db = yb;
      const bool on_now = on;
      const int64_t at_now = at;
      f += STEP;
      row += step_rows;
      head += step_heads;
      if (head >= n) {
        head -= n;
        ++row;
      }
      on = lane_on && f < pairs;
      at = (row0 + row) * p.width + col0 + head * D + 8 * idx;
      fetch();
      uint64_t oa[4], ob[4];
      head_math<L, BWD>(va, vb, da, db, w != nullptr, p.eps, cs, sn, wa, wb, acc, base, idx, oa, ob);
      if (on_now) {
        *reinterpret_cast<uint4*>(p.out + at_now) = pack8(oa);
        *reinterpret_cast<uint4*>(p.out + at_now + HALF) = pack8(ob);
      }
    }
  }
}

// rows of a tile: eight steps of every warp, but no more than leaves every
// block a tile
__device__ __forceinline__ int tile_rows_for(int64_t rows, int n, int hpw) {
  const int want = (8 * NR_WARPS * hpw + n - 1) / n;
  const int64_t share = (rows + gridDim.x - 1) / gridDim.x;
  return (int)min(share, (int64_t)min(want, NR_ROWS));
}

template <int L, bool BWD>
__global__ void __launch_bounds__(NR_THREADS, BWD ? 2 : 3) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int HPW = 32 / L;
  constexpr int D = 16 * L;
  __shared__ __align__(16) float cosines[NR_ROWS * D / 2];
  __shared__ __align__(16) float sines[NR_ROWS * D / 2];
  __shared__ __align__(8) float red[BWD ? NR_WARPS * HPW * D : 1];
#pragma unroll 1
  for (int sec = 0; sec < 2; ++sec) {
    const int n = sec ? p.K : p.H;
    uint64_t acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0ull;
    section<L, BWD>(p, n, sec ? p.H * D : 0, sec ? p.wk : p.wq, tile_rows_for(p.rows, n, HPW), cosines, sines, acc);
    if constexpr (BWD) {
      if (p.part) block_dw<L>(acc, red, p.part + ((int64_t)blockIdx.x * 2 + sec) * D);
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

// The staged form, for more rows than the SMs take at once: a block streams
// tiles of whole rows through a ring of stages in shared memory by bulk
// copies, computes them in place and stores them by bulk copies, so that tens
// of KB are in flight per SM whatever the warps do, and V's columns pass
// through without a register.  Backward a stage holds the rows of dy, computed
// in place, and the query and key columns of x.
constexpr int NR_STAGES = 2;
struct Stages {
  int rows;                  // rows of a stage; 0: not even one fits
  int y_bytes, x_bytes;      // of a row: of dy (x forward), and backward of x
  uint32_t part_q, part_k;   // ceil(2^22 / heads): f * part >> 22 = f / heads, as f * heads < 2^22
};
template <int L, bool BWD>
__global__ void __launch_bounds__(NR_THREADS, 2) norm_rope_staged_kernel(const __grid_constant__ NormRopeParams p,
                                                                         const __grid_constant__ Stages g,
                                                                         unsigned int* err) {
  constexpr int HPW = 32 / L, D = 16 * L, HALF = 8 * L;
  extern __shared__ __align__(128) uint8_t smem[];
  const int stage_bytes = g.rows * (g.y_bytes + g.x_bytes);
  float* cosines = reinterpret_cast<float*>(smem + NR_STAGES * stage_bytes);
  float* sines = cosines + g.rows * HALF;
  float* weights = sines + g.rows * HALF;  // wq, wk in fp32
  __shared__ __align__(8) uint64_t full[NR_STAGES];
  __shared__ int abort_flag;
  const int lane = lane_id(), slot = lane / L, idx = lane % L, base = slot * L;
  const bool lane_on = slot < HPW;
  const bool norm = p.wq != nullptr;
  const __nv_bfloat16* in = BWD ? p.dy : p.x;
  const int64_t tiles = (p.rows + g.rows - 1) / g.rows;
  auto tile_of = [&](int k) { return (int64_t)blockIdx.x + (int64_t)k * gridDim.x; };
  auto load = [&](int k) {  // one thread
    const int64_t row0 = tile_of(k) * g.rows;
    if (row0 >= p.rows) return;
    const int rows = (int)min((int64_t)g.rows, p.rows - row0);
    uint8_t* y = smem + (k % NR_STAGES) * stage_bytes;
    uint8_t* x = y + g.rows * g.y_bytes;
    uint64_t* bar = &full[k % NR_STAGES];
    mbar_expect_tx(bar, rows * (g.y_bytes + g.x_bytes));
    for (int r = 0; r < rows; ++r) {
      bulk_load(y + r * g.y_bytes, in + (row0 + r) * p.width, g.y_bytes, bar);
      if (BWD && g.x_bytes) bulk_load(x + r * g.x_bytes, p.x + (row0 + r) * p.width, g.x_bytes, bar);
    }
  };
  if (threadIdx.x == 0) {
    for (int i = 0; i < NR_STAGES; ++i) mbar_init(&full[i], 1);
    abort_flag = 0;
    fence_mbar_init();
    for (int k = 0; k < NR_STAGES; ++k) load(k);
  }
  if (norm)
    for (int i = threadIdx.x; i < 2 * D; i += NR_THREADS)
      weights[i] = __bfloat162float(i < D ? p.wq[i] : p.wk[i - D]);
  __syncthreads();
  uint64_t accq[8], acck[8], cs[4], sn[4];
#pragma unroll
  for (int i = 0; i < 8; ++i) accq[i] = acck[i] = 0ull;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    cs[i] = f2(1.f, 1.f);
    sn[i] = 0ull;
  }
  bool ok = true;
  // a tile's first row's index in its sequence
  uint32_t index0 = (uint32_t)((int64_t)blockIdx.x * g.rows % p.s);
  const uint32_t index_step = (uint32_t)((int64_t)gridDim.x * g.rows % p.s);
  for (int k = 0; tile_of(k) < tiles; ++k) {
    const int64_t row0 = tile_of(k) * g.rows;
    const int rows = (int)min((int64_t)g.rows, p.rows - row0);
    if (p.rope) angle_table(p, row0, index0, rows, HALF, cosines, sines);
    index0 += index_step;
    if (index0 >= (uint32_t)p.s) index0 -= p.s;
    ok = bounded_wait(&full[k % NR_STAGES], (k / NR_STAGES) & 1, &abort_flag, 960, err);
    ok = __syncthreads_and(ok);
    if (!ok) break;
    uint8_t* y = smem + (k % NR_STAGES) * stage_bytes;
    const uint8_t* x = BWD ? y + g.rows * g.y_bytes : y;
    const int x_stride = BWD ? g.x_bytes : g.y_bytes;
#pragma unroll 1
    for (int sec = 0; sec < 2; ++sec) {
      const int n = sec ? p.K : p.H, col0 = sec ? p.H * D : 0;
      const int pairs = rows * n;
      // Between the sections the stage before this one has been stored, and
      // its next tile still has half of this one's time to arrive (loaded at
      // this tile's end: backward of 32 + 32 + 32 heads of 80 285 us against 249; a
      // check inside the loop below costs more than a better moment gains).
      if (sec == 1 && k > 0 && threadIdx.x == 0) {
        bulk_wait_read0();
        load(k - 1 + NR_STAGES);
      }
      uint64_t wa[4], wb[4];
      if (norm && lane_on) {
        const float* w = weights + sec * D + 8 * idx;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          wa[i] = reinterpret_cast<const uint64_t*>(w)[i];
          wb[i] = reinterpret_cast<const uint64_t*>(w + HALF)[i];
        }
      }
      // the key heads start at the warps that the query heads left idle last
      const int first = sec ? (warp_id() + NR_WARPS - (rows * p.H + HPW - 1) / HPW % NR_WARPS) % NR_WARPS : warp_id();
      for (int f0 = first * HPW; f0 < pairs; f0 += NR_WARPS * HPW) {
        const int f = f0 + slot;
        const bool on = lane_on && f < pairs;
        const int row = on ? (int)((uint32_t)f * (sec ? g.part_k : g.part_q) >> 22) : 0, head = on ? f - row * n : 0;
        const int at = (col0 + head * D + 8 * idx) * 2;
        uint4 va = make_uint4(0u, 0u, 0u, 0u), vb = va, ya = va, yb = va;
        if (on && (!BWD || norm)) {
          va = *reinterpret_cast<const uint4*>(x + row * x_stride + at);
          vb = *reinterpret_cast<const uint4*>(x + row * x_stride + at + 2 * HALF);
        }
        uint8_t* yrow = y + row * g.y_bytes + at;
        if (BWD && on) {
          ya = *reinterpret_cast<const uint4*>(yrow);
          yb = *reinterpret_cast<const uint4*>(yrow + 2 * HALF);
        }
        if (p.rope && on) load_angles(cosines, sines, row * HALF + 8 * idx, cs, sn);
        uint64_t oa[4], ob[4];
        if (sec == 0) head_math<L, BWD>(va, vb, ya, yb, norm, p.eps, cs, sn, wa, wb, accq, base, idx, oa, ob);
        else head_math<L, BWD>(va, vb, ya, yb, norm, p.eps, cs, sn, wa, wb, acck, base, idx, oa, ob);
        if (on) {
          *reinterpret_cast<uint4*>(yrow) = pack8(oa);
          *reinterpret_cast<uint4*>(yrow + 2 * HALF) = pack8(ob);
        }
      }
    }
    fence_proxy_async_smem();
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int r = 0; r < rows; ++r) bulk_store(p.out + (row0 + r) * p.width, y + r * g.y_bytes, g.y_bytes);
      bulk_commit();
    }
  }
  if (threadIdx.x == 0) {
    bulk_wait0();
    if (!ok) {
      // loads in flight land before the shared memory goes
      for (int i = 0; i < NR_STAGES; ++i) {
        drain_wait(&full[i], 0);
        drain_wait(&full[i], 1);
      }
    }
  }
  __syncthreads();
  if constexpr (BWD) {
    if (p.part) {
      float* red = reinterpret_cast<float*>(smem);
      block_dw<L>(accq, red, p.part + (int64_t)blockIdx.x * 2 * D);
      block_dw<L>(acck, red, p.part + ((int64_t)blockIdx.x * 2 + 1) * D);
    }
    let_next_start();
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

template <int L, bool BWD>
int launch_direct(const NormRopeParams& p, int blocks, cudaStream_t st) {
  norm_rope_kernel<L, BWD><<<blocks, NR_THREADS, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? BPT_OK : BPT_ECUDA;
}
template <int L, bool BWD>
int launch_staged(const NormRopeParams& p, const Stages& g, int blocks, int smem, cudaStream_t st) {
  static std::atomic<uint64_t> attr{0};  // devices whose limit is set
  if (smem_limit_once(reinterpret_cast<const void*>(norm_rope_staged_kernel<L, BWD>), 116 * 1024, &attr))
    return BPT_ECUDA;
  unsigned int* err = device_error_word();
  if (!err) return BPT_ECUDA;
  norm_rope_staged_kernel<L, BWD><<<blocks, NR_THREADS, smem, st>>>(p, g, err);
  return cudaGetLastError() == cudaSuccess ? BPT_OK : BPT_ECUDA;
}

// The stages for rows of these sizes, two blocks per SM: two of up to 56 KB.
// Smaller ones leave warps without a head at every stage's end (forward, three
// of 36 KB, when the choice was made: 32768 rows of 32 + 32 + 32 heads of 80 189 us
// against 162, of 64 125 us against 130); three blocks of two of 37 KB, 85 registers a thread, are no faster
// where rows are long (heads of 128, same time: 259 us against 244).
Stages stages_for(const PackedDims& D, int y_bytes, int x_bytes, int* smem) {
  const int table = (int)(2 * D.d * 4);            // weights
  const int angles = (int)(D.d / 2 * 2 * 4);       // of one row
  const int row = y_bytes + x_bytes;
  const int rows = std::min((112 * 1024 - table) / (NR_STAGES * row + angles), std::max(1, 56 * 1024 / row));
  const auto part = [](int64_t n) { return (uint32_t)(((1 << 22) + n - 1) / n); };
  // (a tile has fewer than 1024 heads of either kind, and f * part stays below 2^32)
  const Stages g{std::min(rows, NR_ROWS), y_bytes, x_bytes, part(D.H), part(D.Hkv)};
  // a block's weight gradient sums take the stages' place at the end
  const int sums = NR_WARPS * (32 / (int)(D.d / 16)) * (int)D.d * 4;
  *smem = std::max(NR_STAGES * g.rows * row, sums) + g.rows * angles + table;
  return g;
}

// Launches one direction; *blocks: how many blocks' partials the backward left.
template <bool BWD>
int launch(const NormRopeParams& p, const PackedDims& D, int* blocks, cudaStream_t st) {
  const int nsm = sm_count();
  if (nsm <= 0) return BPT_ECUDA;
  const int heads = (int)((D.H + D.Hkv) * D.d * 2);
  const int y_bytes = p.copy_v ? (int)(D.width * 2) : heads, x_bytes = BWD && p.wq ? heads : 0;
  int smem = 0;
  const Stages g = D.width * 2 <= 112 * 1024 ? stages_for(D, y_bytes, x_bytes, &smem) : Stages{0, 0, 0, 0, 0};
  const bool staged = g.rows && D.rows >= (int64_t)nsm * 2 * g.rows * NR_STAGED_TILES;
  const int hpw = 32 / (int)(D.d / 16);
  if (staged) {
    *blocks = nsm * 2;
  } else {
    // enough for one step of every warp, at most what the SMs hold
    const int64_t want = (D.rows * D.H + (int64_t)hpw * NR_WARPS - 1) / ((int64_t)hpw * NR_WARPS);
    *blocks = (int)std::min<int64_t>(want, (int64_t)nsm * (BWD ? 2 : 3));
  }
  *blocks = std::min(*blocks, NR_MAX_BLOCKS);
  switch (p.d) {
    case 64: return staged ? launch_staged<4, BWD>(p, g, *blocks, smem, st) : launch_direct<4, BWD>(p, *blocks, st);
    case 80: return staged ? launch_staged<5, BWD>(p, g, *blocks, smem, st) : launch_direct<5, BWD>(p, *blocks, st);
    case 96: return staged ? launch_staged<6, BWD>(p, g, *blocks, smem, st) : launch_direct<6, BWD>(p, *blocks, st);
    case 112: return staged ? launch_staged<7, BWD>(p, g, *blocks, smem, st) : launch_direct<7, BWD>(p, *blocks, st);
    case 128: return staged ? launch_staged<8, BWD>(p, g, *blocks, smem, st) : launch_direct<8, BWD>(p, *blocks, st);
    default: return BPT_EUNSUPPORTED;
  }
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
  const Span sp[] = {{wq, wq ? D.d * 2 : 0}, {wk, wk ? D.d * 2 : 0}, {positions, positions ? D.rows * 4 : 0},
                     {qkv, bytes}, {out, bytes}};
  if (overlaps(sp[4], sp, 3)) return BPT_EINVAL;
  if (D.debug && debug_spans(sp, 5)) return BPT_EINVAL;
  NormRopeParams p;
  fill(cfg, D, wq, wk, positions, &p);
  p.x = reinterpret_cast<const __nv_bfloat16*>(qkv);
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.copy_v = qkv != out;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int blocks = 0;
  {
    ProfScope prof(PROF_NORM, 0.0, 2.0 * (p.copy_v ? bytes : bytes - D.rows * D.Hkv * D.d * 2), st);
    rc = launch<false>(p, D, &blocks, st);
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
  const int64_t dw = wq ? D.d * 4 : 0;
  const Span sp[] = {{wq, dw / 2}, {wk, dw / 2}, {positions, positions ? D.rows * 4 : 0}, {dqkv, bytes}, {dout, bytes},
                     {wq ? qkv : nullptr, wq ? bytes : 0}, {wq ? dwq : nullptr, dw}, {wq ? dwk : nullptr, dw},
                     {wq ? ws : nullptr, wq ? (int64_t)ws_need(D) : 0}};
  // (dqkv may be dout)
  if (overlaps(sp[3], sp, 3)) return BPT_EINVAL;
  for (int i = 6; wq && i < 9; ++i)
    if (overlaps(sp[i], sp, i)) return BPT_EINVAL;
  if (D.debug && debug_spans(sp, 9)) return BPT_EINVAL;
  NormRopeParams p;
  fill(cfg, D, wq, wk, positions, &p);
  p.x = reinterpret_cast<const __nv_bfloat16*>(qkv);
  p.dy = reinterpret_cast<const __nv_bfloat16*>(dout);
  p.out = reinterpret_cast<__nv_bfloat16*>(dqkv);
  p.part = wq ? reinterpret_cast<float*>(ws) : nullptr;
  p.copy_v = dout != dqkv;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int blocks = 0;
  {
    const double v = (double)D.rows * D.Hkv * D.d * 2;
    ProfScope prof(PROF_NORM, 0.0, (wq ? 3.0 : 2.0) * (bytes - v) + (p.copy_v ? 2 * v : 0.0), st);
    rc = launch<true>(p, D, &blocks, st);
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
