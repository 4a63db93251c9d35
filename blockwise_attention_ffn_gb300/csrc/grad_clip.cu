// grad_clip.cu -- the global norm of a list of gradients, and clipping by it.
//
//   norm = sqrt(sum over tensors and elements of g^2)
//   out  = g * min(1, max_norm / (norm + 1e-6))
//
// HBM-bound: every gradient is read once for the norm and, since no element
// can be scaled before the last one is summed, once more for the scaled copy;
// only what the L2 still holds of the first reading is not read twice.  So the
// second pass walks the chunks backwards, starting with those read last, and
// its stores are marked evict-first.  Measured on a GB300: 537 MB of fp32
// gradients in 91 us for the norm (5.9 TB/s) and 163 us for the scaled copy
// (6.2 TB/s of traffic, 93% of a plain copy's); a layer's 436 MB in bf16 take
// 213 us, 1.1 times three transfers of it (the second pass finds 9% of it in L2);
// sixteen tensors of a small layer 24 us, of which the two launches and the host's
// call are nearly all.  An output that lies differently against 16 bytes than its
// gradient goes element by element: 134 million of them take 652 us in fp32 (258
// where they lie alike), 540 us in bf16 (136).
//
// Two launches.  The tensors' addresses and sizes travel in the kernels'
// parameters (no copy to the device, so a captured call replays by itself).
// A gradient is cut into chunks of 32 KB, which the blocks take in turn.
// Sums: 32 squares (bf16: 64) in fp32, then fp64, per block one fp64 partial; every block
// of the second launch adds the partials in the same order, so the norm has a
// fixed summation order and no atomics.  A group of squares that leaves
// fp32's range is summed again from values scaled by a power of two, so the
// norm neither overflows nor vanishes before its own fp32 value does.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <string.h>

#include <algorithm>
#include <vector>

#include "../../include/bpt.h"
#include "internal.h"
#include "ptx.cuh"

namespace bpt {
namespace {

constexpr int CLIP_THREADS = 256;
constexpr int CHUNK_BYTES = 32768;
constexpr int MAX_BLOCKS = 152 * 8;  // partial sums in the workspace

struct ClipEntry {
  const void* g;
  void* out;
  int64_t n_dtype;  // elements, times two, plus 1 for bf16
};
template <int N>
struct ClipTable {
  ClipEntry e[N];
  int first[N + 1];  // first chunk of each tensor; first[count] = chunks in all
  int count;
};

__device__ __forceinline__ uint4 load16(const void* p) {
  return __ldg(reinterpret_cast<const uint4*>(p));
}
__device__ __forceinline__ void store16_stream(void* p, uint4 v) {
  asm volatile("st.global.cs.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ float lo16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi16(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// sum of squares of a 16-byte unit scaled by sc (four fp32 or eight bf16)
__device__ __forceinline__ float unit_squares(uint4 v, bool bf16, float sc) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (bf16) {
      const float a = lo16(w[i]) * sc, b = hi16(w[i]) * sc;
      s = fmaf(a, a, s);
      s = fmaf(b, b, s);
    } else {
      const float a = __uint_as_float(w[i]) * sc;
      s = fmaf(a, a, s);
    }
  }
  return s;
}

constexpr int UNITS = CHUNK_BYTES / 16 / CLIP_THREADS;  // 16-byte units per thread and chunk

// squares of UNITS units: fp32, or again from scaled values where the fp32
// sum is near either end of its range (also inf and NaN, which stay so)
__device__ __forceinline__ double squares(const uint4 (&v)[UNITS], bool bf16) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < UNITS; ++i) s += unit_squares(v[i], bf16, 1.f);
  if (s > 1e-25f && s < 1e30f) return (double)s;
  const bool small = s <= 1e-25f;
  const float sc = small ? 0x1p96f : 0x1p-64f;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < UNITS; ++i) s += unit_squares(v[i], bf16, sc);
  return (double)s * (small ? 0x1p-192 : 0x1p128);
}

// one element's bits in the low (bf16) or whole word, for the ragged ends
__device__ __forceinline__ uint32_t load_one(const void* p, int64_t i, bool bf16) {
  return bf16 ? (uint32_t) reinterpret_cast<const uint16_t*>(p)[i] : reinterpret_cast<const uint32_t*>(p)[i];
}

struct Chunk {
  const uint8_t* g;
  uint8_t* out;
  int64_t n;  // elements
  bool bf16;
};
template <int N>
__device__ __forceinline__ Chunk chunk_of(const ClipTable<N>& t, int c) {
  int a = 0, b = t.count;  // first[a] <= c < first[b]
  while (b - a > 1) {
    const int m = (a + b) >> 1;
    if (t.first[m] <= c) a = m;
    else b = m;
  }
  const ClipEntry& e = t.e[a];
  Chunk k;
  k.bf16 = e.n_dtype & 1;
  const int64_t per = k.bf16 ? CHUNK_BYTES / 2 : CHUNK_BYTES / 4;
  const int64_t at = (int64_t)(c - t.first[a]) * per;
  k.n = min(per, (e.n_dtype >> 1) - at);
  const int64_t byte = at * (k.bf16 ? 2 : 4);
  k.g = reinterpret_cast<const uint8_t*>(e.g) + byte;
  k.out = reinterpret_cast<uint8_t*>(e.out) + byte;
  return k;
}
// elements before the first 16-byte boundary of p (at most n)
__device__ __forceinline__ int64_t head_of(const void* p, int64_t n, int size) {
  const int64_t h = ((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / size;
  return h < n ? h : n;
}

template <int N>
__global__ void __launch_bounds__(CLIP_THREADS) clip_norm_kernel(const __grid_constant__ ClipTable<N> t, double* part,
                                                                 int add) {
  double acc = 0.0;
  const int total = t.first[t.count];
  for (int c = blockIdx.x; c < total; c += gridDim.x) {
    const Chunk k = chunk_of(t, c);
    const int size = k.bf16 ? 2 : 4;
    const int64_t head = head_of(k.g, k.n, size);
    const int64_t units = (k.n - head) * size / 16;
    const uint8_t* body = k.g + head * size;
    uint4 v[UNITS];
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      const int64_t u = threadIdx.x + i * CLIP_THREADS;
      v[i] = u < units ? load16(body + u * 16) : make_uint4(0u, 0u, 0u, 0u);
    }
    acc += squares(v, k.bf16);
    // at most 7 elements before and 7 after the whole units
    const int64_t ntail = k.n - head - units * 16 / size;
    if (threadIdx.x < head + ntail) {
      const int64_t i = threadIdx.x < head ? threadIdx.x : k.n - ntail + (threadIdx.x - head);
      uint4 w[UNITS];
#pragma unroll
      for (int j = 0; j < UNITS; ++j) w[j] = make_uint4(0u, 0u, 0u, 0u);
      w[0].x = load_one(k.g, i, k.bf16);
      acc += squares(w, k.bf16);
    }
  }
  let_next_start();
  __shared__ double red[CLIP_THREADS / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < CLIP_THREADS / 32; ++i) s += red[i];
    part[blockIdx.x] = add ? part[blockIdx.x] + s : s;
  }
}

template <int N>
__global__ void __launch_bounds__(CLIP_THREADS) clip_scale_kernel(const __grid_constant__ ClipTable<N> t,
                                                                  const double* part, int nparts, float max_norm,
                                                                  float* norm_out) {
  __shared__ double red[CLIP_THREADS / 32];
  wait_for_previous();
  double acc = 0.0;
  for (int i = threadIdx.x; i < nparts; i += CLIP_THREADS) acc += part[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = acc;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < CLIP_THREADS / 32; ++i) s += red[i];
  const float norm = (float)sqrt(s);
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
  float coef = max_norm / (norm + 1e-6f);
  // under a finite max_norm a NaN norm makes every output NaN
  if (coef > 1.f || max_norm == INFINITY) coef = 1.f;

  const int total = t.first[t.count];
  for (int c = total - 1 - (int)blockIdx.x; c >= 0; c -= gridDim.x) {
    const Chunk k = chunk_of(t, c);
    if (coef == 1.f && k.g == k.out) continue;  // in place and not clipped
    const int size = k.bf16 ? 2 : 4;
    const bool together = ((reinterpret_cast<uintptr_t>(k.g) ^ reinterpret_cast<uintptr_t>(k.out)) & 15) == 0;
    const int64_t head = together ? head_of(k.g, k.n, size) : k.n;
    const int64_t units = (k.n - head) * size / 16;
    const uint8_t* body = k.g + head * size;
    uint8_t* obody = k.out + head * size;
    uint4 v[UNITS];
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      const int64_t u = threadIdx.x + i * CLIP_THREADS;
      if (u < units) v[i] = load16(body + u * 16);
    }
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      const int64_t u = threadIdx.x + i * CLIP_THREADS;
      if (u >= units) continue;
      uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (k.bf16) {
          const __nv_bfloat162 r = __floats2bfloat162_rn(lo16(w[j]) * coef, hi16(w[j]) * coef);
          w[j] = *reinterpret_cast<const uint32_t*>(&r);
        } else {
          w[j] = __float_as_uint(__uint_as_float(w[j]) * coef);
        }
      }
      store16_stream(obody + u * 16, make_uint4(w[0], w[1], w[2], w[3]));
    }
    // the ends, or every element of a chunk whose input and output lie
    // differently against the 16-byte boundaries
    const int64_t body_end = head + units * 16 / size;
    const int64_t ends = k.n - units * 16 / size;
    for (int64_t j = threadIdx.x; j < ends; j += CLIP_THREADS) {
      const int64_t i = j < head ? j : body_end + (j - head);
      if (k.bf16) {
        const float x = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(k.g)[i]);
        reinterpret_cast<__nv_bfloat16*>(k.out)[i] = __float2bfloat16(x * coef);
      } else {
        reinterpret_cast<float*>(k.out)[i] = reinterpret_cast<const float*>(k.g)[i] * coef;
      }
    }
  }
}

// Tensors [at, at + count) as a table; false if their chunks pass 2^31 - 1.
template <int N>
bool fill(ClipTable<N>* tb, const bpt_clip_tensor* t, int at, int count) {
  int64_t chunks = 0;
  tb->count = count;
  for (int i = 0; i < count; ++i) {
    const bpt_clip_tensor& x = t[at + i];
    const bool bf16 = x.dtype == BPT_DTYPE_BF16;
    tb->e[i] = ClipEntry{x.grad, x.out, x.numel * 2 + (bf16 ? 1 : 0)};
    tb->first[i] = (int)chunks;
    chunks += (x.numel * (bf16 ? 2 : 4) + CHUNK_BYTES - 1) / CHUNK_BYTES;
    if (chunks > INT32_MAX - MAX_BLOCKS) return false;
  }
  tb->first[count] = (int)chunks;
  return true;
}

template <int N>
int clip_launches(int n, const bpt_clip_tensor* t, float max_norm, float* norm, double* part, cudaStream_t st) {
  const int nsm = sm_count();
  if (nsm <= 0) return BPT_ECUDA;
  const int cap = std::min(nsm * 8, MAX_BLOCKS);
  ClipTable<N> tb;
  int nparts = 1;
  double bytes = 0;
  for (int i = 0; i < n; ++i) bytes += (double)t[i].numel * (t[i].dtype == BPT_DTYPE_BF16 ? 2 : 4);
  for (int pass = 0; pass < 2; ++pass) {
    ProfScope prof(PROF_MISC, 0.0, (pass ? 2 : 1) * bytes, st);
    // the scaling pass goes through the tables backwards too
    const int tables = std::max(1, (n + N - 1) / N);
    for (int k = 0; k < tables; ++k) {
      const int at = (pass ? tables - 1 - k : k) * N;
      if (!fill(&tb, t, at, std::min(N, n - at))) return BPT_EUNSUPPORTED;
      const int chunks = tb.first[tb.count];
      if (pass == 0) {
        // later tables add to the first one's partials, block by block
        const int grid = k ? nparts : std::max(1, std::min(cap, tables > 1 ? cap : chunks));
        nparts = grid;
        clip_norm_kernel<N><<<grid, CLIP_THREADS, 0, st>>>(tb, part, k);
      } else {
        // (of the last norm kernel; a later table's is an ordinary launch)
        const int grid = std::max(1, std::min(cap, chunks));
        float* out = k == 0 ? norm : nullptr;
        if (k == 0) {
          if (launch_dependent(clip_scale_kernel<N>, grid, 1, dim3(CLIP_THREADS), 0, st, tb, (const double*)part, nparts,
                               max_norm, out) != cudaSuccess)
            return BPT_ECUDA;
        } else {
          clip_scale_kernel<N><<<grid, CLIP_THREADS, 0, st>>>(tb, part, nparts, max_norm, out);
        }
      }
      if (cudaGetLastError() != cudaSuccess) return BPT_ECUDA;
    }
  }
  return BPT_OK;
}

// true if some output's bytes (norm and ws among them) are also another
// tensor's input or output (a tensor's own input may be its output)
bool overlapping(int n, const bpt_clip_tensor* t, const void* norm, const void* ws) {
  struct Range {
    uintptr_t lo, hi;
    bool out;
  };
  std::vector<Range> r;
  r.reserve(2 * (size_t)n + 2);
  const uintptr_t pn = reinterpret_cast<uintptr_t>(norm), pw = reinterpret_cast<uintptr_t>(ws);
  r.push_back(Range{pn, pn + sizeof(float), true});
  r.push_back(Range{pw, pw + bpt_clip_workspace_bytes(), true});
  for (int i = 0; i < n; ++i) {
    const uintptr_t bytes = (uintptr_t)t[i].numel * (t[i].dtype == BPT_DTYPE_BF16 ? 2 : 4);
    if (!bytes) continue;
    const uintptr_t o = reinterpret_cast<uintptr_t>(t[i].out), g = reinterpret_cast<uintptr_t>(t[i].grad);
    r.push_back(Range{o, o + bytes, true});
    if (g != o) r.push_back(Range{g, g + bytes, false});
  }
  std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
  uintptr_t out_end = 0, any_end = 0;
  for (const Range& x : r) {
    if (x.lo < out_end || (x.out && x.lo < any_end)) return true;
    any_end = std::max(any_end, x.hi);
    if (x.out) out_end = std::max(out_end, x.hi);
  }
  return false;
}

}  // namespace
}  // namespace bpt

using namespace bpt;

extern "C" {

size_t bpt_clip_workspace_bytes(void) { return MAX_BLOCKS * sizeof(double); }

int bpt_clip_grads(int32_t n, const bpt_clip_tensor* t, float max_norm, int32_t flags, float* norm, void* ws,
                   size_t ws_bytes, void* stream) {
  if (n < 0 || (n > 0 && !t) || !norm || !ws) return BPT_EINVAL;
  if (!(max_norm > 0.f)) return BPT_EINVAL;
  if (flags & ~BPT_FLAG_DEBUG_CHECKS) return BPT_EINVAL;
  if ((reinterpret_cast<uintptr_t>(norm) & 3) || (reinterpret_cast<uintptr_t>(ws) & 15)) return BPT_EINVAL;
  for (int i = 0; i < n; ++i) {
    if (t[i].dtype != BPT_DTYPE_F32 && t[i].dtype != BPT_DTYPE_BF16) return BPT_EINVAL;
    if (t[i].numel < 0 || t[i].numel > (INT64_MAX >> 4)) return BPT_EINVAL;
    if (t[i].numel == 0) continue;
    const uintptr_t mask = t[i].dtype == BPT_DTYPE_BF16 ? 1 : 3;
    if (!t[i].grad || !t[i].out) return BPT_EINVAL;
    if ((reinterpret_cast<uintptr_t>(t[i].grad) & mask) || (reinterpret_cast<uintptr_t>(t[i].out) & mask))
      return BPT_EINVAL;
  }
  if (ws_bytes < bpt_clip_workspace_bytes()) return BPT_ENOSPC;
  try {
    if (overlapping(n, t, norm, ws)) return BPT_EINVAL;
  } catch (...) {  // no host memory for the check
    return BPT_EUNSUPPORTED;
  }
  const bool debug = (flags & BPT_FLAG_DEBUG_CHECKS) != 0;
  if (debug) {
    const Span own[] = {{norm, 4}, {ws, (int64_t)bpt_clip_workspace_bytes()}};
    if (debug_spans(own, 2)) return BPT_EINVAL;
    for (int i = 0; i < n; ++i) {
      const int64_t bytes = t[i].numel * (t[i].dtype == BPT_DTYPE_BF16 ? 2 : 4);
      const Span sp[] = {{t[i].grad, bytes}, {t[i].out, bytes}};
      if (debug_spans(sp, 2)) return BPT_EINVAL;
    }
  }
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  double* part = reinterpret_cast<double*>(ws);
  // the table is a kernel parameter: a short one costs a launch less
  const int rc = n <= 64 ? clip_launches<64>(n, t, max_norm, norm, part, st)
                         : clip_launches<1000>(n, t, max_norm, norm, part, st);
  if (rc) return rc;
  return debug ? debug_finish(st) : BPT_OK;
}

}  // extern "C"
