// moe.h -- the checked shape of a mixture-of-experts layer, shared by the
// router (moe_route.cu) and the experts' network (moe_ffn.cu).
#pragma once

#include "../../include/bpt.h"
#include "internal.h"

namespace bpt {

struct MoeDims {
  int64_t n, h, f, E, k, pairs;  // pairs = n k
  int act;
  int logit_bytes, weight_bytes;
  bool grads_f32, debug, accum;
};
// 0 or a BPT_* status
int moe_dims(const bpt_moe_config* cfg, MoeDims* out);

// Whether the offsets lo, hi of a group of `rows` rows in all fall or leave
// them.  Where none do, the groups hold [offsets[0], offsets[E]) between them.
__device__ __forceinline__ bool bad_offsets(int lo, int hi, int64_t rows) { return lo < 0 || hi < lo || hi > rows; }
// The group that row r is of (E: none), as the grouped GEMM lays them out where
// some offsets are bad: those groups hold nothing, nor do those that start
// before an earlier one's end.
static __device__ __noinline__ int group_of(const int32_t* offsets, int E, int64_t rows, int r) {
  int end = 0;
  for (int e = 0; e < E; ++e) {
    const int lo = offsets[e], hi = offsets[e + 1];
    if (bad_offsets(lo, hi, rows)) continue;
    if (lo >= end && r >= lo && r < hi) return e;
    end = max(end, hi);
  }
  return E;
}

// The forward for so few rows that an expert's matrices meet about one
// (moe_few.cu): whether they are, its workspace, its launches.
bool moe_few_rows(const MoeDims& D);
size_t moe_few_ws_bytes(const MoeDims& D);
int moe_few_fwd(const MoeDims& D, const bpt_moe_route* r, const void* x, const void* w1, const void* w3, const void* w2, void* y, void* ws,
                cudaStream_t st);

}  // namespace bpt
