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

// The forward for so few rows that an expert's matrices meet about one
// (moe_few.cu): whether they are, its workspace, its launches.
bool moe_few_rows(const MoeDims& D);
size_t moe_few_ws_bytes(const MoeDims& D);
int moe_few_fwd(const MoeDims& D, const bpt_moe_route* r, const void* x, const void* w1, const void* w3, const void* w2, void* y, void* ws,
                cudaStream_t st);

}  // namespace bpt
