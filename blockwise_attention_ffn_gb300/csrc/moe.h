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

}  // namespace bpt
