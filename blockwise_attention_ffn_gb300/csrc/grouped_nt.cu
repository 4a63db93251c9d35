// grouped_nt.cu -- the grouped GEMM's launches of the NT form (the forward's
// products).
#include "grouped_kernel.cuh"

namespace bpt {
namespace gg {

namespace {

template <int ACT>
int launch_act(Params& p, bool pair, bool small, int64_t units, cudaStream_t st) {
  constexpr int NT = GROUPED_NT, EPI = GROUPED_ACT;
  constexpr bool DUAL = ACT == BPT_ACT_SWIGLU;
  constexpr int BN = DUAL ? 128 : 256;
  if (small) return launch<NT, EPI, ACT, 64, true, false, DUAL, false>(p, units, st);
  return pair ? launch<NT, EPI, ACT, BN, true, false, DUAL, true>(p, units, st)
              : launch<NT, EPI, ACT, BN, true, false, DUAL, false>(p, units, st);
}

}  // namespace

int launch_nt(Params& p, int epi, int act, bool gather, bool pair, int bn, int64_t units, cudaStream_t st) {
  const bool small = bn == 64;
  constexpr int NT = GROUPED_NT, STORE = GROUPED_STORE;
  if (epi == GROUPED_STORE) {
    if (small) return launch<NT, STORE, 0, 64, true, false, false, false>(p, units, st);
    if (gather) return 1;
    if (bn == 128) return launch<NT, STORE, 0, 128, false, false, false, false>(p, units, st);
    return pair ? launch<NT, STORE, 0, 256, false, false, false, true>(p, units, st)
                : launch<NT, STORE, 0, 256, false, false, false, false>(p, units, st);
  }
  if (epi != GROUPED_ACT || !gather) return 1;
  if (act == BPT_ACT_SWIGLU) return launch_act<BPT_ACT_SWIGLU>(p, pair, small, units, st);
  if (act == BPT_ACT_GELU_ERF) return launch_act<BPT_ACT_GELU_ERF>(p, pair, small, units, st);
  return launch_act<BPT_ACT_GELU_TANH>(p, pair, small, units, st);
}

}  // namespace gg
}  // namespace bpt
