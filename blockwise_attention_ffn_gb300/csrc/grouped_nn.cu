// grouped_nn.cu -- the grouped GEMM's launches of the NN form (the gradients
// of the rows).
#include "grouped_kernel.cuh"

namespace bpt {
namespace gg {

namespace {

template <int ACT>
int launch_act_bwd(Params& p, bool pair, int64_t units, cudaStream_t st) {
  constexpr int NN = GROUPED_NN, EPI = GROUPED_ACT_BWD;
  return pair ? launch<NN, EPI, ACT, 256, true, false, false, true>(p, units, st)
              : launch<NN, EPI, ACT, 256, true, false, false, false>(p, units, st);
}

}  // namespace

int launch_nn(Params& p, int epi, int act, bool pair, int bn, int64_t units, cudaStream_t st) {
  constexpr int NN = GROUPED_NN, STORE = GROUPED_STORE;
  if (epi == GROUPED_ACT_BWD) {
    if (act == BPT_ACT_SWIGLU) return launch_act_bwd<BPT_ACT_SWIGLU>(p, pair, units, st);
    if (act == BPT_ACT_GELU_ERF) return launch_act_bwd<BPT_ACT_GELU_ERF>(p, pair, units, st);
    return launch_act_bwd<BPT_ACT_GELU_TANH>(p, pair, units, st);
  }
  if (epi != GROUPED_STORE) return 1;
  if (bn == 128) return launch<NN, STORE, 0, 128, false, false, false, false>(p, units, st);
  return pair ? launch<NN, STORE, 0, 256, false, false, false, true>(p, units, st)
              : launch<NN, STORE, 0, 256, false, false, false, false>(p, units, st);
}

}  // namespace gg
}  // namespace bpt
