// grouped_nn.cu -- the grouped GEMM's launches of the NN form (the gradients
// of the rows).
#include "grouped_kernel.cuh"

namespace bpt {
namespace gg {

int launch_nn(Params& p, int epi, bool pair, int64_t units, cudaStream_t st) {
  constexpr int NN = GROUPED_NN;
  if (epi == GROUPED_ACT_BWD)
    return pair ? launch<NN, GROUPED_ACT_BWD, 256, true, false, false, true>(p, units, st)
                : launch<NN, GROUPED_ACT_BWD, 256, true, false, false, false>(p, units, st);
  if (epi != GROUPED_STORE) return 1;
  return pair ? launch<NN, GROUPED_STORE, 256, false, false, false, true>(p, units, st)
              : launch<NN, GROUPED_STORE, 256, false, false, false, false>(p, units, st);
}

}  // namespace gg
}  // namespace bpt
