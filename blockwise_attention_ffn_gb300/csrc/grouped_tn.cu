// grouped_tn.cu -- the grouped GEMM's launches of the TN form (the gradients
// of the matrices).
#include "grouped_kernel.cuh"

namespace bpt {
namespace gg {

int launch_tn(Params& p, bool a_gather, bool b_gather, bool pair, int64_t units, cudaStream_t st) {
  constexpr int TN = GROUPED_TN, STORE = GROUPED_STORE;
  if (a_gather && b_gather) return 1;
  if (a_gather)
    return pair ? launch<TN, STORE, 0, 256, true, false, false, true>(p, units, st)
                : launch<TN, STORE, 0, 256, true, false, false, false>(p, units, st);
  if (b_gather)
    return pair ? launch<TN, STORE, 0, 256, false, true, false, true>(p, units, st)
                : launch<TN, STORE, 0, 256, false, true, false, false>(p, units, st);
  return pair ? launch<TN, STORE, 0, 256, false, false, false, true>(p, units, st)
              : launch<TN, STORE, 0, 256, false, false, false, false>(p, units, st);
}

}  // namespace gg
}  // namespace bpt
