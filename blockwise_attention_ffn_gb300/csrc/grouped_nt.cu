// grouped_nt.cu -- the grouped GEMM's launches of the NT form (the forward's
// products).
#include "grouped_kernel.cuh"

namespace bpt {
namespace gg {

int launch_nt(Params& p, int epi, bool gather, bool dual, bool pair, bool small, int64_t units, cudaStream_t st) {
  constexpr int NT = GROUPED_NT, STORE = GROUPED_STORE, ACT = GROUPED_ACT;
  if (epi == GROUPED_STORE) {
    if (small) return launch<NT, STORE, 64, true, false, false, false>(p, units, st);
    if (gather) return 1;
    return pair ? launch<NT, STORE, 256, false, false, false, true>(p, units, st)
                : launch<NT, STORE, 256, false, false, false, false>(p, units, st);
  }
  if (epi != GROUPED_ACT || !gather) return 1;
  if (dual) {
    if (small) return launch<NT, ACT, 64, true, false, true, false>(p, units, st);
    return pair ? launch<NT, ACT, 128, true, false, true, true>(p, units, st)
                : launch<NT, ACT, 128, true, false, true, false>(p, units, st);
  }
  if (small) return launch<NT, ACT, 64, true, false, false, false>(p, units, st);
  return pair ? launch<NT, ACT, 256, true, false, false, true>(p, units, st)
              : launch<NT, ACT, 256, true, false, false, false>(p, units, st);
}

}  // namespace gg
}  // namespace bpt
