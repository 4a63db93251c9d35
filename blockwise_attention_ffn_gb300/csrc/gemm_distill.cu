// gemm_distill.cu -- the tcgen05 GEMM's launches with the distillation loss's
// epilogues (gemm_kernel.cuh: distill_tile, slab_tile).
#include "gemm_kernel.cuh"

namespace bpt {
namespace gk {

int launch_distill(GemmParams& p, bool pair, cudaStream_t st) {
  return pair ? launch<256, false, false, false, true, 1>(p, st) : launch<256, false, false, false, false, 1>(p, st);
}

int launch_slabs(GemmParams& p, bool pair, cudaStream_t st) {
  return pair ? launch<256, false, true, false, true, 2>(p, st) : launch<256, false, true, false, false, 2>(p, st);
}

}  // namespace gk
}  // namespace bpt
