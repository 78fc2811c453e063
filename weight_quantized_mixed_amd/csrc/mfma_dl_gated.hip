// Direct-load MFMA path: the instances for gated plans (their epilogue joins the gate and
// up sums; a translation unit of their own, so that both sets compile at the same time).
#include "mfma_dl_kernel.hpp"

namespace qg {

hipError_t launch_mfma_dl_gated(int fmt, int tile, const RunArgs& a, hipStream_t st) {
  return launch_any_tile<true>(fmt, tile, a, st);
}

}  // namespace qg
