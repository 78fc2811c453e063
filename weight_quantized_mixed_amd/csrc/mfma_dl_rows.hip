// Direct-load MFMA path: the instances of the gradient products, fp16 weights whose rows of
// sums have a scale each (kept apart so that the plain ones keep their registers).
#include "mfma_dl_kernel.hpp"

namespace qg {
namespace {

template <int T>
hipError_t launch_rows(const RunArgs& a, hipStream_t st) {
  return launch_t<FMT_F16, T, false, false, false, true>(a, st);
}

}  // namespace

hipError_t launch_mfma_dl_rows(int tile, const RunArgs& a, hipStream_t st) {
  switch (tile) {  // the tiles that choose_dl_tile gives fp16
    case DL_32x64: return launch_rows<DL_32x64>(a, st);
    case DL_32x128: return launch_rows<DL_32x128>(a, st);
    case DL_32x256: return launch_rows<DL_32x256>(a, st);
    case DL_64x128: return launch_rows<DL_64x128>(a, st);
    case DL_64x256: return launch_rows<DL_64x256>(a, st);
    case DL_128x256: return launch_rows<DL_128x256>(a, st);
#if !QG_BIG4
    case DL_256x256: return launch_rows<DL_256x256>(a, st);
#endif
  }
  return hipErrorInvalidValue;
}

}  // namespace qg
