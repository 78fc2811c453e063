// The attention tiles of calls with a window, in a file of their own so that they compile
// beside the others.
#include "attention_kernel.hpp"

namespace qg {
namespace {

template <int DP>
hipError_t launch_dim(const WindowArgs& a, const AttnSplit& p, hipStream_t st) {
  if (p.kind_s == TILE_KEYS) return launch_kinds<DP, TILE_NONE, TILE_KEYS>(a, p, st);
  if (p.kind_s == TILE_ROWS64) return launch_kinds<DP, TILE_NONE, TILE_ROWS64>(a, p, st);
  if constexpr (DP <= 128) return launch_kinds<DP, TILE_NONE, TILE_ROWS128>(a, p, st);
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_window_tiles(const WindowArgs& a, const AttnSplit& p, hipStream_t st) {
  return a.D <= 64 ? launch_dim<64>(a, p, st) : a.D <= 128 ? launch_dim<128>(a, p, st) : launch_dim<256>(a, p, st);
}

}  // namespace qg
