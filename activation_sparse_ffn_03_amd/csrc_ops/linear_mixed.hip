// Tiles of dx = dz w: w's lines are k (its units), its columns the result's.
#include "linear_tiled.h"

namespace twell {

hipError_t launch_linear_mixed(int tile, const LinearArgs& a, hipStream_t s) {
  if (tile == LinearBig::BU) return launch_linear_tile<LinearBig, true, false, TWELL_ACT_NONE>(a, s);
  return launch_linear_tile<LinearMid, true, false, TWELL_ACT_NONE>(a, s);
}

}  // namespace twell
