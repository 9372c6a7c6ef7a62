// Tiles of dw = dz^T x: both operands' lines are k (the tokens).
#include "linear_tiled.h"

namespace twell {

hipError_t launch_linear_cols(int tile, const LinearArgs& a, hipStream_t s) {
  if (tile == LinearBig::BU) return launch_linear_tile<LinearBig, true, true, TWELL_ACT_NONE>(a, s);
  return launch_linear_tile<LinearMid, true, true, TWELL_ACT_NONE>(a, s);
}

}  // namespace twell
