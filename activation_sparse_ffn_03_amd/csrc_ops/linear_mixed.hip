// Tiles of dx = dz w: w's lines are k (its units), its columns the result's.
#include "linear_tiled.h"

namespace twell {

hipError_t launch_linear_mixed(LinearTileSize tile, const LinearArgs& a, hipStream_t s) {
  switch (tile) {
    case LINEAR_BIG: return launch_linear_tile<LinearBig, true, false, TWELL_ACT_NONE, false>(a, s);
    case LINEAR_WIDE: return launch_linear_tile<LinearWide, true, false, TWELL_ACT_NONE, false>(a, s);
    case LINEAR_MID: return launch_linear_tile<LinearMid, true, false, TWELL_ACT_NONE, false>(a, s);
    default: return launch_linear_tile<LinearFew, true, false, TWELL_ACT_NONE, false>(a, s);
  }
}

}  // namespace twell
