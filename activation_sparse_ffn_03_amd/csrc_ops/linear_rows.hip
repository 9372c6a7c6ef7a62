// Tiles of y = x w^T: both operands' k are neighbouring.
#include "linear_tiled.h"

namespace twell {

template <class C>
static hipError_t launch_act(const LinearArgs& a, hipStream_t s) {
  switch (a.splits > 1 ? TWELL_ACT_NONE : a.out.act) {
    case TWELL_ACT_RELU: return launch_linear_tile<C, false, false, TWELL_ACT_RELU>(a, s);
    case TWELL_ACT_SILU: return launch_linear_tile<C, false, false, TWELL_ACT_SILU>(a, s);
    case TWELL_ACT_GELU: return launch_linear_tile<C, false, false, TWELL_ACT_GELU>(a, s);
    default: return launch_linear_tile<C, false, false, TWELL_ACT_NONE>(a, s);
  }
}

hipError_t launch_linear_rows(int tile, const LinearArgs& a, hipStream_t s) {
  return tile == LinearBig::BU ? launch_act<LinearBig>(a, s) : launch_act<LinearMid>(a, s);
}

}  // namespace twell
