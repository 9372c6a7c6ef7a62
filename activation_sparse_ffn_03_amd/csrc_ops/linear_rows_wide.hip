// Tiles of y = x w^T: both operands' k are neighbouring.
#include "linear_tiled.h"

namespace twell {

hipError_t launch_linear_rows_wide(const LinearArgs& a, hipStream_t s) { return launch_linear_act<LinearWide>(a, s); }

}  // namespace twell
