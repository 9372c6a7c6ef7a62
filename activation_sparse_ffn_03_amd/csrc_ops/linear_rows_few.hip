// Tiles of y = x w^T: both operands' k are neighbouring.
#include "linear_tiled.h"

namespace twell {

hipError_t launch_linear_rows_few(const LinearArgs& a, hipStream_t s) { return launch_linear_act<LinearFew>(a, s); }

}  // namespace twell
