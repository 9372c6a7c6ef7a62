// Both products of a small layer's gradients, dx = dz w and dw = dz^T x, in one
// launch: neither fills the chip, and neither reads what the other writes.
#include "linear_tiled.h"

namespace twell {
namespace {

// The first `of_dx` workgroups take dx, a tile each, the others dw.
template <bool ANY>
__global__ __launch_bounds__(256, LinearFew::OCC) void linear_pair(LinearArgs dx, LinearArgs dw, uint32_t ub, uint32_t of_dx) {
  __shared__ __attribute__((aligned(1024))) char smem[LinearFew::LDS];
  if (blockIdx.x < of_dx)
    linear_items<LinearFew, true, false, ANY, false, TWELL_ACT_NONE, false>(dx, of_dx / ub, ub, blockIdx.x, of_dx, smem);
  else
    linear_items<LinearFew, true, true, ANY, false, TWELL_ACT_NONE, false>(dw, (gridDim.x - of_dx) / ub, ub, blockIdx.x - of_dx,
                                                                           gridDim.x - of_dx, smem);
}

}  // namespace

hipError_t launch_linear_pair(const LinearArgs& dx, const LinearArgs& dw, hipStream_t s) {
  using C = LinearFew;
  const int64_t ub = (dx.out.units + C::BU - 1) / C::BU;
  const int64_t of_dx = (dx.out.rows + C::BT - 1) / C::BT * ub, of_dw = (dw.out.rows + C::BT - 1) / C::BT * ub;
  if (dx.out.units != dw.out.units || dx.any != dw.any || of_dx + of_dw > 256 * C::OCC) return hipErrorInvalidValue;
  const dim3 grid((unsigned)(of_dx + of_dw));
  if (dx.any)
    TWELL_LAUNCH("linear_pair", linear_pair<true>, grid, 256, 0, s, dx, dw, (uint32_t)ub, (uint32_t)of_dx);
  else
    TWELL_LAUNCH("linear_pair", linear_pair<false>, grid, 256, 0, s, dx, dw, (uint32_t)ub, (uint32_t)of_dx);
  return hipGetLastError();
}

}  // namespace twell
