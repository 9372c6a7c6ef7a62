// What the norm in front of a block and the join of a block's output to the
// stream share on the device.
#pragma once

#include <cfloat>

#include "chunk8.h"
#include "ops_kernels.h"

namespace twell {

// Codes of 8 quotients n / sc. With FAST the row's largest magnitude is finite
// and its scale normal, so that every quotient is at most 448.001 and the
// hardware conversion (nearest, ties to even) is right as it stands. Otherwise
// quotients are held to +-448 first and NaN gets the code 0x7F.
template <bool FAST>
__device__ __forceinline__ u32x2_t encode8(const float (&n)[8], float sc) {
  float v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    v[k] = n[k] / sc;
    if constexpr (!FAST) v[k] = v[k] > 448.f ? 448.f : v[k] < -448.f ? -448.f : v[k];
  }
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
  u32x2_t r = {(uint32_t)lo, (uint32_t)hi};
  if constexpr (!FAST) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int s = 8 * (k & 3);
      if (v[k] != v[k]) r[k >> 2] = (r[k >> 2] & ~(0xFFu << s)) | (0x7Fu << s);
    }
  }
  return r;
}

// Where a row's sum of squares overflows its elements are scaled by this, so
// that the sum is below their mean square.
constexpr float kShrink = 1.f / 128;
static_assert(kNormMaxCols <= 128 * 128, "the sum of the shrunk squares of a row");

// 448 * 2^-126: from here the scale is a normal number.
constexpr uint32_t kNormalScaleBits = 0x04E00000u;

}  // namespace twell
