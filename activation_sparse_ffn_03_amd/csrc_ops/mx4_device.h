// MX4 blocks on the device: 32 consecutive elements of a row as E2M1 codes
// (sign, 2 exponent bits, 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6) with one
// E8M0 scale 2^(code - 127).
#pragma once

#include "chunk8.h"

namespace twell {

// Scale code of a block from the bit pattern of its largest magnitude:
// floor(log2 max) - 2, so that the block's largest element lands in [4, 8) and
// is held to 6 at most; not below 2^-127. 255 (NaN) for a block with NaN or
// infinity.
__device__ __forceinline__ uint32_t mx4_scale_code(uint32_t mbits) {
  if (mbits >= 0x7F800000u) return 255u;
  const int e = (int)(mbits >> 23) - 2;
  return e < 0 ? 0u : (uint32_t)e;
}

// The scale as the operand of the conversions below, which read its exponent
// field (a field of 0 stands for 2^-127).
__device__ __forceinline__ float mx4_scale_operand(uint32_t code) { return __uint_as_float(code << 23); }

// Codes of 8 elements over a finite block's scale, element k in bits 4k. The
// conversion rounds to nearest with ties to even; a sweep of all fp32 patterns
// below 8 scales for nine scale codes, and of all bf16 patterns for all 253,
// found it equal to the definition (subnormals, signed zeros and the lowest
// scale included).
__device__ __forceinline__ uint32_t mx4_codes(const Raw8<float>& x, float sc) {
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, x.get(0), x.get(1), sc, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, x.get(2), x.get(3), sc, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, x.get(4), x.get(5), sc, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, x.get(6), x.get(7), sc, 3);
  return r;
}
__device__ __forceinline__ uint32_t mx4_codes(const Raw8<uint16_t>& x, float sc) {
  // words copied out first: a bit cast of a vector's element reads element 0
  const uint32_t w0 = x.v[0], w1 = x.v[1], w2 = x.v[2], w3 = x.v[3];
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2_t, w0), sc, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2_t, w1), sc, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2_t, w2), sc, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2_t, w3), sc, 3);
  return r;
}

}  // namespace twell
