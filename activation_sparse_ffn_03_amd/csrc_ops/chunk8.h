// Row access of the operators around the block.
//
// A row is dealt to its threads in chunks of 8 elements (16 bytes of bf16, 32
// of fp32): thread t of T takes chunks t, t + T, ...; elements behind the row's
// end read as zeros and are not written. TAIL is set when the row
// length is not a multiple of 8: rows then start at any element, so chunks are
// read and written with element-aligned vector accesses (global memory takes
// them at any alignment on gfx950), and the row's last, partial chunk one
// element at a time. Without TAIL every chunk is 16-byte aligned.
#pragma once

#include "../csrc/twell_device.h"

namespace twell {

typedef uint32_t u32x4_a2_t __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_a4_t __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2_a1_t __attribute__((ext_vector_type(2), aligned(1)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

// Two floats to bf16, nearest with ties to even, NaN kept (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16x2_t));
}

template <typename T>
struct Raw8;

template <>
struct Raw8<uint16_t> {
  u32x4_t v;
  template <bool TAIL>
  __device__ __forceinline__ void load(const uint16_t* row, int i, int cols) {
    v = u32x4_t{0u, 0u, 0u, 0u};
    const uint16_t* p = row + 8 * i;
    if constexpr (!TAIL) {
      if (8 * i < cols) v = *reinterpret_cast<const u32x4_t*>(p);
    } else if (8 * i + 8 <= cols) {
      v = *reinterpret_cast<const u32x4_a2_t*>(p);
    } else {
#pragma unroll
      for (int k = 0; k < 7; ++k)
        if (8 * i + k < cols) v[k >> 1] |= (uint32_t)p[k] << (16 * (k & 1));
    }
  }
  // bit pattern of the largest magnitude, as fp32
  __device__ __forceinline__ uint32_t max_bits() const {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) m = max(m, max((v[k] & 0x7FFFu) << 16, v[k] & 0x7FFF0000u));
    return m;
  }
  __device__ __forceinline__ float get(int k) const { return k & 1 ? bf16hi_to_f32(v[k >> 1]) : bf16lo_to_f32(v[k >> 1]); }
};

template <>
struct Raw8<float> {
  u32x4_t v[2];
  template <bool TAIL>
  __device__ __forceinline__ void load(const float* row, int i, int cols) {
    v[0] = v[1] = u32x4_t{0u, 0u, 0u, 0u};
    const float* p = row + 8 * i;
    if constexpr (!TAIL) {
      if (8 * i < cols) {
        v[0] = *reinterpret_cast<const u32x4_t*>(p);
        v[1] = *reinterpret_cast<const u32x4_t*>(p + 4);
      }
    } else if (8 * i + 8 <= cols) {
      v[0] = *reinterpret_cast<const u32x4_a4_t*>(p);
      v[1] = *reinterpret_cast<const u32x4_a4_t*>(p + 4);
    } else {
#pragma unroll
      for (int k = 0; k < 7; ++k)
        if (8 * i + k < cols) v[k >> 2][k & 3] = __float_as_uint(p[k]);
    }
  }
  __device__ __forceinline__ uint32_t max_bits() const {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, v[k >> 2][k & 3] & 0x7FFFFFFFu);
    return m;
  }
  __device__ __forceinline__ float get(int k) const { return __uint_as_float(v[k >> 2][k & 3]); }
};

// Writes chunk i of a row; for bf16 the values are rounded.
template <bool TAIL>
__device__ __forceinline__ void store8(uint16_t* row, int i, int cols, const float (&x)[8]) {
  const u32x4_t v = {pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
  uint16_t* p = row + 8 * i;
  if constexpr (!TAIL) {
    if (8 * i < cols) *reinterpret_cast<u32x4_t*>(p) = v;
  } else if (8 * i + 8 <= cols) {
    *reinterpret_cast<u32x4_a2_t*>(p) = v;
  } else {
#pragma unroll
    for (int k = 0; k < 7; ++k)
      if (8 * i + k < cols) p[k] = (uint16_t)(v[k >> 1] >> (16 * (k & 1)));
  }
}
template <bool TAIL>
__device__ __forceinline__ void store8(float* row, int i, int cols, const float (&x)[8]) {
  float* p = row + 8 * i;
  if constexpr (!TAIL) {
    if (8 * i < cols) {
      *reinterpret_cast<f32x4_t*>(p) = f32x4_t{x[0], x[1], x[2], x[3]};
      *reinterpret_cast<f32x4_t*>(p + 4) = f32x4_t{x[4], x[5], x[6], x[7]};
    }
  } else if (8 * i + 8 <= cols) {
    *reinterpret_cast<u32x4_a4_t*>(p) = __builtin_bit_cast(u32x4_t, f32x4_t{x[0], x[1], x[2], x[3]});
    *reinterpret_cast<u32x4_a4_t*>(p + 4) = __builtin_bit_cast(u32x4_t, f32x4_t{x[4], x[5], x[6], x[7]});
  } else {
#pragma unroll
    for (int k = 0; k < 7; ++k)
      if (8 * i + k < cols) p[k] = x[k];
  }
}

// Weight chunks of this thread as floats (bf16 or fp32 storage, uniform).
template <int T, int C, bool TAIL>
__device__ __forceinline__ void load_weight(const void* w, int is_bf16, int t, int cols, float (&wv)[C][8]) {
  if (is_bf16) {
    Raw8<uint16_t> raw[C];
#pragma unroll
    for (int c = 0; c < C; ++c) raw[c].template load<TAIL>(static_cast<const uint16_t*>(w), t + T * c, cols);
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) wv[c][k] = raw[c].get(k);
  } else {
    Raw8<float> raw[C];
#pragma unroll
    for (int c = 0; c < C; ++c) raw[c].template load<TAIL>(static_cast<const float*>(w), t + T * c, cols);
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) wv[c][k] = raw[c].get(k);
  }
}

// Largest of a 32-bit pattern over the wave, in every lane: quad and row
// steps by DPP, then across the four rows of 16 lanes.
__device__ __forceinline__ uint32_t wave_max_bits(uint32_t m) {
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, false));
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, false));
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x141, 0xF, 0xF, false));
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x140, 0xF, 0xF, false));
  const uint32_t a = (uint32_t)__builtin_amdgcn_readlane((int)m, 0), b = (uint32_t)__builtin_amdgcn_readlane((int)m, 16);
  const uint32_t c = (uint32_t)__builtin_amdgcn_readlane((int)m, 32), d = (uint32_t)__builtin_amdgcn_readlane((int)m, 48);
  return max(max(a, b), max(c, d));
}

}  // namespace twell
