// Row access of the operators around the block.
//
// A row is dealt to its threads in chunks of 8 elements (16 bytes of bf16, 32
// of fp32): thread t of T takes chunks t, t + T, ...; elements behind the row's
// end read as zeros and are not written.
#pragma once

#include "../csrc/twell_device.h"

namespace twell {

typedef uint32_t u32x4_a2_t __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_a4_t __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2_a1_t __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32x2_a2_t __attribute__((ext_vector_type(2), aligned(2)));
typedef float f32x4_a4_t __attribute__((ext_vector_type(4), aligned(4)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

// Two floats to bf16, nearest with ties to even, NaN kept (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16x2_t));
}

// How a row's chunks lie:
//   ROWS_ALIGNED  rows are whole chunks, every chunk 16-byte aligned;
//   ROWS_ANY      rows of 8 elements or more that start at any element: accesses
//                 are element-aligned vectors (global memory takes them at any
//                 alignment on gfx950), and a partial last chunk is moved back
//                 to the row's last 8 elements, the first `dup` of which belong
//                 to the chunk before, too: both compute and write the same, and
//                 a sum over the row leaves them out. Nothing is written before
//                 all of a row is read, so that an output may be its input;
//   ROWS_SHORT    rows of fewer than 8 elements, one at a time.
enum RowKind { ROWS_ALIGNED, ROWS_ANY, ROWS_SHORT };

template <int KIND>
__device__ __forceinline__ int chunk_col(int i, int cols) {
  return KIND == ROWS_ANY ? min(8 * i, cols - 8) : 8 * i;
}
// Whether element k of chunk i counts in a sum.
template <int KIND>
__device__ __forceinline__ bool chunk_counts(int i, int k, int cols) {
  return KIND != ROWS_ANY || chunk_col<KIND>(i, cols) + k >= 8 * i;
}

template <typename T>
struct Raw8;

template <>
struct Raw8<uint16_t> {
  u32x4_t v;
  template <int KIND>
  __device__ __forceinline__ void load(const uint16_t* row, int i, int cols) {
    if constexpr (KIND == ROWS_SHORT) {
      load_filled<true>(row, i, cols);
    } else {
      v = u32x4_t{0u, 0u, 0u, 0u};
      const uint16_t* p = row + chunk_col<KIND>(i, cols);
      if (8 * i < cols) {
        if constexpr (KIND == ROWS_ALIGNED) v = *reinterpret_cast<const u32x4_t*>(p);
        else v = *reinterpret_cast<const u32x4_a2_t*>(p);
      }
    }
  }
  // Chunk i as it is: a partial last one is filled with zeros (TAIL: there may
  // be one, and rows start at any element). Of a partial one the row's last 8
  // elements are loaded, and moved down by `settle`, to be called when all
  // loads are on their way.
  template <bool TAIL>
  __device__ __forceinline__ void load_filled(const uint16_t* row, int i, int cols) {
    v = u32x4_t{0u, 0u, 0u, 0u};
    const uint16_t* p = row + 8 * i;
    if constexpr (!TAIL) {
      if (8 * i < cols) v = *reinterpret_cast<const u32x4_t*>(p);
    } else if (cols >= 8) {
      if (8 * i < cols) v = *reinterpret_cast<const u32x4_a2_t*>(p - max(8 * i + 8 - cols, 0));
    } else {
#pragma unroll
      for (int k = 0; k < 7; ++k)
        if (8 * i + k < cols) v[k >> 1] |= (uint32_t)p[k] << (16 * (k & 1));
    }
  }
  template <bool TAIL>
  __device__ __forceinline__ void settle(int i, int cols) {
    const int s = 8 * i + 8 - cols;
    if (!TAIL || cols < 8 || s <= 0 || s >= 8) return;
    if (s & 4) v = u32x4_t{v[2], v[3], 0u, 0u};
    if (s & 2) v = u32x4_t{v[1], v[2], v[3], 0u};
    if (s & 1) v = u32x4_t{v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16, v[3] >> 16};
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
  template <int KIND>
  __device__ __forceinline__ void load(const float* row, int i, int cols) {
    if constexpr (KIND == ROWS_SHORT) {
      load_filled<true>(row, i, cols);
    } else {
      v[0] = v[1] = u32x4_t{0u, 0u, 0u, 0u};
      const float* p = row + chunk_col<KIND>(i, cols);
      if (8 * i < cols) {
        if constexpr (KIND == ROWS_ALIGNED) {
          v[0] = *reinterpret_cast<const u32x4_t*>(p);
          v[1] = *reinterpret_cast<const u32x4_t*>(p + 4);
        } else {
          v[0] = *reinterpret_cast<const u32x4_a4_t*>(p);
          v[1] = *reinterpret_cast<const u32x4_a4_t*>(p + 4);
        }
      }
    }
  }
  template <bool TAIL>
  __device__ __forceinline__ void load_filled(const float* row, int i, int cols) {
    v[0] = v[1] = u32x4_t{0u, 0u, 0u, 0u};
    const float* p = row + 8 * i;
    if constexpr (!TAIL) {
      if (8 * i < cols) {
        v[0] = *reinterpret_cast<const u32x4_t*>(p);
        v[1] = *reinterpret_cast<const u32x4_t*>(p + 4);
      }
    } else if (cols >= 8) {
      if (8 * i < cols) {
        p -= max(8 * i + 8 - cols, 0);
        v[0] = *reinterpret_cast<const u32x4_a4_t*>(p);
        v[1] = *reinterpret_cast<const u32x4_a4_t*>(p + 4);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 7; ++k)
        if (8 * i + k < cols) v[k >> 2][k & 3] = __float_as_uint(p[k]);
    }
  }
  template <bool TAIL>
  __device__ __forceinline__ void settle(int i, int cols) {
    const int s = 8 * i + 8 - cols;
    if (!TAIL || cols < 8 || s <= 0 || s >= 8) return;
    if (s & 4) {
      v[0] = v[1];
      v[1] = u32x4_t{0u, 0u, 0u, 0u};
    }
    if (s & 2) {
      v[0] = u32x4_t{v[0][2], v[0][3], v[1][0], v[1][1]};
      v[1] = u32x4_t{v[1][2], v[1][3], 0u, 0u};
    }
    if (s & 1) {
      v[0] = u32x4_t{v[0][1], v[0][2], v[0][3], v[1][0]};
      v[1] = u32x4_t{v[1][1], v[1][2], v[1][3], 0u};
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
template <int KIND>
__device__ __forceinline__ void store8(uint16_t* row, int i, int cols, const float (&x)[8]) {
  const u32x4_t v = {pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
  uint16_t* p = row + chunk_col<KIND>(i, cols);
  if constexpr (KIND == ROWS_SHORT) {
#pragma unroll
    for (int k = 0; k < 7; ++k)
      if (8 * i + k < cols) p[k] = (uint16_t)(v[k >> 1] >> (16 * (k & 1)));
  } else if (8 * i < cols) {
    if constexpr (KIND == ROWS_ALIGNED) *reinterpret_cast<u32x4_t*>(p) = v;
    else *reinterpret_cast<u32x4_a2_t*>(p) = v;
  }
}
template <int KIND>
__device__ __forceinline__ void store8(float* row, int i, int cols, const float (&x)[8]) {
  float* p = row + chunk_col<KIND>(i, cols);
  const u32x4_t lo = __builtin_bit_cast(u32x4_t, f32x4_t{x[0], x[1], x[2], x[3]});
  const u32x4_t hi = __builtin_bit_cast(u32x4_t, f32x4_t{x[4], x[5], x[6], x[7]});
  if constexpr (KIND == ROWS_SHORT) {
#pragma unroll
    for (int k = 0; k < 7; ++k)
      if (8 * i + k < cols) p[k] = x[k];
  } else if (8 * i < cols) {
    if constexpr (KIND == ROWS_ALIGNED) {
      *reinterpret_cast<u32x4_t*>(p) = lo;
      *reinterpret_cast<u32x4_t*>(p + 4) = hi;
    } else {
      *reinterpret_cast<u32x4_a4_t*>(p) = lo;
      *reinterpret_cast<u32x4_a4_t*>(p + 4) = hi;
    }
  }
}
// Chunk i as it is, of a partial last one the elements there are.
template <bool TAIL, typename T>
__device__ __forceinline__ void store8_exact(T* row, int i, int cols, const float (&x)[8]) {
  if constexpr (!TAIL) {
    store8<ROWS_ALIGNED>(row, i, cols, x);
  } else if (8 * i + 8 <= cols) {
    store8<ROWS_ANY>(row, i, cols, x);
  } else {
    store8<ROWS_SHORT>(row, i, cols, x);
  }
}
// Eight bytes a chunk.
template <int KIND>
__device__ __forceinline__ void store8(uint8_t* row, int i, int cols, const u32x2_t& v) {
  uint8_t* p = row + chunk_col<KIND>(i, cols);
  if constexpr (KIND == ROWS_SHORT) {
#pragma unroll
    for (int k = 0; k < 7; ++k)
      if (8 * i + k < cols) p[k] = (uint8_t)(v[k >> 2] >> (8 * (k & 3)));
  } else if (8 * i < cols) {
    if constexpr (KIND == ROWS_ALIGNED) *reinterpret_cast<u32x2_t*>(p) = v;
    else *reinterpret_cast<u32x2_a1_t*>(p) = v;
  }
}

// Weight chunks of this thread as floats (bf16 or fp32 storage, uniform).
template <int T, int C, int KIND>
__device__ __forceinline__ void load_weight(const void* w, int is_bf16, int t, int cols, float (&wv)[C][8]) {
  if (is_bf16) {
    Raw8<uint16_t> raw[C];
#pragma unroll
    for (int c = 0; c < C; ++c) raw[c].template load<KIND>(static_cast<const uint16_t*>(w), t + T * c, cols);
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) wv[c][k] = raw[c].get(k);
  } else {
    Raw8<float> raw[C];
#pragma unroll
    for (int c = 0; c < C; ++c) raw[c].template load<KIND>(static_cast<const float*>(w), t + T * c, cols);
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) wv[c][k] = raw[c].get(k);
  }
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t m) {
  return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, CTRL, 0xF, 0xF, false));
}

// Sum, and largest 32-bit pattern, over each group of G lanes of a wave, in
// every lane of it: quad and row steps by DPP give the 16 lanes of a row theirs.
template <int G>
__device__ __forceinline__ float group_sum(float v) {
  if constexpr (G == 64) return wave_sum_dpp(v);
  v = dpp_add<0xB1, 0xF>(v);   // lanes 1 0 3 2
  v = dpp_add<0x4E, 0xF>(v);   // lanes 2 3 0 1
  v = dpp_add<0x141, 0xF>(v);  // mirror of 8
  v = dpp_add<0x140, 0xF>(v);  // mirror of 16
  if constexpr (G == 32) v += __shfl_xor(v, 16, 64);
  return v;
}
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t m) {
  m = dpp_max<0x140>(dpp_max<0x141>(dpp_max<0x4E>(dpp_max<0xB1>(m))));
  if constexpr (G == 32) m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
  if constexpr (G == 64) {
    const uint32_t a = (uint32_t)__builtin_amdgcn_readlane((int)m, 0), b = (uint32_t)__builtin_amdgcn_readlane((int)m, 16);
    const uint32_t c = (uint32_t)__builtin_amdgcn_readlane((int)m, 32), d = (uint32_t)__builtin_amdgcn_readlane((int)m, 48);
    m = max(max(a, b), max(c, d));
  }
  return m;
}

// Calls f(KIND) with the kind of rows of `cols` elements.
template <typename F>
auto row_kind(int cols, F f) {
  if (cols % 8 == 0) return f(std::integral_constant<int, ROWS_ALIGNED>{});
  if (cols >= 8) return f(std::integral_constant<int, ROWS_ANY>{});
  return f(std::integral_constant<int, ROWS_SHORT>{});
}

}  // namespace twell
