// Dropout's random numbers, from a counter and a key alone: Philox4x32-10
// (Salmon, Moraes, Dror, Shaw: "Parallel random numbers: as easy as 1, 2, 3",
// 2011), checked against that paper's test vectors.
//
// Element (row, col) of a [rows][cols] array uses 16 of the 128 bits of the
// block with counter (col / 8, row, step, site) and key seed: half col & 1 of
// word (col & 7) / 2. It is dropped when that number is below `drop`, the
// dropped share in 1/65536, so that a kept element times 65536 / (65536 - drop)
// has the element as its mean exactly. 16 bits an element and not 32: the ten
// rounds are 20 products of 32 bits to 64 a block, at a quarter of the rate of
// an addition, and with four elements a block they and not memory would bound
// a bf16 array. The mask depends on nothing else, no grid, chunk or order, and
// is made again wherever it is needed.
#pragma once

#include "chunk8.h"

namespace twell {

// What a kernel needs: seed and step are read from device memory, so that a
// captured call draws anew when the caller advances the step between replays.
struct DropArgs {
  const uint64_t* rng;  // [2] seed, step (modulo 2^32); not read when drop is 0
  uint32_t site;
  uint32_t drop;   // 0: nothing is dropped, 65536: everything
  float scale;     // 65536 / (65536 - drop), 0 when everything is dropped
};

__device__ __forceinline__ u32x4_t philox4x32(u32x4_t c, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = (uint64_t)c[0] * 0xD2511F53u, b = (uint64_t)c[2] * 0xCD9E8D57u;
    c = u32x4_t{(uint32_t)(b >> 32) ^ c[1] ^ k0, (uint32_t)b, (uint32_t)(a >> 32) ^ c[3] ^ k1, (uint32_t)a};
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return c;
}

// The generator of one call.
struct DropBits {
  uint32_t k0 = 0, k1 = 0, step = 0, site = 0, drop = 0;
  DropBits() = default;
  __device__ __forceinline__ explicit DropBits(const DropArgs& d) : site(d.site), drop(d.drop) {
    const uint64_t seed = d.rng[0];
    k0 = (uint32_t)seed;
    k1 = (uint32_t)(seed >> 32);
    step = (uint32_t)d.rng[1];
  }
  // Bit k: element 8 g + k of the row is kept.
  __device__ __forceinline__ uint32_t group(uint32_t row, uint32_t g) const {
    const u32x4_t w = philox4x32(u32x4_t{g, row, step, site}, k0, k1);
    uint32_t keep = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t v = k & 1 ? w[k >> 1] >> 16 : w[k >> 1] & 0xFFFFu;
      keep |= (v >= drop ? 1u : 0u) << k;
    }
    return keep;
  }
  // Bit k: element k of chunk i is kept, wherever the chunk lies (chunk_col);
  // none of a chunk behind the row's end.
  template <int KIND>
  __device__ __forceinline__ uint32_t chunk(uint32_t row, int i, int cols) const {
    if (8 * i >= cols) return 0;
    uint32_t keep = group(row, i);
    if constexpr (KIND == ROWS_ANY) {
      const int back = 8 * i - chunk_col<KIND>(i, cols);  // elements of the group before
      if (back > 0) keep = (group(row, i - 1) >> (8 - back)) | (keep << back);
    }
    return keep;
  }
};

}  // namespace twell
