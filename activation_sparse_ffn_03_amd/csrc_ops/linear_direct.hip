// Products of few rows, y = x w^T, straight from memory into registers: a
// workgroup takes 16 FU units by 16 FT rows, each of its waves every WAVES-th 64
// columns of all of it on v_mfma_f32_16x16x32_bf16; the waves' sums are added in
// LDS in a fixed order, and the result finished as in the tiles.
//
// Bound by reading w once. Lane l holds 16 neighbouring columns, 32 bytes, of
// line l & 15 (the lanes of a line one cache line of 128 bytes), for two matrix
// instructions: which columns share an instruction is free as long as both
// operands agree. Its results are units 4 (l >> 4) + r of row l & 15.
#include "linear_device.h"
#include "../csrc/twell_trace.h"

namespace twell {
namespace {

template <int FU, int FT, int WAVES, bool TAIL, int ACT>
__global__ __launch_bounds__(64 * WAVES) void linear_direct(LinearArgs a, int64_t row_tiles) {
  __shared__ f32x4_t red[WAVES][FU * FT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int line = lane & 15, kb = lane >> 4;
  const int64_t L = xcd_run_block(blockIdx.x, gridDim.x);  // neighbours in one L2 share their weights
  const int64_t r0 = L % row_tiles * (16 * FT);
  const int u0 = (int)(L / row_tiles) * (16 * FU);
  const LinearOut& o = a.out;
  const int cols = (int)a.k, steps = (cols + 63) / 64;

  // Lines behind the last unit or row read the last one: their results are not
  // stored.
  const uint16_t *w[FU], *x[FT];
#pragma unroll
  for (int i = 0; i < FU; ++i) w[i] = a.p.p + (int64_t)min(u0 + 16 * i + line, o.units - 1) * a.p.ld;
#pragma unroll
  for (int j = 0; j < FT; ++j) x[j] = a.q.p + min(r0 + 16 * j + line, o.rows - 1) * a.q.ld;
  f32x4_t acc[FU][FT];
#pragma unroll
  for (int i = 0; i < FU; ++i)
#pragma unroll
    for (int j = 0; j < FT; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  // what the epilogue reads, ahead of the weights
  static_assert(FU * FT <= WAVES, "a wave finishes one fragment at most");
  const int64_t row = r0 + 16 * (wave % FT) + line;
  const int unit = u0 + 16 * (wave / FT) + 4 * kb;
  const bool mine = wave < FU * FT && row < o.rows && unit < o.units;
  float bias[4] = {0.f, 0.f, 0.f, 0.f}, res[4] = {0.f, 0.f, 0.f, 0.f};
  if (mine && o.bias != nullptr) load_some<4>(o.bias, o.bias_bf16, unit, o.units - unit, bias);
  if (mine && o.residual != nullptr) load_some<4>(o.residual, o.res_bf16, row * o.units + unit, o.units - unit, res);

  // several steps' loads in flight at a time
  constexpr int DEPTH = FU + FT > 4 ? 2 : 4;
  for (int k0 = wave; k0 < steps; k0 += DEPTH * WAVES) {
    Raw8<uint16_t> rw[DEPTH][2][FU], rx[DEPTH][2][FT];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = 8 * (k0 + d * WAVES) + 2 * kb + h;  // chunks behind the line's end are zeros
#pragma unroll
        for (int i = 0; i < FU; ++i) rw[d][h][i].template load_filled<TAIL>(w[i], c, cols);
#pragma unroll
        for (int j = 0; j < FT; ++j) rx[d][h][j].template load_filled<TAIL>(x[j], c, cols);
      }
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = 8 * (k0 + d * WAVES) + 2 * kb + h;
#pragma unroll
        for (int i = 0; i < FU; ++i) rw[d][h][i].template settle<TAIL>(c, cols);
#pragma unroll
        for (int j = 0; j < FT; ++j) rx[d][h][j].template settle<TAIL>(c, cols);
#pragma unroll
        for (int i = 0; i < FU; ++i)
#pragma unroll
          for (int j = 0; j < FT; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, rw[d][h][i].v),
                                                                __builtin_bit_cast(bf16x8_t, rx[d][h][j].v), acc[i][j], 0, 0, 0);
      }
  }

#pragma unroll
  for (int i = 0; i < FU; ++i)
#pragma unroll
    for (int j = 0; j < FT; ++j) red[wave][i * FT + j][lane] = acc[i][j];
  __syncthreads();
  if (!mine) return;
  f32x4_t s = red[0][wave][lane];
#pragma unroll
  for (int v = 1; v < WAVES; ++v) s += red[v][wave][lane];
  float z[4] = {s[0], s[1], s[2], s[3]};
  finish_units<ACT, 4>(o, row, unit, o.units - unit, z, bias, res);
}

template <int FU, int FT, int WAVES, int ACT>
hipError_t launch_cfg(const LinearArgs& a, hipStream_t s) {
  const int64_t rt = (a.out.rows + 16 * FT - 1) / (16 * FT), ut = (a.out.units + 16 * FU - 1) / (16 * FU);
  const dim3 grid((unsigned)(rt * ut));
  if (a.k % 8 == 0)
    TWELL_LAUNCH("linear_direct", (linear_direct<FU, FT, WAVES, false, ACT>), grid, 64 * WAVES, 0, s, a, rt);
  else
    TWELL_LAUNCH("linear_direct", (linear_direct<FU, FT, WAVES, true, ACT>), grid, 64 * WAVES, 0, s, a, rt);
  return hipGetLastError();
}

template <int ACT>
hipError_t launch_act(const LinearArgs& a, hipStream_t s) {
  if (a.out.rows <= 16) return launch_cfg<1, 1, 8, ACT>(a, s);
  if (a.out.rows <= 32) return launch_cfg<1, 2, 8, ACT>(a, s);
  return launch_cfg<2, 4, 8, ACT>(a, s);
}

}  // namespace

hipError_t launch_linear_direct(const LinearArgs& a, hipStream_t s) {
  switch (a.out.act) {
    case TWELL_ACT_RELU: return launch_act<TWELL_ACT_RELU>(a, s);
    case TWELL_ACT_SILU: return launch_act<TWELL_ACT_SILU>(a, s);
    case TWELL_ACT_GELU: return launch_act<TWELL_ACT_GELU>(a, s);
    default: return launch_act<TWELL_ACT_NONE>(a, s);
  }
}

}  // namespace twell
