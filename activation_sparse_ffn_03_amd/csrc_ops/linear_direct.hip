// Products of few rows, and small ones of up to 512, y = x w^T: a workgroup takes
// 16 FU units by up to 8 XG rows, each of its waves every WAVES-th 64 columns of
// all of it; the waves' sums are added in LDS in a fixed order, and the result
// finished as in the tiles.
//
// Bound by reading w once. v_mfma_f32_16x16x32_bf16 wants lane l to hold 8 columns
// of line l & 15 (its results are units 4 (l >> 4) + r of row l & 15), but loads
// done that way touch 16 cache lines each, and a compute unit's path to memory
// takes about 4 cycles a line, whatever is used of it (1 x 4096 x 11008 16.5 us,
// 24 x 5632 x 2048 15.1, however many loads are in flight). So a load takes 8
// whole lines of 128 bytes, lane l piece l & 7 of line l >> 3, and the wave turns
// them in LDS of its own, without barriers: piece p of line r lies at piece
// p ^ (r & 7), which keeps both sides' accesses on different banks: 14.6 us (6.2
// TB/s, most of w from the 256 MB cache) and, in 256 workgroups of 16 rows, 7.6.
//
// A wave has DEPTH steps' loads on their way all the time; loads lie in no branch,
// since the compiler waits for all of them where branches meet.
#include "linear_device.h"
#include "../csrc/twell_trace.h"

namespace twell {
namespace {

// Chunk c of a line of `cols` columns: zeros behind its end. The load is done in
// any case, of a chunk behind the end of the last one. LINES: as chunk8.h's kinds.
template <int LINES>
struct Chunk {
  u32x4_t v;
  __device__ __forceinline__ void load(const uint16_t* line, int c, int cols) {
    if constexpr (LINES == ROWS_ALIGNED) v = *reinterpret_cast<const u32x4_t*>(line + min(8 * c, cols - 8));
    else if constexpr (LINES == ROWS_ANY) v = *reinterpret_cast<const u32x4_a2_t*>(line + min(8 * c, cols - 8));
    else {
      v = u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
      for (int k = 0; k < 7; ++k)
        if (8 * c + k < cols) v[k >> 1] |= (uint32_t)line[k] << (16 * (k & 1));
    }
  }
  __device__ __forceinline__ u32x4_t get(int c, int cols) const {
    Raw8<uint16_t> r;
    r.v = v;
    if constexpr (LINES == ROWS_ANY) r.template settle<true>(c, cols);  // of a partial one the line's last 8 were loaded
    if (LINES != ROWS_SHORT && 8 * c >= cols) r.v = u32x4_t{0u, 0u, 0u, 0u};
    return r.v;
  }
};

template <int FU, int XG, int WAVES, int DEPTH, int LINES, int ACT>
__global__ __launch_bounds__(64 * WAVES) void linear_direct(LinearArgs a, int64_t row_tiles) {
  constexpr int FT = (XG + 1) / 2, WG = 2 * FU, LINES_HELD = 8 * WG + 16 * FT;
  __shared__ u32x4_t turn[WAVES][LINES_HELD * 8];
  __shared__ f32x4_t red[WAVES][FU * FT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t L = xcd_run_block(blockIdx.x, gridDim.x);  // neighbours in one L2 share their weights
  const int64_t r0 = L % row_tiles * (8 * XG);
  const int u0 = (int)(L / row_tiles) * (16 * FU);
  const LinearOut& o = a.out;
  const int cols = (int)a.k, steps = (cols + 63) / 64;

  // Lines behind the last unit or row read the last one: their results are not
  // stored.
  const int lr = lane >> 3, piece = lane & 7;
  const uint16_t *w[WG], *x[XG];
#pragma unroll
  for (int i = 0; i < WG; ++i) w[i] = a.p.p + (int64_t)min(u0 + 8 * i + lr, o.units - 1) * a.p.ld;
#pragma unroll
  for (int j = 0; j < XG; ++j) x[j] = a.q.p + min(r0 + 8 * j + lr, o.rows - 1) * a.q.ld;
  Chunk<LINES> rw[DEPTH][WG], rx[DEPTH][XG];
  auto load = [&](int d, int step) {
    const int c = 8 * step + piece;
#pragma unroll
    for (int i = 0; i < WG; ++i) rw[d][i].load(w[i], c, cols);
#pragma unroll
    for (int j = 0; j < XG; ++j) rx[d][j].load(x[j], c, cols);
  };
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) load(d, wave + d * WAVES);

  // what the epilogue reads
  static_assert(FU * FT <= WAVES, "a wave finishes one fragment at most");
  const int line = lane & 15, kb = lane >> 4;
  const int64_t row = r0 + 16 * (wave % FT) + line;
  const int unit = u0 + 16 * (wave / FT) + 4 * kb;
  const bool mine = wave < FU * FT && row < min(o.rows, r0 + 8 * XG) && unit < o.units;
  float bias[4] = {0.f, 0.f, 0.f, 0.f}, res[4] = {0.f, 0.f, 0.f, 0.f};
  if (mine && o.bias != nullptr) load_some<4>(o.bias, o.bias_bf16, unit, o.units - unit, bias);
  if (mine && o.residual != nullptr) load_some<4>(o.residual, o.res_bf16, row * o.units + unit, o.units - unit, res);

  f32x4_t acc[FU][FT];
#pragma unroll
  for (int i = 0; i < FU; ++i)
#pragma unroll
    for (int j = 0; j < FT; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  u32x4_t* const own = turn[wave];
  u32x4_t* const to = own + 8 * lr + (piece ^ lr);
  if constexpr (XG % 2 == 1) to[64 * (WG + XG)] = u32x4_t{0u, 0u, 0u, 0u};  // rows that no load brings
  auto multiply = [&](int d, int step) {
    const int c = 8 * step + piece;
#pragma unroll
    for (int i = 0; i < WG; ++i) to[64 * i] = rw[d][i].get(c, cols);
#pragma unroll
    for (int j = 0; j < XG; ++j) to[64 * (WG + j)] = rx[d][j].get(c, cols);
    // A wave's LDS operations are done in their order; the statements keep the
    // compiler to it, which sees no lane's write of what another reads.
    asm volatile("" ::: "memory");
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u32x4_t* from = own + 8 * line + ((kb + 4 * h) ^ (line & 7));
      u32x4_t xv[FT];
#pragma unroll
      for (int j = 0; j < FT; ++j) xv[j] = from[64 * WG + 128 * j];
#pragma unroll
      for (int i = 0; i < FU; ++i) {
        const u32x4_t wv = from[128 * i];
#pragma unroll
        for (int j = 0; j < FT; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, wv),
                                                              __builtin_bit_cast(bf16x8_t, xv[j]), acc[i][j], 0, 0, 0);
      }
    }
    asm volatile("" ::: "memory");
  };
  int step = wave;
  for (; step + DEPTH * WAVES < steps; step += DEPTH * WAVES) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      multiply(d, step + d * WAVES);
      load(d, step + (d + DEPTH) * WAVES);
    }
  }
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) multiply(d, step + d * WAVES);  // steps behind the last are zeros

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

template <int FU, int XG, int WAVES, int DEPTH, int ACT>
hipError_t launch_cfg(const LinearArgs& a, hipStream_t s) {
  const int64_t rt = (a.out.rows + 8 * XG - 1) / (8 * XG), ut = (a.out.units + 16 * FU - 1) / (16 * FU);
  const dim3 grid((unsigned)(rt * ut));
  return row_kind((int)a.k, [&](auto kind) {
    TWELL_LAUNCH("linear_direct", (linear_direct<FU, XG, WAVES, DEPTH, decltype(kind)::value, ACT>), grid, 64 * WAVES, 0, s,
                 a, rt);
    return hipGetLastError();
  });
}

template <int ACT>
hipError_t launch_act(const LinearArgs& a, hipStream_t s) {
  switch (linear_direct_groups(a.out.rows, a.k, a.out.units)) {
    case 1: return launch_cfg<1, 1, 8, 4, ACT>(a, s);
    case 2: return launch_cfg<1, 2, 8, 4, ACT>(a, s);
    case 3: return launch_cfg<1, 3, 8, 2, ACT>(a, s);
    default: return launch_cfg<1, 4, 8, 3, ACT>(a, s);
  }
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
