// Launch interface between the C ABI of the operators around the block
// (ops_api.hip) and their kernels. Everything here is host code.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace twell {

// Widest row the norm takes: a row is held in the registers of one workgroup.
constexpr int kNormMaxCols = 16384;

struct NormArgs {
  int64_t rows;
  int cols;
  int res_bf16, delta_bf16, w_bf16, out_bf16;
  const void* residual;  // [rows][cols]
  const void* delta;     // [rows][cols] or null
  const void* w;         // [cols]
  float eps;
  void* residual_out;    // [rows][cols] or null; may be `residual` itself
  void* out;             // [rows][cols] or null
  uint8_t* q;            // [rows][cols] or null
  float* q_scale;        // [rows], with q
  float* rstd;           // [rows] or null
};
hipError_t launch_add_rms_norm(const NormArgs& a, hipStream_t s);

struct NormBwdArgs {
  int64_t rows;
  int cols;
  int g_bf16, res_bf16, w_bf16;
  const void* d_out;       // [rows][cols]
  const void* d_residual;  // [rows][cols], type of the residual, or null
  const void* residual;    // [rows][cols]
  const float* rstd;       // [rows]
  const void* w;           // [cols]
  void* dr;                // [rows][cols], type of the residual
  float* dw;               // [cols]
  float* part;             // [norm_bwd_groups][cols] (workspace; unused for one group)
};
// Rows that a workgroup of the norm's backward takes side by side.
inline int norm_bwd_rows(int cols) {
  return cols <= 128 ? 16 : cols <= 512 ? 8 : cols <= 2048 ? 4 : cols <= 4096 ? 2 : 1;
}
// Workgroups of the norm's backward; each keeps one partial dw row. One a
// compute unit (two of the 256 threads that rows of up to 256 get), and no more
// than there are rows for: more partial rows cost the second launch more than
// they gain the first (4096x512 with two 9.2 us, with one 8.5).
inline int norm_bwd_groups(int64_t rows, int cols) {
  const int64_t need = (rows + norm_bwd_rows(cols) - 1) / norm_bwd_rows(cols), most = cols <= 256 ? 512 : 256;
  return (int)(need < 1 ? 1 : need > most ? most : need);
}
hipError_t launch_add_rms_norm_bwd(const NormBwdArgs& a, hipStream_t s);

// MX4 rows: 64 bytes of codes for every 128 columns begun, 16 scale bytes for
// every 512 begun.
constexpr int kMx4MaxCols = 1 << 20;
__host__ __device__ inline int mx4_code_bytes(int cols) { return (cols + 127) / 128 * 64; }
__host__ __device__ inline int mx4_scale_bytes(int cols) { return (cols + 511) / 512 * 16; }
// Scale codes arranged for the tiled product: [stage of 256 columns][row][8],
// the even blocks' four codes, then the odd blocks'.
struct Mx4Arrange {
  const uint8_t* scale;  // [rows] MX4 rows' scales
  uint8_t* out;          // [ceil(cols / 256)][pitch][8]
  int64_t rows, pitch;
};
// With `arranged` the scale codes are written there (pitch `pitch`) in place of
// `scale`, and `also` is arranged by further workgroups of the same launch.
hipError_t launch_quantize_mx4(const void* in, int is_bf16, int64_t rows, int cols, uint8_t* q, uint8_t* scale,
                               uint8_t* arranged, int64_t pitch, const Mx4Arrange* also, hipStream_t s);
hipError_t launch_mx4_arrange(const Mx4Arrange& a, const Mx4Arrange& b, int cols, hipStream_t s);
hipError_t launch_dequantize_mx4(const uint8_t* q, const uint8_t* scale, int64_t rows, int cols, int out_bf16,
                                 void* out, hipStream_t s);

// How a product of n tokens, cols columns and `units` units runs.
enum Mx4Plan {
  MX4_FUSED,   // few tokens: straight from memory, x quantised in LDS
  MX4_DIRECT,  // straight from memory
  MX4_MID,     // 128 x 128 tiles through LDS
  MX4_BIG      // 256 x 256 tiles through LDS
};
constexpr int kMx4MidTile = 128, kMx4BigTile = 256;
// Blocks of x (columns rounded up to 256) up to which each workgroup quantises
// x itself: one launch in place of two (us at 2, 4, 8 x 4096 x 11008: 6.7, 8.4,
// 10.6 against 10.4, 10.9, 11.6; 16 x 2048 x 5632: 5.7 against 7.3).
constexpr int kMx4FusedBlocks = 1024;
inline bool mx4_fused(int64_t n, int cols) { return n <= 16 && n * ((cols + 255) / 256) * 8 <= kMx4FusedBlocks; }
// Multiplications, and results, from either of which tiles through LDS are
// faster than straight from memory: with few columns the stores count, which go
// in whole lines from tiles (us with the quantisation, tiles against straight:
// 64 x 2048 x 5632, 0.74e9, 10.7 against 10.2; 1000 x 2048 x 256, 0.52e9, 11.2
// against 9.3; 32 x 4096 x 11008, 1.4e9, 15.2 against 16.4; 64 x 4096 x 11008,
// 2.9e9, 15.8 against 22.5; without it: 1000 x 128 x 1000, 1.0e6 results, 4.6
// against 3.7; 4000 x 256 x 513, 2.1e6, 5.1 against 8.0; 300 x 256 x 8192,
// 2.5e6, 5.1 against 7.8; 8192 x 128 x 2048 12.2 against 27.6; 16384 x 64 x
// 14336 98 against 348).
constexpr int64_t kMx4TiledWork = 600000000, kMx4TiledResults = 1500000;
inline Mx4Plan mx4_plan(int64_t n, int cols, int units, bool x_is_mx4) {
  if (!x_is_mx4 && mx4_fused(n, cols)) return MX4_FUSED;
  if (n <= 16 || units < kMx4MidTile || (n < kMx4MidTile && cols <= 256)) return MX4_DIRECT;
  if (n * cols < kMx4TiledWork / units && n < kMx4TiledResults / units) return MX4_DIRECT;
  if (n < kMx4BigTile || units < kMx4BigTile) return MX4_MID;
  // 256 x 256 tiles once there are more of them than compute units (us without
  // the quantisation, 256 against 128: 1003 x 1990 x 8100, 128 tiles, 18.1
  // against 14.6; 2048 x 4096 x 11008, 344 tiles, 58.5 against 60.3; 5000 x 2048
  // x 8101, 640 tiles, 52.5 against 55.7; 4096 x 4096 x 11008, 688 tiles, 92
  // against 107; 8192 x 200 x 8192, 1024 tiles, 32.1 against 34.5)
  const int64_t tiles = ((n + 255) / 256) * ((units + 255) / 256);
  return tiles > 256 ? MX4_BIG : MX4_MID;
}
inline bool mx4_tiled(Mx4Plan p) { return p == MX4_MID || p == MX4_BIG; }
// Rows that the arranged scales of x are given: those of one tile at least.
__host__ __device__ inline int64_t mx4_arranged_rows(int64_t n) { return n < kMx4MidTile ? kMx4MidTile : n; }
inline size_t mx4_arranged_bytes(int64_t rows, int cols) { return (size_t)((cols + 255) / 256) * rows * 8; }

// y[i][c] = sum over blocks b of 2^(xs + ws - 254) * sum_k xq wq.
struct Mx4ProductArgs {
  int64_t n;
  int cols, units;
  const uint8_t* x_q;      // MX4 rows of x (not MX4_FUSED)
  const uint8_t* x_scale;  // MX4_DIRECT
  const void* x;           // MX4_FUSED: bf16 / fp32 rows
  int x_bf16;
  const uint8_t* w_q;
  const uint8_t* w_scale;
  const uint8_t* x_arr;    // MX4_MID, MX4_BIG: arranged scales, pitch mx4_arranged_rows(n) and units
  const uint8_t* w_arr;
  void* y;  // [n][units]
  int y_bf16;
};
hipError_t launch_mx4_product(Mx4Plan plan, const Mx4ProductArgs& a, hipStream_t s);

}  // namespace twell
