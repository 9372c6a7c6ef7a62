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
  MX4_FUSED,   // straight from memory, x quantised in LDS
  MX4_DIRECT,  // straight from memory
  MX4_MID,     // 128 x 128 tiles through LDS
  MX4_BIG      // 256 x 256 tiles through LDS
};
constexpr int kMx4MidTile = 128, kMx4BigTile = 256;
// Estimates (us, beside about 3 that every product takes) for straight from
// memory in tiles of 16 f x 16 f and for tiles through LDS. A tile goes through
// its columns in stages of 256, at what a stage takes a workgroup that has a
// compute unit to itself, and all tiles together read their rows at about
// 5 MB/us; tiles through LDS also have their scales arranged. Measured without
// the quantisation (us; f = 1, 2, 4, then LDS):
//   32 x 7442 x 799      5.5  9.3 16.3  17.9     300 x 2048 x 256    4.8  5.2  9.1  6.8
//   352 x 7541 x 448    11.8  9.5 17.0  18.5     400 x 3776 x 448    9.8  7.8 13.9  9.4
//   24 x 2048 x 5632     6.3  5.1  8.1   6.8     88 x 5603 x 3552   20.9 14.7 16.6 12.5
//   128 x 5504 x 5119   24.0 16.1 13.7  14.9     64 x 4096 x 11008  31.3 18.6 14.8 10.4
//   1208 x 1984 x 1024  27.7 16.1 14.9   7.2     864 x 4672 x 2395  70.3 36.5 29.7 15.0
//   300 x 256 x 8192       -  7.8  8.4   5.1     1000 x 128 x 1000     -  3.7  4.5  4.6
//   100000 x 1024 x 64  69.5 37.6 26.4     -     8192 x 128 x 2048     - 31.3 27.7 12.2
inline double mx4_direct_us(int64_t n, int cols, int units, int f) {
  const double tiles = (double)((n + 16 * f - 1) / (16 * f)) * ((units + 16 * f - 1) / (16 * f));
  const int count = (cols + 255) / 256;
  const double stages = f == 1 ? 0.085 * count : f == 2 ? 0.2 * count : 2 + 0.5 * count;
  const double reads = tiles * 32 * f * mx4_code_bytes(cols) / 5e6;
  return stages > reads ? stages : reads;
}
inline double mx4_tiled_us(int64_t n, int cols, int units) {
  const double tiles = (double)((n + 127) / 128) * ((units + 127) / 128);
  return 1.3 + 0.47 * ((cols + 255) / 256) * (tiles > 256 ? tiles / 256 : 1);
}
inline int mx4_direct_tile(int64_t n, int cols, int units) {  // f of the fastest
  int best = 1;
  for (int f = 2; f <= 4; f *= 2)
    if (mx4_direct_us(n, cols, units, f) < mx4_direct_us(n, cols, units, best)) best = f;
  return best;
}
// A product that quantises x itself: one launch in place of two, and each
// workgroup quantises the rows of its tile (16 tokens, or 32 where there are
// more) into LDS, up to this many blocks (columns rounded up to 256). With the
// waves' sums that is 58 KB, two workgroups a compute unit. The edge is a middle
// between two shapes (us, one launch against two): long rows of up to 16 tokens
// lose before it (5, 8, 12, 13, 16 x 4096 x 11008 10.2, 11.3, 13.4, 13.7, 15.0
// against 11.7, 12.3, 13.0, 13.2, 13.7; 8, 12, 13, 16 x 4096 x 4096 6.7, 7.8,
// 8.1, 8.6 against 7.0, 7.3, 7.3, 7.6: equal at about 1300 blocks), shorter rows
// of more tokens win beyond it, too (17, 20, 24 x 2048 x 5632 6.0, 6.1, 6.8
// against 7.2, 7.4, 7.5; 25, 28, 32, which take two launches, 7.0, 7.3, 7.7
// against 7.4, 7.7, 7.8).
constexpr int kMx4FusedBlocks = 1536;
inline int mx4_fused_blocks(int64_t n, int cols) { return (int)(n < 32 ? n : 32) * ((cols + 255) / 256) * 8; }
// Up to 16 tokens wherever x fits (us, against two launches: 2, 4 x 4096 x 11008
// 6.7, 8.4 against 10.4, 10.9; 16 x 3000 x 5632 7.3 against 9.1; 16 x 2048 x 5632
// 5.4 against 7.3; it loses up to 0.5 just below the edge, see there), above by
// estimate: 512 blocks at a time, again and again where there are more workgroups
// than compute units, against 2.5 for a launch (us, against two launches: 24 x
// 1024 x 4096 4.5 : 6.2, 32 x 1024 x 4096 5.0 : 6.4, 60 x 1500 x 1500 7.0 : 7.4,
// 64 x 2048 x 5632 12.0 : 10.7, 100 x 1024 x 4096 7.6 : 8.4, 200 x 512 x 1024
// 4.2 : 6.3).
inline bool mx4_fused(int64_t n, int cols, int units, double two_launches_us) {
  if (mx4_fused_blocks(n, cols) > kMx4FusedBlocks) return false;
  if (n <= 16) return true;
  const double groups = (double)((n + 31) / 32) * ((units + 31) / 32);
  const double stages = 0.2 * ((cols + 255) / 256), reads = groups * 32 * mx4_code_bytes(cols) / 5e6;
  const double rounds = (mx4_fused_blocks(n, cols) + 511) / 512 * (groups > 256 ? groups / 256 : 1);
  return (stages > reads ? stages : reads) + 0.9 * rounds <= two_launches_us + 2.5;
}
inline Mx4Plan mx4_plan(int64_t n, int cols, int units, bool x_is_mx4) {
  const double direct = mx4_direct_us(n, cols, units, mx4_direct_tile(n, cols, units));
  // tiles need their rows, units and two stages of columns; up to 16 tokens most of a tile would be left empty
  const bool tiles_fit = n > 16 && units >= kMx4MidTile && (n >= kMx4MidTile || cols > 256);
  const double tiled = tiles_fit ? mx4_tiled_us(n, cols, units) : direct;
  if (!x_is_mx4 && mx4_fused(n, cols, units, direct < tiled ? direct : tiled)) return MX4_FUSED;
  if (direct <= tiled) return MX4_DIRECT;
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
