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
// Row width up to which the backward gives a row to one wave (above: to a
// workgroup of four).
constexpr int kNormBwdWaveCols = 2048;
// Workgroups of the norm's backward; each keeps one partial dw row. Two a
// compute unit, and no more than there are rows for.
inline int norm_bwd_groups(int64_t rows, int cols) {
  const int64_t need = cols <= kNormBwdWaveCols ? (rows + 3) / 4 : rows;
  return (int)(need < 1 ? 1 : need > 512 ? 512 : need);
}
hipError_t launch_add_rms_norm_bwd(const NormBwdArgs& a, hipStream_t s);

// MX4 rows: 64 bytes of codes for every 128 columns begun, 16 scale bytes for
// every 512 begun.
constexpr int kMx4MaxCols = 1 << 20;
__host__ __device__ inline int mx4_code_bytes(int cols) { return (cols + 127) / 128 * 64; }
__host__ __device__ inline int mx4_scale_bytes(int cols) { return (cols + 511) / 512 * 16; }
hipError_t launch_quantize_mx4(const void* in, int is_bf16, int64_t rows, int cols, uint8_t* q, uint8_t* scale,
                               hipStream_t s);
hipError_t launch_dequantize_mx4(const uint8_t* q, const uint8_t* scale, int64_t rows, int cols, int out_bf16,
                                 void* out, hipStream_t s);

// y[i][c] = sum over blocks b of 2^(xs + ws - 254) * sum_k xq wq. Either x_q
// and x_scale hold x's MX4 rows, or x holds bf16 / fp32 rows that the kernel
// quantises itself (mx4_product_quantises).
struct Mx4ProductArgs {
  int64_t n;
  int cols, units;
  const uint8_t* x_q;
  const uint8_t* x_scale;
  const void* x;  // null: x_q and x_scale
  int x_bf16;
  const uint8_t* w_q;
  const uint8_t* w_scale;
  void* y;  // [n][units]
  int y_bf16;
};
// Tokens up to which the product quantises x in its registers.
constexpr int kMx4FusedTokens = 16;
inline bool mx4_product_quantises(int64_t n) { return n <= kMx4FusedTokens; }
hipError_t launch_mx4_product(const Mx4ProductArgs& a, hipStream_t s);

}  // namespace twell
