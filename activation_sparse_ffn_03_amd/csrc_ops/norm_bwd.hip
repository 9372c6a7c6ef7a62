// Backward of the residual-adding RMS norm.
//
// With xh = r' * rho, u = d_out * w and c = mean(u * xh):
//   dr = d_residual + rho * (u - xh * c)   (the gradient of the stream and of what was added to it)
//   dw = sum over rows of d_out * xh
//
// Bound by memory: one pass over d_out, r' and d_residual. A workgroup takes a
// run of consecutive rows, keeps its part of dw in registers (thread t owns the
// same columns in every row) and leaves one partial row; a second launch adds
// the partial rows in a fixed order, so dw does not change from run to run.
#include "chunk8.h"
#include "ops_kernels.h"
#include "../csrc/twell_trace.h"

namespace twell {
namespace {

constexpr int kThreads = 256;

template <typename TR, typename TG, int WPR, int C, int KIND>
__global__ __launch_bounds__(kThreads) void norm_bwd_kernel(NormBwdArgs a) {
  constexpr int T = 64 * WPR;
  constexpr int RPI = 4 / WPR;  // rows a workgroup takes at a time
  const int wave = threadIdx.x >> 6;
  const int t = WPR == 1 ? (int)(threadIdx.x & 63) : (int)threadIdx.x;
  const int cols = a.cols;
  // run of rows of this workgroup
  const int64_t per = a.rows / gridDim.x, rem = a.rows % gridDim.x, b = blockIdx.x;
  const int64_t r0 = b * per + (b < rem ? b : rem), r1 = r0 + per + (b < rem ? 1 : 0);

  float w[C][8], dw[C][8];
  load_weight<T, C, KIND>(a.w, a.w_bf16, t, cols, w);
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[c][k] = 0.f;

  __shared__ float red[2][4];
  int flip = 0;
  for (int64_t row = r0 + (WPR == 1 ? wave : 0); row < r1; row += RPI) {
    const int64_t off = row * cols;
    Raw8<TR> rr[C], rs[C];
    Raw8<TG> rg[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      rr[c].template load<KIND>(static_cast<const TR*>(a.residual) + off, t + T * c, cols);
      rg[c].template load<KIND>(static_cast<const TG*>(a.d_out) + off, t + T * c, cols);
    }
    if (a.d_residual != nullptr) {
#pragma unroll
      for (int c = 0; c < C; ++c)
        rs[c].template load<KIND>(static_cast<const TR*>(a.d_residual) + off, t + T * c, cols);
    }
    const float rho = a.rstd[row];
    float dot = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float xh = rr[c].get(k) * rho, g = rg[c].get(k);
        if (chunk_counts<KIND>(t + T * c, k, cols)) dot = fmaf(g * w[c][k], xh, dot);
        dw[c][k] = fmaf(g, xh, dw[c][k]);
      }
    dot = wave_sum_dpp(dot);
    if constexpr (WPR > 1) {
      // two buffers: a wave may write the next row's sum while another still
      // reads this row's
      if ((threadIdx.x & 63) == 0) red[flip][wave] = dot;
      lds_barrier();
      dot = red[flip][0] + red[flip][1] + red[flip][2] + red[flip][3];
      flip ^= 1;
    }
    const float cm = dot / (float)cols;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float d[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float xh = rr[c].get(k) * rho;
        d[k] = rho * (rg[c].get(k) * w[c][k] - xh * cm);
        if (a.d_residual != nullptr) d[k] += rs[c].get(k);
      }
      store8<KIND>(static_cast<TR*>(a.dr) + off, t + T * c, cols, d);
    }
  }

  float* part = gridDim.x == 1 ? a.dw : a.part + (int64_t)blockIdx.x * cols;
  if constexpr (WPR == 1) {
    // the four waves' sums, added in the order of the waves
    __shared__ float acc[C][8][64];
    for (int v = 0; v < 4; ++v) {
      if (wave == v) {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if (v > 0) dw[c][k] += acc[c][k][t];
            acc[c][k][t] = dw[c][k];
          }
      }
      __syncthreads();
    }
    if (wave < 3) return;  // the last wave holds the sums
  }
#pragma unroll
  for (int c = 0; c < C; ++c) store8<KIND>(part, t + T * c, cols, dw[c]);
}

// dw[col] = sum over the partial rows: a workgroup takes 64 columns, each of
// its 16 waves every 16th row in ascending order, then the 16 sums in order.
__global__ __launch_bounds__(1024) void norm_dw_sum(const float* __restrict__ part, int groups, int cols,
                                                    float* __restrict__ dw) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + lane;
  float s = 0.f;
  if (col < cols) {
#pragma unroll 8
    for (int g = wave; g < groups; g += 16) s += part[(int64_t)g * cols + col];
  }
  red[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && col < cols) {
    for (int i = 1; i < 16; ++i) s += red[i][lane];
    dw[col] = s;
  }
}

template <typename TR, typename TG, int WPR, int C>
hipError_t launch_cfg(const NormBwdArgs& a, hipStream_t s) {
  const int groups = norm_bwd_groups(a.rows, a.cols);
  row_kind(a.cols, [&](auto kind) {
    constexpr int KIND = decltype(kind)::value;
    if constexpr (KIND != ROWS_SHORT || (WPR == 1 && C == 1))
      TWELL_LAUNCH("add_rms_norm_bwd", (norm_bwd_kernel<TR, TG, WPR, C, KIND>), dim3(groups), kThreads, 0, s, a);
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || groups == 1) return e;
  TWELL_LAUNCH("norm_dw_sum", norm_dw_sum, dim3((a.cols + 63) / 64), 1024, 0, s, a.part, groups, a.cols, a.dw);
  return hipGetLastError();
}

template <typename TR, typename TG>
hipError_t launch_typed(const NormBwdArgs& a, hipStream_t s) {
  if (a.cols <= 512) return launch_cfg<TR, TG, 1, 1>(a, s);
  if (a.cols <= 1024) return launch_cfg<TR, TG, 1, 2>(a, s);
  if (a.cols <= kNormBwdWaveCols) return launch_cfg<TR, TG, 1, 4>(a, s);
  if (a.cols <= 4096) return launch_cfg<TR, TG, 4, 2>(a, s);
  if (a.cols <= 8192) return launch_cfg<TR, TG, 4, 4>(a, s);
  return launch_cfg<TR, TG, 4, 8>(a, s);
}

}  // namespace

hipError_t launch_add_rms_norm_bwd(const NormBwdArgs& a, hipStream_t s) {
  if (a.res_bf16) return a.g_bf16 ? launch_typed<uint16_t, uint16_t>(a, s) : launch_typed<uint16_t, float>(a, s);
  return a.g_bf16 ? launch_typed<float, uint16_t>(a, s) : launch_typed<float, float>(a, s);
}

}  // namespace twell
