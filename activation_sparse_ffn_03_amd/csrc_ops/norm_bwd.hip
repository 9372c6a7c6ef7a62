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

// A row is taken by T threads, C chunks of 8 elements each, NT / T rows side
// by side; with one chunk the next rows are on their way while these are
// worked on (with two there are no registers for it).
template <typename TR, typename TG, int NT, int T, int C, int KIND>
__global__ __launch_bounds__(NT) void norm_bwd_kernel(NormBwdArgs a) {
  constexpr int ROWS = NT / T;        // rows a workgroup takes at a time
  constexpr int G = T < 64 ? T : 64;  // lanes of a wave that share a row
  constexpr int WPR = T / G;          // waves of a row
  const int wave = threadIdx.x >> 6, t = threadIdx.x % T;
  const int cols = a.cols;
  // run of rows of this workgroup
  const int64_t per = a.rows / gridDim.x, rem = a.rows % gridDim.x, b = blockIdx.x;
  const int64_t r0 = b * per + (b < rem ? b : rem), r1 = r0 + per + (b < rem ? 1 : 0);
  const bool has_stream = a.d_residual != nullptr;

  struct Row {
    Raw8<TR> r[C], s[C];
    Raw8<TG> g[C];
    float rho;
  };
  auto fetch = [&](int64_t row, Row& x) {
    const int64_t off = row * cols;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      x.r[c].template load<KIND>(static_cast<const TR*>(a.residual) + off, t + T * c, cols);
      x.g[c].template load<KIND>(static_cast<const TG*>(a.d_out) + off, t + T * c, cols);
    }
    if (has_stream) {
#pragma unroll
      for (int c = 0; c < C; ++c) x.s[c].template load<KIND>(static_cast<const TR*>(a.d_residual) + off, t + T * c, cols);
    }
    x.rho = a.rstd[row];
  };
  const int side = threadIdx.x / T;  // which of the rows side by side
  int64_t row = r0 + side;
  constexpr bool AHEAD = C == 1;
  Row now, next;
  if (AHEAD && row < r1) fetch(row, now);

  float w[C][8], dw[C][8];
  load_weight<T, C, KIND>(a.w, a.w_bf16, t, cols, w);
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[c][k] = 0.f;

  __shared__ float red[2][ROWS][WPR];
  int flip = 0;
  for (int64_t first = r0; first < r1; first += ROWS, row += ROWS) {  // the same number of times in every wave
    const bool here = row < r1;
    if constexpr (AHEAD) {
      if (row + ROWS < r1) fetch(row + ROWS, next);
    } else if (here) {
      fetch(row, now);
    }
    float dot = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float xh = now.r[c].get(k) * now.rho, g = now.g[c].get(k);
        if (chunk_counts<KIND>(t + T * c, k, cols)) dot = fmaf(g * w[c][k], xh, dot);
        if (here) dw[c][k] = fmaf(g, xh, dw[c][k]);
      }
    dot = group_sum<G>(dot);
    if constexpr (WPR > 1) {
      // two buffers: a wave may write the next row's sum while another still
      // reads this row's
      if ((threadIdx.x & 63) == 0) red[flip][side][wave % WPR] = dot;
      lds_barrier();
      dot = 0.f;
#pragma unroll
      for (int i = 0; i < WPR; ++i) dot += red[flip][side][i];
      flip ^= 1;
    }
    const float cm = dot / (float)cols;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float d[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float xh = now.r[c].get(k) * now.rho;
        d[k] = now.rho * (now.g[c].get(k) * w[c][k] - xh * cm);
        if (has_stream) d[k] += now.s[c].get(k);
      }
      if (here) store8<KIND>(static_cast<TR*>(a.dr) + row * cols, t + T * c, cols, d);
    }
    if constexpr (AHEAD) now = next;
  }

  float* part = gridDim.x == 1 ? a.dw : a.part + (int64_t)blockIdx.x * cols;
  if constexpr (ROWS > 1) {
    // the sums of the rows taken side by side, added in their order
    __shared__ float acc[ROWS][C][8][T];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[side][c][k][t] = dw[c][k];
    __syncthreads();
    if (side > 0) return;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k)
        for (int i = 1; i < ROWS; ++i) dw[c][k] += acc[i][c][k][t];
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

template <typename TR, typename TG, int NT, int T, int C>
hipError_t launch_cfg(const NormBwdArgs& a, hipStream_t s) {
  const int groups = norm_bwd_groups(a.rows, a.cols);
  row_kind(a.cols, [&](auto kind) {
    constexpr int KIND = decltype(kind)::value;
    if constexpr (KIND != ROWS_SHORT || T == 16)
      TWELL_LAUNCH("add_rms_norm_bwd", (norm_bwd_kernel<TR, TG, NT, T, C, KIND>), dim3(groups), NT, 0, s, a);
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || groups == 1) return e;
  TWELL_LAUNCH("norm_dw_sum", norm_dw_sum, dim3((a.cols + 63) / 64), 1024, 0, s, a.part, groups, a.cols, a.dw);
  return hipGetLastError();
}

// Eight elements a thread, and as many threads a workgroup as keep a compute
// unit's loads in flight (norm_bwd_rows holds NT / T for each width). bf16
// stream and fp32 d_out, both launches, against a wave a row up to 2048 columns
// and a workgroup of four waves a row above without the loads ahead:
// 8192x2048 39.5 : 40.1 us, 512x2048 6.8 : 7.9, 4096x512 8.5 : 9.1, 8192x4096
// 71.2 : 74.4, 2048x128 (fp32) 5.6 : 6.5, 131x1000 (fp32) 5.7 : 6.1; with bf16
// d_out 1119x2688 10.8 : 11.6, 2892x5760 35.1 : 36.0. (8192x2048 has to move
// 168 MB, 34 us at a large copy's rate; the second launch takes 4 of the 39.5.)
// Narrow rows in a wide workgroup pay for adding up their partial sums: 2048x128
// takes 8.5 us with 1024 threads. 1024x16384 (its two chunks a thread) 45.4 us.
template <typename TR, typename TG>
hipError_t launch_typed(const NormBwdArgs& a, hipStream_t s) {
  if (a.cols <= 128) return launch_cfg<TR, TG, 256, 16, 1>(a, s);
  if (a.cols <= 256) return launch_cfg<TR, TG, 256, 32, 1>(a, s);
  if (a.cols <= 512) return launch_cfg<TR, TG, 512, 64, 1>(a, s);
  if (a.cols <= 1024) return launch_cfg<TR, TG, 512, 128, 1>(a, s);
  if (a.cols <= 2048) return launch_cfg<TR, TG, 1024, 256, 1>(a, s);
  if (a.cols <= 4096) return launch_cfg<TR, TG, 1024, 512, 1>(a, s);
  if (a.cols <= 8192) return launch_cfg<TR, TG, 1024, 1024, 1>(a, s);
  return launch_cfg<TR, TG, 1024, 1024, 2>(a, s);
}

}  // namespace

hipError_t launch_add_rms_norm_bwd(const NormBwdArgs& a, hipStream_t s) {
  if (a.res_bf16) return a.g_bf16 ? launch_typed<uint16_t, uint16_t>(a, s) : launch_typed<uint16_t, float>(a, s);
  return a.g_bf16 ? launch_typed<float, uint16_t>(a, s) : launch_typed<float, float>(a, s);
}

}  // namespace twell
