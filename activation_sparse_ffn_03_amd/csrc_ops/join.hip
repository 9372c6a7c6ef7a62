// The join of a block's output y to the residual stream, with norms before and
// after the block:
//
//   v     = y * rho_y * post_w            rho_y = 1 / sqrt(mean(y^2) + eps)   (or v = y)
//   u     = dropout(v)                    (or u = v)
//   r'    = alpha * r + gate * u          rounded to the stream's type as it is stored
//   rho   = 1 / sqrt(mean(r'^2) + eps)
//   n     = r' * rho * w,  out = n in bf16 or fp32,  codes as add_rms_norm's
//
// all in fp32 up to what is stored. The second norm is that of the stream as
// stored, as add_rms_norm's is: with alpha 1 and nothing else asked for this is
// add_rms_norm, bit for bit. v and u are not stored: they are read nowhere else,
// and the backward makes them again from y.
//
// Bound by memory: r and y are read once, r', out and the codes written once;
// the row stays in registers over its four passes. 8192 x 2048, bf16 and an fp32 y,
// 30 us with dropout, 5.6 TB/s, and 26-27 without; 16384 x 4096 with codes 117-125,
// 4.8-5.1; one row 4.1.
#include "counter_rng.h"
#include "norm_device.h"
#include "../csrc/twell_trace.h"

namespace twell {
namespace {

// TR, TY: types of the stream and of y; T threads a row, C chunks each, as in
// norm.hip.
template <int T>
constexpr int join_threads() { return T > 64 ? T : 256; }
template <typename TR, typename TY, int T, int C, int KIND>
__global__ __launch_bounds__(join_threads<T>()) void join_rms_norm_kernel(JoinArgs a) {
  constexpr int G = T < 64 ? T : 64;  // lanes of a wave that share a row
  constexpr int WPR = T / G;          // waves of a row
  const int wave = threadIdx.x >> 6;
  const int64_t row = WPR > 1 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * (256 / T) + threadIdx.x / T;
  if (row >= a.rows) return;  // whole groups of lanes, and with WPR > 1 whole workgroups
  const int t = threadIdx.x % T;
  const int cols = a.cols;
  const int64_t off = row * cols;
  const uint32_t whole_row = (uint32_t)(a.first_row + row);  // rows of the whole array are below 2^31

  Raw8<TR> rr[C];
  Raw8<TY> ry[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    ry[c].template load<KIND>(static_cast<const TY*>(a.y) + off, t + T * c, cols);
    rr[c].template load<KIND>(static_cast<const TR*>(a.residual) + off, t + T * c, cols);
  }
  float w[C][8], x[C][8];
  load_weight<T, C, KIND>(a.w, a.w_bf16, t, cols, w);
  // what u is multiplied with on its way to the stream, and v = y * rho_y * post
  float post[C][8], gate[C][8];
  const bool has_post = a.post_w != nullptr, has_gate = a.gate != nullptr;
  if (has_post) load_weight<T, C, KIND>(a.post_w, a.post_bf16, t, cols, post);
  if (has_gate) {
    const int64_t at = (int64_t)(whole_row / a.per_gate) * cols;
    load_weight<T, C, KIND>(static_cast<const char*>(a.gate) + at * (a.gate_bf16 ? 2 : 4), a.gate_bf16, t, cols, gate);
  }
  uint32_t keep[C];
  if (a.drop != 0) {
    const DropBits bits(DropArgs{a.rng, a.site, a.drop, a.drop_scale});
#pragma unroll
    for (int c = 0; c < C; ++c) keep[c] = bits.chunk<KIND>(whole_row, t + T * c, cols);
  }

  __shared__ float red_sum[4][WPR];
  __shared__ uint32_t red_max[WPR];
  // The row's sum in every thread of it, the same bits in all.
  auto row_sum = [&](float s, float* red) {
    s = group_sum<G>(s);
    if constexpr (WPR > 1) {
      if ((threadIdx.x & 63) == 0) red[wave] = s;
      lds_barrier();
      s = 0.f;
#pragma unroll
      for (int i = 0; i < WPR; ++i) s += red[i];
    }
    return s;
  };
  // Mean of the squares of x, taken again over shrunk elements where their sum
  // overflows (all threads of the row or none).
  auto mean_square = [&](int first) {
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (chunk_counts<KIND>(t + T * c, k, cols)) ss = fmaf(x[c][k], x[c][k], ss);
    ss = row_sum(ss, red_sum[first]);
    if (!(ss > FLT_MAX)) return ss / (float)cols;
    ss = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (chunk_counts<KIND>(t + T * c, k, cols)) ss = fmaf(x[c][k] * kShrink, x[c][k] * kShrink, ss);
    return row_sum(ss, red_sum[first + 1]) * (1.f / (kShrink * kShrink) / (float)cols);
  };

#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int k = 0; k < 8; ++k) x[c][k] = ry[c].get(k);
  if (has_post) {
    const float rho_y = 1.0f / sqrtf(mean_square(0) + a.eps);
    if (a.post_rstd != nullptr && t == 0) a.post_rstd[row] = rho_y;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) x[c][k] = x[c][k] * rho_y * post[c][k];
  }
  if (a.drop != 0) {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) x[c][k] = keep[c] >> k & 1 ? x[c][k] * a.drop_scale : 0.f;
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float r = rr[c].get(k);
      x[c][k] = has_gate ? fmaf(gate[c][k], x[c][k], a.alpha * r) : fmaf(a.alpha, r, x[c][k]);
    }
    if constexpr (std::is_same_v<TR, uint16_t>) {
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        const uint32_t p = pack_bf16(x[c][k], x[c][k + 1]);
        x[c][k] = bf16lo_to_f32(p);
        x[c][k + 1] = bf16hi_to_f32(p);
      }
    }
  }
  const float mean = mean_square(2);
  if (a.residual_out != nullptr) {  // behind the sum: every thread has read its part of the row
#pragma unroll
    for (int c = 0; c < C; ++c) store8<KIND>(static_cast<TR*>(a.residual_out) + off, t + T * c, cols, x[c]);
  }
  const float rho = 1.0f / sqrtf(mean + a.eps);
  if (a.rstd != nullptr && t == 0) a.rstd[row] = rho;

  uint32_t mb = 0;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[c][k] = x[c][k] * rho * w[c][k];
      mb = max(mb, __float_as_uint(x[c][k]) & 0x7FFFFFFFu);
    }
  if (a.out != nullptr) {
    if (a.out_bf16) {
#pragma unroll
      for (int c = 0; c < C; ++c) store8<KIND>(static_cast<uint16_t*>(a.out) + off, t + T * c, cols, x[c]);
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c) store8<KIND>(static_cast<float*>(a.out) + off, t + T * c, cols, x[c]);
    }
  }
  if (a.q == nullptr) return;

  // Elements past the row's end hold 0, or NaN in a row whose rho is NaN.
  mb = group_max<G>(mb);
  if constexpr (WPR > 1) {
    if ((threadIdx.x & 63) == 0) red_max[wave] = mb;
    lds_barrier();
#pragma unroll
    for (int i = 0; i < WPR; ++i) mb = max(mb, red_max[i]);
  }
  float sc = __uint_as_float(mb) / 448.0f;
  sc = sc > 0.f ? sc : 1.0f;  // NaN fails the test
  if (t == 0) a.q_scale[row] = sc;
  auto encode = [&](auto fast) {
#pragma unroll
    for (int c = 0; c < C; ++c) store8<KIND>(a.q + off, t + T * c, cols, encode8<decltype(fast)::value>(x[c], sc));
  };
  if (mb < 0x7F800000u && mb >= kNormalScaleBits)
    encode(std::true_type{});
  else
    encode(std::false_type{});
}

template <typename TR, typename TY, int T, int C>
hipError_t launch_cfg(const JoinArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)(T > 64 ? a.rows : (a.rows + 256 / T - 1) / (256 / T)));
  return row_kind(a.cols, [&](auto kind) {
    constexpr int KIND = decltype(kind)::value;
    if constexpr (KIND != ROWS_SHORT || T == 16)
      TWELL_LAUNCH("join_rms_norm", (join_rms_norm_kernel<TR, TY, T, C, KIND>), grid, join_threads<T>(), 0, s, a);
    return hipGetLastError();
  });
}

template <typename TR, typename TY>
hipError_t launch_typed(const JoinArgs& a, hipStream_t s) {
  const int n = a.cols;
  if (n <= 128) return launch_cfg<TR, TY, 16, 1>(a, s);
  if (n <= 256) return launch_cfg<TR, TY, 32, 1>(a, s);
  if (n <= 512) return launch_cfg<TR, TY, 64, 1>(a, s);
  if (n <= 1024) return launch_cfg<TR, TY, 128, 1>(a, s);
  if (n <= 2048) return launch_cfg<TR, TY, 256, 1>(a, s);
  if (n <= 4096) return launch_cfg<TR, TY, 512, 1>(a, s);
  if (n <= 8192) return launch_cfg<TR, TY, 512, 2>(a, s);
  return launch_cfg<TR, TY, 512, 4>(a, s);
}

hipError_t launch_rows(const JoinArgs& a, hipStream_t s) {
  if (a.res_bf16) return a.y_bf16 ? launch_typed<uint16_t, uint16_t>(a, s) : launch_typed<uint16_t, float>(a, s);
  return a.y_bf16 ? launch_typed<float, uint16_t>(a, s) : launch_typed<float, float>(a, s);
}

}  // namespace

// A launch holds less than 2^32 threads, up to 512 for a row: more rows than
// that allows take several.
hipError_t launch_join_rms_norm(const JoinArgs& all, hipStream_t s) {
  constexpr int64_t kLaunchRows = 1 << 22;
  JoinArgs a = all;
  auto skip = [&](auto*& p, size_t bytes_a_row) {
    using P = std::remove_reference_t<decltype(p)>;
    if (p != nullptr)
      p = reinterpret_cast<P>(reinterpret_cast<uintptr_t>(p) + kLaunchRows * bytes_a_row);
  };
  const size_t er = a.res_bf16 ? 2 : 4, ey = a.y_bf16 ? 2 : 4, eo = a.out_bf16 ? 2 : 4, cols = (size_t)a.cols;
  for (int64_t left = all.rows; left > 0; left -= kLaunchRows) {
    a.rows = left < kLaunchRows ? left : kLaunchRows;
    const hipError_t e = launch_rows(a, s);
    if (e != hipSuccess) return e;
    a.first_row += kLaunchRows;
    skip(a.residual, cols * er);
    skip(a.y, cols * ey);
    skip(a.residual_out, cols * er);
    skip(a.out, cols * eo);
    skip(a.q, cols);
    skip(a.q_scale, 4);
    skip(a.rstd, 4);
    skip(a.post_rstd, 4);
  }
  return hipSuccess;
}

}  // namespace twell
