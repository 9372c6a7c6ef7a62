// Root-mean-square norm with the residual's addition and an E4M3 output.
//
//   r'    = residual + delta              (fp32 sum, rounded to the stream's type as it is stored)
//   rho   = 1 / sqrt(mean(r'^2) + eps)    (fp32)
//   n     = r' * rho * w                  (fp32)
//   out   = n in bf16 or fp32
//   scale = max|n| / 448 (1 when that is not > 0), q = E4M3(n / scale)
//
// The norm is that of the residual as stored, so that the backward, which
// reads the stored residual, differentiates exactly what was computed, and so
// that adding first and norming later give the same. The codes come from the
// fp32 n and not from the rounded out: one rounding, and for an fp32 out they
// are bit for bit those of quantising it. The sum of squares is held in fp32;
// where it overflows (a row of 16384 equal elements from 1.5e17 on) it is taken
// again over elements scaled down, so that only a mean of squares beyond fp32 (a
// root mean square above 1.8e19) gives a norm of 0.
//
// Bound by memory: the stream and the addition are read once, the new stream,
// out and the codes written once; the row stays in registers between its three
// passes (sum of squares, largest magnitude, encoding).
#include "norm_device.h"
#include "ops_kernels.h"
#include "../csrc/twell_trace.h"

namespace twell {
namespace {

// TR: the stream's type; TD: the addition's (void: none). A row is taken by T
// threads, C chunks of 8 elements each: up to 64 threads several rows share a
// workgroup of four waves and need no barrier, above that a row has one of its
// own.
template <int T>
constexpr int norm_threads() { return T > 64 ? T : 256; }
template <typename TR, typename TD, int T, int C, int KIND>
__global__ __launch_bounds__(norm_threads<T>()) void add_rms_norm_kernel(NormArgs a) {
  constexpr bool ADD = !std::is_void_v<TD>;
  using TDs = std::conditional_t<ADD, TD, TR>;
  constexpr int G = T < 64 ? T : 64;  // lanes of a wave that share a row
  constexpr int WPR = T / G;          // waves of a row
  const int wave = threadIdx.x >> 6;
  const int64_t row = WPR > 1 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * (256 / T) + threadIdx.x / T;
  if (row >= a.rows) return;  // whole groups of lanes, and with WPR > 1 whole workgroups
  const int t = threadIdx.x % T;
  const int cols = a.cols;
  const int64_t off = row * cols;

  Raw8<TR> rr[C];
  Raw8<TDs> rd[ADD ? C : 1];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    rr[c].template load<KIND>(static_cast<const TR*>(a.residual) + off, t + T * c, cols);
    if constexpr (ADD) rd[c].template load<KIND>(static_cast<const TD*>(a.delta) + off, t + T * c, cols);
  }
  float w[C][8];
  load_weight<T, C, KIND>(a.w, a.w_bf16, t, cols, w);

  float x[C][8];
  float ss = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[c][k] = rr[c].get(k);
      if constexpr (ADD) x[c][k] += rd[c].get(k);
    }
    if constexpr (ADD && std::is_same_v<TR, uint16_t>) {
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        const uint32_t p = pack_bf16(x[c][k], x[c][k + 1]);
        x[c][k] = bf16lo_to_f32(p);
        x[c][k + 1] = bf16hi_to_f32(p);
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (chunk_counts<KIND>(t + T * c, k, cols)) ss = fmaf(x[c][k], x[c][k], ss);
  }
  __shared__ float red_sum[2][WPR];
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
  ss = row_sum(ss, red_sum[0]);
  float mean = ss / (float)cols;
  if (ss > FLT_MAX) {  // all threads of the row or none
    ss = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (chunk_counts<KIND>(t + T * c, k, cols)) ss = fmaf(x[c][k] * kShrink, x[c][k] * kShrink, ss);
    mean = row_sum(ss, red_sum[1]) * (1.f / (kShrink * kShrink) / (float)cols);
  }
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

  // Elements past the row's end hold 0 * rho * 0: 0, or NaN in a row whose rho
  // is not finite, which cannot be (eps > 0) unless the row itself holds NaN.
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

template <typename TR, typename TD, int T, int C>
hipError_t launch_cfg(const NormArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)(T > 64 ? a.rows : (a.rows + 256 / T - 1) / (256 / T)));
  return row_kind(a.cols, [&](auto kind) {
    constexpr int KIND = decltype(kind)::value;
    if constexpr (KIND != ROWS_SHORT || T == 16)
      TWELL_LAUNCH("add_rms_norm", (add_rms_norm_kernel<TR, TD, T, C, KIND>), grid, norm_threads<T>(), 0, s, a);
    return hipGetLastError();
  });
}

// As many threads as there are chunks, up to 512, then several chunks a thread
// (us, other counts beside the chosen one: 16384 x 95 bf16 with codes 16
// threads 5.4, 32 7.0, 64 10.3; 8192 x 768 128 threads 11.9, 64 12.2, 256 14.5;
// 7248 x 1135 256 threads 10.3, 128 10.7, 512 13.7; 4096 x 2048 fp32 256
// threads 25.5, 128 27.2, 64 28.3; 16384 x 4096 bf16 512 threads 103, 256 105,
// 64 115; 1 x 4096 512 threads 2.9, 256 3.1, 128 3.8).
template <typename TR, typename TD>
hipError_t launch_typed(const NormArgs& a, hipStream_t s) {
  const int n = a.cols;
  if (n <= 128) return launch_cfg<TR, TD, 16, 1>(a, s);
  if (n <= 256) return launch_cfg<TR, TD, 32, 1>(a, s);
  if (n <= 512) return launch_cfg<TR, TD, 64, 1>(a, s);
  if (n <= 1024) return launch_cfg<TR, TD, 128, 1>(a, s);
  if (n <= 2048) return launch_cfg<TR, TD, 256, 1>(a, s);
  if (n <= 4096) return launch_cfg<TR, TD, 512, 1>(a, s);
  if (n <= 8192) return launch_cfg<TR, TD, 512, 2>(a, s);
  return launch_cfg<TR, TD, 512, 4>(a, s);
}

}  // namespace

static hipError_t launch_rows(const NormArgs& a, hipStream_t s) {
  if (a.res_bf16) {
    if (a.delta == nullptr) return launch_typed<uint16_t, void>(a, s);
    return a.delta_bf16 ? launch_typed<uint16_t, uint16_t>(a, s) : launch_typed<uint16_t, float>(a, s);
  }
  if (a.delta == nullptr) return launch_typed<float, void>(a, s);
  return a.delta_bf16 ? launch_typed<float, uint16_t>(a, s) : launch_typed<float, float>(a, s);
}

// A launch holds less than 2^32 threads, up to 512 for a row: more rows than
// that allows take several.
hipError_t launch_add_rms_norm(const NormArgs& all, hipStream_t s) {
  constexpr int64_t kLaunchRows = 1 << 22;
  NormArgs a = all;
  auto skip = [&](auto*& p, size_t bytes_a_row) {
    using P = std::remove_reference_t<decltype(p)>;
    if (p != nullptr)
      p = reinterpret_cast<P>(reinterpret_cast<uintptr_t>(p) + kLaunchRows * bytes_a_row);
  };
  const size_t er = a.res_bf16 ? 2 : 4, ed = a.delta_bf16 ? 2 : 4, eo = a.out_bf16 ? 2 : 4, cols = (size_t)a.cols;
  for (int64_t left = all.rows; left > 0; left -= kLaunchRows) {
    a.rows = left < kLaunchRows ? left : kLaunchRows;
    const hipError_t e = launch_rows(a, s);
    if (e != hipSuccess) return e;
    skip(a.residual, cols * er);
    skip(a.delta, cols * ed);
    skip(a.residual_out, cols * er);
    skip(a.out, cols * eo);
    skip(a.q, cols);
    skip(a.q_scale, 4);
    skip(a.rstd, 4);
  }
  return hipSuccess;
}

}  // namespace twell
