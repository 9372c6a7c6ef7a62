// Dropout: out = x * 65536 / (65536 - drop) where the generator keeps an
// element (counter_rng.h), 0 where it drops it, whatever x holds there. The
// product is fp32, rounded once for bf16. Its gradient is the same call on the
// gradient with the same seed, step and site.
//
// Bound by memory (x read and written once) as long as the generator's 20
// 64-bit products a chunk of 8 elements stay below it: 8192 x 2048 in bf16 11.4 us,
// 5.9 TB/s, in fp32 21.5, 6.2; 61 x 999 2.5.
#include "counter_rng.h"
#include "ops_kernels.h"
#include "../csrc/twell_trace.h"

namespace twell {
namespace {

// A workgroup of 256 threads takes 256 / T rows of T threads, U chunks each;
// workgroups along a row are numbered first. Chunks are taken as they are and
// not moved back, since out may be x: two threads must not both read and write
// an element.
template <typename TX, int T, int U, bool TAIL>
__global__ __launch_bounds__(256) void dropout_kernel(DropoutArgs a, uint32_t across) {
  constexpr int R = 256 / T;
  const uint32_t down = blockIdx.x / across;
  const int first = (int)(blockIdx.x - down * across) * (T * U) + threadIdx.x % T;
  const int64_t row = (int64_t)down * R + threadIdx.x / T;
  if (row >= a.rows) return;
  const TX* x = static_cast<const TX*>(a.x) + row * a.cols;
  TX* out = static_cast<TX*>(a.out) + row * a.cols;
  Raw8<TX> raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (8 * (first + T * u) < a.cols) raw[u].template load_filled<TAIL>(x, first + T * u, a.cols);
  const DropBits bits(DropArgs{a.rng, a.site, a.drop, a.drop_scale});
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = first + T * u;
    if (8 * i >= a.cols) break;
    const uint32_t keep = bits.group(a.first_row + (uint32_t)row, i);
    raw[u].template settle<TAIL>(i, a.cols);
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = keep >> k & 1 ? raw[u].get(k) * a.drop_scale : 0.f;
    store8_exact<TAIL>(out, i, a.cols, v);
  }
}

template <typename TX, int T, int U>
hipError_t launch_cfg(DropoutArgs a, hipStream_t s) {
  const int chunks = (a.cols + 7) / 8;
  const uint32_t across = (uint32_t)((chunks + T * U - 1) / (T * U));
  // less than 2^32 threads a launch
  const int64_t most = ((1 << 24) - 1) / across * (256 / T);
  for (int64_t left = a.rows; left > 0; left -= most) {
    a.rows = left < most ? left : most;
    const dim3 grid((unsigned)((a.rows + 256 / T - 1) / (256 / T)) * across);
    if (a.cols % 8 == 0)
      TWELL_LAUNCH("dropout", (dropout_kernel<TX, T, U, false>), grid, 256, 0, s, a, across);
    else
      TWELL_LAUNCH("dropout", (dropout_kernel<TX, T, U, true>), grid, 256, 0, s, a, across);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    a.first_row += (uint32_t)most;
    a.x = static_cast<const TX*>(a.x) + most * a.cols;
    a.out = static_cast<TX*>(a.out) + most * a.cols;
  }
  return hipSuccess;
}

template <typename TX>
hipError_t launch_typed(const DropoutArgs& a, hipStream_t s) {
  const int n = a.cols;
  if (n <= 64) return launch_cfg<TX, 8, 1>(a, s);
  if (n <= 256) return launch_cfg<TX, 32, 1>(a, s);
  if (n <= 1024) return launch_cfg<TX, 128, 1>(a, s);
  return launch_cfg<TX, 256, 1>(a, s);
}

}  // namespace

hipError_t launch_dropout(const DropoutArgs& a, hipStream_t s) {
  return a.bf16 ? launch_typed<uint16_t>(a, s) : launch_typed<float>(a, s);
}

}  // namespace twell
