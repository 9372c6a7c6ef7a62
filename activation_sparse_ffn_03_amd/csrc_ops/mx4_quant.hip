// MX4 quantisation of rows and back.
//
// A row of cols elements becomes 64 bytes of codes for every 128 columns begun
// (the depth of the scaled matrix instruction) and 16 scale bytes for every 512
// begun, zeros behind the last column: the products read whole 16-byte pieces
// of both and need no tail.
//
// A wave takes 512 columns of a row, eight a lane: loads and stores are
// contiguous over the wave, and a block lies in four neighbouring lanes, whose
// largest magnitude two lane swaps find. Bound by memory: 2 or 4 bytes read and
// 17/32 written per element, and the other way round.
#include "mx4_device.h"
#include "ops_kernels.h"
#include "../csrc/twell_trace.h"

namespace twell {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;  // 512-column pieces a wave has in flight

// The 512-column pieces of this wave: kUnits in a row, in row-major order.
struct Units {
  int64_t row[kUnits], rows;
  int seg[kUnits];
  __device__ __forceinline__ Units(int64_t rows_, int cols) : rows(rows_) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int segs = (cols + 511) / 512;
    const int64_t u = ((int64_t)blockIdx.x * (kThreads / 64) + wave) * kUnits;
    row[0] = u / segs;
    seg[0] = (int)(u - row[0] * segs);
#pragma unroll
    for (int k = 1; k < kUnits; ++k) {
      const bool next = seg[k - 1] + 1 == segs;
      row[k] = row[k - 1] + next;
      seg[k] = next ? 0 : seg[k - 1] + 1;
    }
  }
  __device__ __forceinline__ bool valid(int k) const { return row[k] < rows; }
};

// One row's scale codes of 512 columns (16 bytes) to their places in the two
// stages; threads of a wave take neighbouring rows, whose 8 bytes lie together.
__device__ __forceinline__ void arrange(const Mx4Arrange& a, int64_t i, int cols) {
  const int segs = (cols + 511) / 512;
  const int64_t seg = i / a.rows, r = i - seg * a.rows;
  if (seg >= segs) return;
  const u32x4_t v = *reinterpret_cast<const u32x4_t*>(a.scale + (r * segs + seg) * 16);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t stage = 2 * seg + h;
    if (256 * stage >= cols) return;
    *reinterpret_cast<uint2*>(a.out + (stage * a.pitch + r) * 8) =
        uint2{__builtin_amdgcn_perm(v[2 * h + 1], v[2 * h], 0x06040200u),
              __builtin_amdgcn_perm(v[2 * h + 1], v[2 * h], 0x07050301u)};
  }
}
unsigned arrange_blocks(const Mx4Arrange& a, int cols) {
  return (unsigned)((a.rows * ((cols + 511) / 512) + kThreads - 1) / kThreads);
}

__global__ __launch_bounds__(kThreads) void mx4_arrange_kernel(Mx4Arrange a, Mx4Arrange b, unsigned blocks_a, int cols) {
  if (blockIdx.x < blocks_a)
    arrange(a, (int64_t)blockIdx.x * kThreads + threadIdx.x, cols);
  else
    arrange(b, (int64_t)(blockIdx.x - blocks_a) * kThreads + threadIdx.x, cols);
}

// Workgroups from `blocks` on arrange `also`.
template <typename TS, bool TAIL>
__global__ __launch_bounds__(kThreads) void mx4_quantize_kernel(const TS* __restrict__ in, int64_t rows, int cols,
                                                                uint8_t* __restrict__ q, uint8_t* __restrict__ scale,
                                                                uint8_t* __restrict__ arranged, int64_t pitch,
                                                                unsigned blocks, Mx4Arrange also) {
  if (blockIdx.x >= blocks) {
    arrange(also, (int64_t)(blockIdx.x - blocks) * kThreads + threadIdx.x, cols);
    return;
  }
  const int lane = threadIdx.x & 63;
  const int cbytes = mx4_code_bytes(cols), sbytes = mx4_scale_bytes(cols);
  Units u(rows, cols);
  Raw8<TS> raw[kUnits];
#pragma unroll
  for (int k = 0; k < kUnits; ++k)
    raw[k].template load_filled<TAIL>(in + u.row[k] * cols, 64 * u.seg[k] + lane, u.valid(k) ? cols : 0);
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    if (!u.valid(k)) return;
    raw[k].template settle<TAIL>(64 * u.seg[k] + lane, cols);
    uint32_t m = raw[k].max_bits();
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, false));  // lanes 1 0 3 2
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, false));  // lanes 2 3 0 1
    const uint32_t code = mx4_scale_code(m);
    const uint32_t c = code == 255u ? 0u : mx4_codes(raw[k], mx4_scale_operand(code));
    const int at = 256 * u.seg[k] + 4 * lane;  // of the row's code bytes
    if (at < cbytes) *reinterpret_cast<uint32_t*>(q + u.row[k] * cbytes + at) = c;
    // blocks behind the row's last hold zeros: code 0
    if ((lane & 3) == 0) {
      const int b = lane / 4;
      if (arranged == nullptr) {
        scale[u.row[k] * sbytes + 16 * u.seg[k] + b] = (uint8_t)code;
      } else {
        const int64_t stage = 2 * u.seg[k] + b / 8;
        if (256 * stage < cols) arranged[(stage * pitch + u.row[k]) * 8 + 4 * (b & 1) + b / 2 % 4] = (uint8_t)code;
      }
    }
  }
}

// Value of code n of w over the block's scale factor.
__device__ __forceinline__ void mx4_values(uint32_t w, float s, float (&x)[8]) {
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    const uint32_t b = (w >> (4 * k)) & 0xFFu;
    const f32x2_t v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(b, 1.0f, 0);
    x[k] = v[0] * s;
    x[k + 1] = v[1] * s;
  }
}

template <typename TS, bool TAIL>
__global__ __launch_bounds__(kThreads) void mx4_dequantize_kernel(const uint8_t* __restrict__ q,
                                                                  const uint8_t* __restrict__ scale, int64_t rows,
                                                                  int cols, TS* __restrict__ out) {
  const int lane = threadIdx.x & 63;
  const int cbytes = mx4_code_bytes(cols), sbytes = mx4_scale_bytes(cols);
  Units u(rows, cols);
  uint32_t w[kUnits], sc[kUnits];
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    const bool in = u.valid(k) && 512 * u.seg[k] + 8 * lane < cols;
    w[k] = in ? *reinterpret_cast<const uint32_t*>(q + u.row[k] * cbytes + 256 * u.seg[k] + 4 * lane) : 0u;
    sc[k] = in ? scale[u.row[k] * sbytes + 16 * u.seg[k] + lane / 4] : 0u;
  }
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    if (!u.valid(k)) return;
    // 2^(code - 127) in fp32: code 0 is the subnormal 2^-127, 255 is NaN. Every
    // product is exact: at most two significant bits, not below 2^-128.
    const float s = __uint_as_float(sc[k] == 0u ? 0x00400000u : sc[k] == 255u ? 0x7FC00000u : sc[k] << 23);
    float x[8];
    mx4_values(w[k], s, x);
    store8_exact<TAIL>(out + u.row[k] * cols, 64 * u.seg[k] + lane, cols, x);
  }
}

unsigned unit_blocks(int64_t rows, int cols) {
  const int64_t units = rows * ((cols + 511) / 512);
  return (unsigned)((units + kUnits * (kThreads / 64) - 1) / (kUnits * (kThreads / 64)));
}

template <typename TS>
hipError_t quantize_typed(const void* in, int64_t rows, int cols, uint8_t* q, uint8_t* scale, uint8_t* arranged,
                          int64_t pitch, const Mx4Arrange* also, hipStream_t s) {
  const unsigned blocks = unit_blocks(rows, cols);
  const Mx4Arrange more = also != nullptr ? *also : Mx4Arrange{};
  const dim3 grid(blocks + (also != nullptr ? arrange_blocks(more, cols) : 0u));
  if (cols % 8 == 0)
    TWELL_LAUNCH("quantize_mx4", (mx4_quantize_kernel<TS, false>), grid, kThreads, 0, s, (const TS*)in, rows, cols, q,
                 scale, arranged, pitch, blocks, more);
  else
    TWELL_LAUNCH("quantize_mx4", (mx4_quantize_kernel<TS, true>), grid, kThreads, 0, s, (const TS*)in, rows, cols, q,
                 scale, arranged, pitch, blocks, more);
  return hipGetLastError();
}

template <typename TS>
hipError_t dequantize_typed(const uint8_t* q, const uint8_t* scale, int64_t rows, int cols, void* out, hipStream_t s) {
  const dim3 grid(unit_blocks(rows, cols));
  if (cols % 8 == 0)
    TWELL_LAUNCH("dequantize_mx4", (mx4_dequantize_kernel<TS, false>), grid, kThreads, 0, s, q, scale, rows, cols,
                 (TS*)out);
  else
    TWELL_LAUNCH("dequantize_mx4", (mx4_dequantize_kernel<TS, true>), grid, kThreads, 0, s, q, scale, rows, cols,
                 (TS*)out);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_mx4(const void* in, int is_bf16, int64_t rows, int cols, uint8_t* q, uint8_t* scale,
                               uint8_t* arranged, int64_t pitch, const Mx4Arrange* also, hipStream_t s) {
  return is_bf16 ? quantize_typed<uint16_t>(in, rows, cols, q, scale, arranged, pitch, also, s)
                 : quantize_typed<float>(in, rows, cols, q, scale, arranged, pitch, also, s);
}

hipError_t launch_mx4_arrange(const Mx4Arrange& a, const Mx4Arrange& b, int cols, hipStream_t s) {
  const unsigned blocks = arrange_blocks(a, cols);
  TWELL_LAUNCH("mx4_arrange", mx4_arrange_kernel, dim3(blocks + arrange_blocks(b, cols)), kThreads, 0, s, a, b, blocks,
               cols);
  return hipGetLastError();
}

hipError_t launch_dequantize_mx4(const uint8_t* q, const uint8_t* scale, int64_t rows, int cols, int out_bf16,
                                 void* out, hipStream_t s) {
  return out_bf16 ? dequantize_typed<uint16_t>(q, scale, rows, cols, out, s)
                  : dequantize_typed<float>(q, scale, rows, cols, out, s);
}

}  // namespace twell
