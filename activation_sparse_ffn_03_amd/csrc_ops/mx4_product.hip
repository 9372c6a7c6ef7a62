// Product of MX4 rows: y[i][c] = sum over blocks of 2^(xs + ws - 254) * sum_k xq wq,
// on v_mfma_scale_f32_16x16x128_f8f6f4, which multiplies 16 x 128 by 128 x 16
// four-bit codes and applies both operands' block scales: lane l supplies 16
// bytes, block l >> 4 of row l & 15, of each operand, and the block's scale code
// in one byte of a register; its results are rows 4 (l >> 4) + r of the first
// operand, column l & 15 of the second (checked with an in-bounds probe, as
// was that a scale code of 255 makes its row NaN). Products of two codes are
// exact, sums are held in fp32.
//
// The weights are the first operand, the tokens the second: a lane then holds
// four neighbouring units of one token and stores them together.
//
//   mx4_product_direct  few tokens or few tiles: each wave of a workgroup takes
//                       every WAVES-th 128 columns of the whole tile, straight
//                       from memory into registers; the waves' sums are added
//                       in LDS in a fixed order. With bf16 or fp32 x it also
//                       quantises x in registers.
//   mx4_product_tiled   many tokens: tiles through a ring of LDS stages.
#include "mx4_device.h"
#include "ops_kernels.h"
#include "../csrc/twell_trace.h"

namespace twell {
namespace {

enum { X_MX4 = 0, X_BF16 = 1, X_F32 = 2 };

__device__ __forceinline__ i32x8_t operand(const u32x4_t& v) {
  // the last four words are not read for four-bit operands
  return i32x8_t{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
}

// acc += A . B^T with both operands E2M1 (format 4), the lowest byte of sa and
// sb as scale codes.
__device__ __forceinline__ f32x4_t mfma(const u32x4_t& a, const u32x4_t& b, const f32x4_t& acc, uint32_t sa,
                                        uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(a), operand(b), acc, 4, 4, 0, (int)sa, 0, (int)sb);
}

// Four neighbouring units of one token. WHOLE: units is a multiple of 4, so
// that the four exist together and are aligned.
template <bool BF16, bool WHOLE>
__device__ __forceinline__ void store_units(void* y, int64_t token, int64_t n, int unit, int units, const f32x4_t& v) {
  if (token >= n || unit >= units) return;
  const int64_t at = token * units + unit;
  if constexpr (BF16) {
    uint16_t* p = static_cast<uint16_t*>(y) + at;
    const u32x2_t w = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    if constexpr (WHOLE) {
      *reinterpret_cast<u32x2_t*>(p) = w;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (unit + k < units) p[k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
    }
  } else {
    float* p = static_cast<float*>(y) + at;
    if constexpr (WHOLE) {
      *reinterpret_cast<f32x4_t*>(p) = v;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (unit + k < units) p[k] = v[k];
    }
  }
}
// Calls put(BF16, WHOLE) with what the product's output has.
template <typename Put>
__device__ __forceinline__ void store_kind(const Mx4ProductArgs& a, Put put) {
  const bool whole = a.units % 4 == 0;
  if (a.y_bf16) {
    if (whole) put(std::true_type{}, std::true_type{});
    else put(std::true_type{}, std::false_type{});
  } else {
    if (whole) put(std::false_type{}, std::true_type{});
    else put(std::false_type{}, std::false_type{});
  }
}

// ---------------------------------------------------------------- direct

// Block kb of 128 columns kt of one row of x, quantised: codes and scale code.
template <typename TX, bool TAIL>
__device__ __forceinline__ u32x4_t quantize_block(const TX* row, int kt, int kb, int cols, uint32_t& code) {
  Raw8<TX> raw[4];
  uint32_t m = 0;
#pragma unroll
  for (int c = 0; c < 4; ++c) raw[c].template load<TAIL>(row, 16 * kt + 4 * kb + c, cols);
#pragma unroll
  for (int c = 0; c < 4; ++c) m = max(m, raw[c].max_bits());
  code = mx4_scale_code(m);
  const float sc = mx4_scale_operand(code);
  u32x4_t q;
#pragma unroll
  for (int c = 0; c < 4; ++c) q[c] = code == 255u ? 0u : mx4_codes(raw[c], sc);
  return q;
}

// Tile of 16 FU units by 16 FT tokens.
template <int XT, int FU, int FT, int WAVES, bool TAIL>
__global__ __launch_bounds__(64 * WAVES) void mx4_product_direct(Mx4ProductArgs a, int token_tiles) {
  __shared__ f32x4_t red[WAVES][FU * FT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int row = lane & 15, kb = lane >> 4;
  const int64_t L = xcd_run_block(blockIdx.x, gridDim.x);  // neighbours in one L2 share their weights
  const int64_t t0 = L % token_tiles * (16 * FT);
  const int u0 = (int)(L / token_tiles) * (16 * FU);
  const int cbytes = mx4_code_bytes(a.cols), sbytes = mx4_scale_bytes(a.cols);
  const int KT = cbytes / 64;

  // Rows behind the last unit or token read the last one: their results are
  // not stored.
  const uint8_t *wq[FU], *ws[FU], *xq[FT], *xs[FT];
  int64_t tok[FT];
#pragma unroll
  for (int i = 0; i < FU; ++i) {
    const int64_t u = min(u0 + 16 * i + row, a.units - 1);
    wq[i] = a.w_q + u * cbytes + 16 * kb;
    ws[i] = a.w_scale + u * sbytes + kb;
  }
#pragma unroll
  for (int j = 0; j < FT; ++j) {
    const int64_t t = t0 + 16 * j + row;
    tok[j] = t < a.n ? t : a.n - 1;
    xq[j] = a.x_q + tok[j] * cbytes + 16 * kb;
    xs[j] = a.x_scale + tok[j] * sbytes + kb;
  }
  f32x4_t acc[FU][FT];
#pragma unroll
  for (int i = 0; i < FU; ++i)
#pragma unroll
    for (int j = 0; j < FT; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  // several steps' loads in flight at a time; a step behind the last is zeros
  constexpr int DEPTH = FU * FT >= 16 ? 2 : 4;
  for (int k0 = wave; k0 < KT; k0 += DEPTH * WAVES) {
    u32x4_t aw[DEPTH][FU], bx[DEPTH][FT];
    uint32_t sa[DEPTH][FU], sb[DEPTH][FT];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      const int kt = k0 + d * WAVES;
      const bool in = kt < KT;
#pragma unroll
      for (int i = 0; i < FU; ++i) {
        aw[d][i] = in ? *reinterpret_cast<const u32x4_t*>(wq[i] + 64 * kt) : u32x4_t{0u, 0u, 0u, 0u};
        sa[d][i] = in ? ws[i][4 * kt] : 0;
      }
#pragma unroll
      for (int j = 0; j < FT; ++j) {
        if constexpr (XT == X_MX4) {
          bx[d][j] = in ? *reinterpret_cast<const u32x4_t*>(xq[j] + 64 * kt) : u32x4_t{0u, 0u, 0u, 0u};
          sb[d][j] = in ? xs[j][4 * kt] : 0;
        } else {
          using TX = std::conditional_t<XT == X_BF16, uint16_t, float>;
          bx[d][j] = quantize_block<TX, TAIL>(static_cast<const TX*>(a.x) + tok[j] * a.cols, kt, kb, a.cols, sb[d][j]);
        }
      }
    }
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
#pragma unroll
      for (int i = 0; i < FU; ++i)
#pragma unroll
        for (int j = 0; j < FT; ++j) acc[i][j] = mfma(aw[d][i], bx[d][j], acc[i][j], sa[d][i], sb[d][j]);
  }

#pragma unroll
  for (int i = 0; i < FU; ++i)
#pragma unroll
    for (int j = 0; j < FT; ++j) red[wave][i * FT + j][lane] = acc[i][j];
  __syncthreads();
  for (int f = wave; f < FU * FT; f += WAVES) {
    f32x4_t s = red[0][f][lane];
#pragma unroll
    for (int v = 1; v < WAVES; ++v) s += red[v][f][lane];
    store_kind(a, [&](auto bf16, auto whole) {
      store_units<decltype(bf16)::value, decltype(whole)::value>(a.y, t0 + 16 * (f % FT) + row, a.n,
                                                                 u0 + 16 * (f / FT) + 4 * kb, a.units, s);
    });
  }
}

// ---------------------------------------------------------------- tiled

// BU units by BT tokens per workgroup of WU x WT waves, ST stages of 128
// columns (64 bytes a row).
template <int BU_, int BT_, int WU_, int WT_, int ST_, int OCC_>
struct TileCfg {
  static constexpr int BU = BU_, BT = BT_, WU = WU_, WT = WT_, ST = ST_, OCC = OCC_;
  static constexpr int NW = WU * WT, NT = 64 * NW;
  static constexpr int FU = BU / WU / 16, FT = BT / WT / 16;
  static constexpr int ROWS = BU + BT;
  static constexpr int STAGE = ROWS * 64;
  static constexpr int GPW = ROWS / 16 / NW;  // 1 KB loads of a wave per stage
  static constexpr int SPW = (ROWS / 64 + NW - 1) / NW;  // scale loads (64 rows, 16 bytes each) of a wave per four stages
  static constexpr int SCALES = SPW * NW * 1024;  // one of two buffers
  static constexpr int LDS = ST * STAGE + 2 * SCALES;
  static_assert(BU % (16 * WU) == 0 && BT % (16 * WT) == 0, "whole fragments");
  static_assert(ROWS % (16 * NW) == 0, "stage loads split evenly over the waves");
  static_assert(ST >= 2 && ST <= 4, "ring depth");
  static_assert(LDS <= 160 * 1024, "LDS of a compute unit");
};

// XOR key of the 16-byte pieces of a 64-byte LDS row that keeps the fragment
// reads (16 rows, one piece each per 16 lanes) free of bank conflicts.
__device__ __forceinline__ int piece_key(int r) { return ((r >> 3) & 1) | ((((r >> 1) ^ (r >> 3)) & 1) << 1); }

// Workgroup -> tile: each XCD takes a contiguous run of tiles, walked in
// groups of kGroup token blocks so that the tiles in flight share rows in L2.
__device__ __forceinline__ void tile_of(int64_t L, int tb, int ub, int group, int& t, int& u) {
  const int64_t per = (int64_t)group * ub;
  const int first = (int)(L / per) * group;
  const int g = min(tb - first, group);
  const int in = (int)(L % per);
  t = first + in % g;
  u = in / g;
}

template <class C>
__global__ __launch_bounds__(C::NT, C::OCC) void mx4_product_tiled(Mx4ProductArgs a, int tb, int ub) {
  __shared__ __attribute__((aligned(1024))) char smem[C::LDS];
  constexpr int FU = C::FU, FT = C::FT;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wu = wave / C::WT, wt = wave % C::WT;
  const int row = lane & 15, kb = lane >> 4;
  int tt, tu;
  tile_of(xcd_run_block(blockIdx.x, gridDim.x), tb, ub, 8, tt, tu);
  const int64_t t0 = (int64_t)tt * C::BT;
  const int u0 = tu * C::BU;
  const int cbytes = mx4_code_bytes(a.cols), sbytes = mx4_scale_bytes(a.cols);
  const int KT = cbytes / 64;

  // Row r of a stage: unit u0 + r, then token t0 + r - BU; rows behind the
  // last unit or token read row 0, their results are not stored.
  auto code_row = [&](int r) {
    if (r < C::BU) return a.w_q + (int64_t)(u0 + r < a.units ? u0 + r : 0) * cbytes;
    const int64_t t = t0 + r - C::BU;
    return a.x_q + (t < a.n ? t : 0) * cbytes;
  };
  auto scale_row = [&](int r) {
    if (r < C::BU) return a.w_scale + (int64_t)(u0 + r < a.units ? u0 + r : 0) * sbytes;
    const int64_t t = t0 + r - C::BU;
    return a.x_scale + (t < a.n ? t : 0) * sbytes;
  };
  const uint8_t* src[C::GPW];
  uint32_t dst[C::GPW];
  const int rin = lane >> 2, pos = lane & 3;
#pragma unroll
  for (int g = 0; g < C::GPW; ++g) {
    const int r = (wave + C::NW * g) * 16 + rin;
    src[g] = code_row(r) + ((pos ^ piece_key(r & 15)) << 4);
    dst[g] = (uint32_t)((r - rin) * 64);
  }
  const uint8_t* ssrc[C::SPW];
  uint32_t sdst[C::SPW];
#pragma unroll
  for (int g = 0; g < C::SPW; ++g) {
    const int first = (wave + C::NW * g) * 64;
    ssrc[g] = scale_row(min(first + lane, C::ROWS - 1));
    sdst[g] = (uint32_t)(C::ST * C::STAGE + first * 16);
  }
  const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)(smem));
  auto issue = [&](int kt) {
    if (kt % 4 == 0) {
#pragma unroll
      for (int g = 0; g < C::SPW; ++g)
        dma_16B(ssrc[g] + 4 * kt, lds0 + sdst[g] + (uint32_t)((kt / 4 % 2) * C::SCALES));
    }
    const uint32_t sb = lds0 + (uint32_t)((kt % C::ST) * C::STAGE);
#pragma unroll
    for (int g = 0; g < C::GPW; ++g) dma_16B(src[g] + (size_t)kt * 64, sb + dst[g]);
  };

  f32x4_t acc[FU][FT];
#pragma unroll
  for (int i = 0; i < FU; ++i)
#pragma unroll
    for (int j = 0; j < FT; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

#pragma unroll
  for (int st = 0; st < C::ST - 1; ++st)
    if (st < KT) issue(st);

  uint32_t sa[FU], sb[FT];
  // byte kb of each word of a row's 16 scale bytes: its block kb in the four
  // stages they cover
  const uint32_t pick = (uint32_t)kb | ((uint32_t)(kb + 4) << 8);
  auto scales_of = [&](int r, int buf) {
    const u32x4_t v = *reinterpret_cast<const u32x4_t*>(smem + C::ST * C::STAGE + buf * C::SCALES + r * 16);
    const uint32_t lo = __builtin_amdgcn_perm(v[1], v[0], pick), hi = __builtin_amdgcn_perm(v[3], v[2], pick);
    return (lo & 0xFFFFu) | (hi << 16);
  };
  const int at = (kb ^ piece_key(row)) << 4;
  for (int kt = 0; kt < KT; ++kt) {
    // Stage kt is complete for this wave once only the later stages' loads are
    // pending (scale loads among them make the wait stricter, never looser);
    // the barrier extends that to every wave, and says that every wave is done
    // with the stage refilled below.
    const int later = min(C::ST - 2, KT - 1 - kt);
    if (later >= 2) wait_vmcnt<2 * C::GPW>();
    else if (later == 1) wait_vmcnt<C::GPW>();
    else wait_vmcnt<0>();
    lds_barrier();
    if (kt + C::ST - 1 < KT) issue(kt + C::ST - 1);
    const char* A = smem + (kt % C::ST) * C::STAGE;
    if (kt % 4 == 0) {
      const int buf = kt / 4 % 2;
#pragma unroll
      for (int i = 0; i < FU; ++i) sa[i] = scales_of((wu * FU + i) * 16 + row, buf);
#pragma unroll
      for (int j = 0; j < FT; ++j) sb[j] = scales_of(C::BU + (wt * FT + j) * 16 + row, buf);
    } else {
#pragma unroll
      for (int i = 0; i < FU; ++i) sa[i] >>= 8;
#pragma unroll
      for (int j = 0; j < FT; ++j) sb[j] >>= 8;
    }
    u32x4_t av[FU], bv[FT];
#pragma unroll
    for (int i = 0; i < FU; ++i) av[i] = *reinterpret_cast<const u32x4_t*>(A + ((wu * FU + i) * 16 + row) * 64 + at);
#pragma unroll
    for (int j = 0; j < FT; ++j)
      bv[j] = *reinterpret_cast<const u32x4_t*>(A + (C::BU + (wt * FT + j) * 16 + row) * 64 + at);
#pragma unroll
    for (int i = 0; i < FU; ++i)
#pragma unroll
      for (int j = 0; j < FT; ++j) acc[i][j] = mfma(av[i], bv[j], acc[i][j], sa[i], sb[j]);
  }

  auto put = [&](auto bf16, auto whole) {
#pragma unroll
    for (int j = 0; j < FT; ++j)
#pragma unroll
      for (int i = 0; i < FU; ++i)
        store_units<decltype(bf16)::value, decltype(whole)::value>(
            a.y, t0 + (wt * FT + j) * 16 + row, a.n, u0 + (wu * FU + i) * 16 + 4 * kb, a.units, acc[i][j]);
  };
  store_kind(a, put);
}

template <int XT, int FU, int FT, int WAVES>
hipError_t launch_direct(const Mx4ProductArgs& a, hipStream_t s) {
  const int64_t tt = (a.n + 16 * FT - 1) / (16 * FT), ut = (a.units + 16 * FU - 1) / (16 * FU);
  const dim3 grid((unsigned)(tt * ut));
  if (XT == X_MX4 || a.cols % 8 == 0)
    TWELL_LAUNCH("mx4_product_direct", (mx4_product_direct<XT, FU, FT, WAVES, false>), grid, 64 * WAVES, 0, s, a,
                 (int)tt);
  else
    TWELL_LAUNCH("mx4_product_direct", (mx4_product_direct<XT, FU, FT, WAVES, true>), grid, 64 * WAVES, 0, s, a,
                 (int)tt);
  return hipGetLastError();
}

template <class C>
hipError_t launch_tiled(const Mx4ProductArgs& a, hipStream_t s) {
  const int tb = (int)((a.n + C::BT - 1) / C::BT), ub = (a.units + C::BU - 1) / C::BU;
  TWELL_LAUNCH("mx4_product_tiled", mx4_product_tiled<C>, dim3((unsigned)((int64_t)tb * ub)), C::NT, 0, s, a, tb, ub);
  return hipGetLastError();
}

using Big = TileCfg<256, 256, 2, 4, 4, 1>;

}  // namespace

hipError_t launch_mx4_product(const Mx4ProductArgs& a, hipStream_t s) {
  if (a.x != nullptr)
    return a.x_bf16 ? launch_direct<X_BF16, 1, 1, 8>(a, s) : launch_direct<X_F32, 1, 1, 8>(a, s);
  if (a.n <= 16) return launch_direct<X_MX4, 1, 1, 8>(a, s);
  if (a.n <= 32) return launch_direct<X_MX4, 1, 2, 8>(a, s);
  if (a.n <= 64) return launch_direct<X_MX4, 1, 4, 8>(a, s);
  const int64_t tiles = ((a.n + 255) / 256) * ((a.units + 255) / 256);
  if (tiles < 128) return launch_direct<X_MX4, 4, 4, 4>(a, s);
  return launch_tiled<Big>(a, s);
}

}  // namespace twell
