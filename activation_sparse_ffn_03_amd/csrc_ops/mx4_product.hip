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
//                       quantises x, into LDS.
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

// acc += A . B^T with both operands E2M1 (format 4) and byte B of sa and sb as
// scale codes: 16 x 128 by 128 x 16 ...
template <int B = 0>
__device__ __forceinline__ f32x4_t mfma(const u32x4_t& a, const u32x4_t& b, const f32x4_t& acc, uint32_t sa,
                                        uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(a), operand(b), acc, 4, 4, B, (int)sa, B, (int)sb);
}
// ... and 32 x 64 by 64 x 32.
template <int B = 0>
__device__ __forceinline__ f32x16_t mfma(const u32x4_t& a, const u32x4_t& b, const f32x16_t& acc, uint32_t sa,
                                         uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(a), operand(b), acc, 4, 4, B, (int)sa, B, (int)sb);
}

// Four neighbouring units of one token (fewer at the row's end), at any element.
__device__ __forceinline__ void store_units(const Mx4ProductArgs& a, int64_t token, int unit, const f32x4_t& v) {
  if (token >= a.n || unit >= a.units) return;
  const int64_t at = token * a.units + unit;
  const int have = a.units - unit;
  if (a.y_bf16) {
    uint16_t* p = static_cast<uint16_t*>(a.y) + at;
    const u32x2_t w = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    if (have >= 4) {
      *reinterpret_cast<u32x2_a2_t*>(p) = w;
    } else {
      for (int k = 0; k < have; ++k) p[k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
    }
  } else {
    float* p = static_cast<float*>(a.y) + at;
    if (have >= 4) {
      *reinterpret_cast<f32x4_a4_t*>(p) = v;
    } else {
      for (int k = 0; k < have; ++k) p[k] = v[k];
    }
  }
}

// ---------------------------------------------------------------- direct

// Block b of a row of x, quantised: codes and scale code (zeros behind its end).
template <typename TX, bool TAIL>
__device__ __forceinline__ u32x4_t quantize_block(const TX* row, int b, int cols, uint32_t& code) {
  Raw8<TX> raw[4];
  uint32_t m = 0;
#pragma unroll
  for (int c = 0; c < 4; ++c) raw[c].template load_filled<TAIL>(row, 4 * b + c, cols);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    raw[c].template settle<TAIL>(4 * b + c, cols);
    m = max(m, raw[c].max_bits());
  }
  code = mx4_scale_code(m);
  const float sc = mx4_scale_operand(code);
  u32x4_t q;
#pragma unroll
  for (int c = 0; c < 4; ++c) q[c] = code == 255u ? 0u : mx4_codes(raw[c], sc);
  return q;
}

// Tile of 16 FU units by 16 FT tokens. A wave's step is 256 columns, a whole
// cache line of codes a row: lane l holds blocks 2 (l >> 4) and 2 (l >> 4) + 1
// of its row's eight, one for each of two matrix instructions (which blocks
// share an instruction is free as long as both operands agree).
// With bf16 or fp32 x (a tile's rows of at most kMx4FusedBlocks blocks) each
// workgroup quantises its tokens into LDS, one block a thread at a time, while
// its first weights are on their way.
template <int XT, int FU, int FT, int WAVES, bool TAIL>
__global__ __launch_bounds__(64 * WAVES) void mx4_product_direct(Mx4ProductArgs a, int token_tiles) {
  __shared__ f32x4_t red[WAVES][FU * FT][64];
  constexpr int XBLOCKS = XT == X_MX4 ? 1 : kMx4FusedBlocks;
  __shared__ u32x4_t x_codes[XBLOCKS];
  __shared__ uint8_t x_scales[XBLOCKS];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int row = lane & 15, kb = lane >> 4;
  const int64_t L = xcd_run_block(blockIdx.x, gridDim.x);  // neighbours in one L2 share their weights
  const int64_t t0 = L % token_tiles * (16 * FT);
  const int u0 = (int)(L / token_tiles) * (16 * FU);
  const int cbytes = mx4_code_bytes(a.cols), sbytes = mx4_scale_bytes(a.cols);
  const int steps = (cbytes + 127) / 128;

  // Rows behind the last unit or token read the last one: their results are
  // not stored.
  const uint8_t *wq[FU], *ws[FU], *xq[FT], *xs[FT];
#pragma unroll
  for (int i = 0; i < FU; ++i) {
    const int64_t u = min(u0 + 16 * i + row, a.units - 1);
    wq[i] = a.w_q + u * cbytes + 32 * kb;
    ws[i] = a.w_scale + u * sbytes + 2 * kb;
  }
#pragma unroll
  for (int j = 0; j < FT; ++j) {
    const int64_t t = min(t0 + 16 * j + row, a.n - 1);
    if constexpr (XT == X_MX4) {
      xq[j] = a.x_q + t * cbytes + 32 * kb;
      xs[j] = a.x_scale + t * sbytes + 2 * kb;
    } else {
      xq[j] = reinterpret_cast<const uint8_t*>(x_codes + (t - t0) * 8 * steps + 2 * kb);
      xs[j] = x_scales + (t - t0) * 8 * steps + 2 * kb;
    }
  }
  f32x4_t acc[FU][FT];
#pragma unroll
  for (int i = 0; i < FU; ++i)
#pragma unroll
    for (int j = 0; j < FT; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  // several steps' loads in flight at a time; blocks behind the rows' last are
  // zeros (rows end with a whole 128 columns, 2 blocks of each lane or none)
  constexpr int DEPTH = FU * FT >= 16 ? 1 : 2;
  u32x4_t aw[DEPTH][2][FU], bx[DEPTH][2][FT];
  uint32_t sa[DEPTH][FU], sb[DEPTH][FT];
  auto load_w = [&](int k0) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      const int kt = k0 + d * WAVES;
      const bool in = 128 * kt + 32 * kb < cbytes;
#pragma unroll
      for (int i = 0; i < FU; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          aw[d][h][i] = in ? *reinterpret_cast<const u32x4_t*>(wq[i] + 128 * kt + 16 * h) : u32x4_t{0u, 0u, 0u, 0u};
        sa[d][i] = in ? *reinterpret_cast<const uint16_t*>(ws[i] + 8 * kt) : 0u;
      }
    }
  };
  if constexpr (XT != X_MX4) {
    load_w(wave);
    using TX = std::conditional_t<XT == X_BF16, uint16_t, float>;
    const int rows = (int)min((int64_t)16 * FT, a.n - t0);
    for (int b = threadIdx.x; b < rows * 8 * steps; b += 64 * WAVES) {
      const int t = b / (8 * steps);
      uint32_t code;
      x_codes[b] = quantize_block<TX, TAIL>(static_cast<const TX*>(a.x) + (t0 + t) * a.cols, b - t * 8 * steps, a.cols,
                                            code);
      x_scales[b] = (uint8_t)code;
    }
    lds_barrier();
  }
  for (int k0 = wave; k0 < steps; k0 += DEPTH * WAVES) {
    if (XT == X_MX4 || k0 != wave) load_w(k0);
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      const int kt = k0 + d * WAVES;
      const bool in = 128 * kt + 32 * kb < cbytes;
#pragma unroll
      for (int j = 0; j < FT; ++j) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          bx[d][h][j] = in ? *reinterpret_cast<const u32x4_t*>(xq[j] + 128 * kt + 16 * h)
                           : u32x4_t{0u, 0u, 0u, 0u};
        sb[d][j] = in ? *reinterpret_cast<const uint16_t*>(xs[j] + 8 * kt) : 0u;
      }
    }
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
#pragma unroll
      for (int i = 0; i < FU; ++i)
#pragma unroll
        for (int j = 0; j < FT; ++j) acc[i][j] = mfma<0>(aw[d][0][i], bx[d][0][j], acc[i][j], sa[d][i], sb[d][j]);
#pragma unroll
      for (int i = 0; i < FU; ++i)
#pragma unroll
        for (int j = 0; j < FT; ++j) acc[i][j] = mfma<1>(aw[d][1][i], bx[d][1][j], acc[i][j], sa[d][i], sb[d][j]);
    }
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
    store_units(a, t0 + 16 * (f % FT) + row, u0 + 16 * (f / FT) + 4 * kb, s);
  }
}

// ---------------------------------------------------------------- tiled

// A workgroup of WU x WT waves, each FU x FT fragments of 32 x 32: BU units by
// BT tokens. A stage is 256 columns: 128 bytes of codes a row, a whole cache
// line (an L2 channel serves one request a clock, of 64 bytes or of 128), and
// 8 scale bytes a row, arranged beforehand. LDS holds two.
template <int FU_, int FT_, int WU_, int WT_, int OCC_>
struct TileCfg {
  static constexpr int FU = FU_, FT = FT_, WU = WU_, WT = WT_, OCC = OCC_;
  static constexpr int NW = WU * WT, NT = 64 * NW;
  static constexpr int BU = 32 * FU * WU, BT = 32 * FT * WT, ROWS = BU + BT;
  static constexpr int CODES = ROWS * 128, STAGE = CODES + ROWS * 8;
  // a wave's rows of 128 output bytes, of 32 or 16 tokens at a time; 16 bytes
  // more a row keep both sides' accesses on different banks
  static constexpr int TOK = OCC > 1 ? 16 : 32;
  static constexpr int OUT = TOK * 144;
  static constexpr int LDS = 2 * STAGE + NW * OUT;
  static constexpr int UG = BU / 8 / NW, TG = BT / 8 / NW;  // 1 KB loads of 8 rows, of a wave and stage
  static constexpr int SROWS = ROWS / 128;                  // 1 KB loads of 128 rows' scales, of all waves;
  static constexpr int SG = (SROWS + NW - 1) / NW;          // of a wave: with fewer than waves some are made twice
  static constexpr int LOADS = UG + TG + SG;
  static constexpr int MIN_STORES = 2 * FU * FT;            // of a wave at a tile's end: 16-byte stores of bf16
  static_assert(LOADS / 2 + MIN_STORES <= 63, "vmcnt");
  static_assert(NW == 4, "the key of the LDS rows");
  static_assert(BU % 128 == 0 && BT % 128 == 0 && (SROWS % NW == 0 || SROWS < NW), "loads split evenly over the waves");
  static_assert(OCC * LDS <= 160 * 1024, "LDS of a compute unit");
};

// 16 bytes per lane from base + off straight into LDS, lane l's at lds + 16 l.
// A load that takes M0 has to be one wait state behind its write; the compiler
// does not see to that inside a statement.
__device__ __forceinline__ void dma_16B(const uint8_t* base, uint32_t off, uint32_t lds) {
  const uint32_t m = __builtin_amdgcn_readfirstlane(lds);
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(m) : "memory");
}
// vmcnt(M) if `many` (uniform) is not 0, else vmcnt(N). The branch is inside
// the statement: one that the compiler sees would split the loop's body, and
// it then moves matrix instructions across.
template <int M, int N>
__device__ __forceinline__ void wait_vmcnt_either(uint32_t many) {
  asm volatile(
      "s_cmp_eq_u32 %0, 0\n\ts_cbranch_scc1 .Lfew%=\n\ts_waitcnt vmcnt(%1)\n\ts_branch .Lend%=\n.Lfew%=:\n\t"
      "s_waitcnt vmcnt(%2)\n.Lend%=:" ::"s"(__builtin_amdgcn_readfirstlane(many)), "n"(M), "n"(N) : "memory", "scc");
}

// Workgroup -> tile: each XCD takes a contiguous run of tiles, walked in
// groups of 4 token blocks so that the tiles in flight share rows in L2 (us for
// 16384 x 4096 x 11008: 357 in groups of 2, 4 and 6, 364 of 8, 371 of 16).
__device__ __forceinline__ void tile_of(int64_t L, int tb, int ub, int& t, int& u) {
  constexpr int kGroup = 4;
  const int64_t per = (int64_t)kGroup * ub;
  const int first = (int)(L / per) * kGroup;
  const int g = min(tb - first, kGroup);
  const int in = (int)(L % per);
  t = first + in % g;
  u = in / g;
}

// A wave's results to memory, through LDS, 32 tokens by 128 bytes at a time
// (16 by 128 where two workgroups share the LDS), so that a store writes whole
// lines (8 tokens, 128 bytes each) instead of 32-byte pieces, each of which is
// a request of its own to L2. Rows of y may begin at any element: global memory
// takes 16 bytes at any address, a line's 128 then touch two (us
// without the quantisation, this way against 8 or 2 bytes a lane from the
// registers: 1003 x 1990 x 8100 14.6 : 18.1, x 8101 14.7 : 34.0, 5000 x 2048 x
// 8101 55.7 : 141; rows of whole lines, x 8192, 14.5).
template <class C, bool FEW>
__device__ __forceinline__ void store_tile(const Mx4ProductArgs& a, const f32x16_t (&acc)[C::FU][C::FT], int64_t t0,
                                           int u0, char* out) {
  const int lane = threadIdx.x & 63, row = lane & 31, half = lane >> 5;
  const int esz = a.y_bf16 ? 2 : 4;
  char* y = static_cast<char*>(a.y) + (t0 * a.units + u0) * esz;
  const int64_t pitch = (int64_t)a.units * esz;
  const int64_t left = a.n - t0;  // tokens there are
  constexpr int TOK = C::TOK;
  // TOK tokens from tok0, bytes [at, at + 128) of the wave's units. A wave's
  // LDS operations are done in their order; the statements around the reads
  // keep the compiler to it, which sees no lane's write of what another reads.
  auto flush = [&](int tok0, int at) {
    asm volatile("" ::: "memory");
#pragma unroll
    for (int r = 0; r < TOK / 8; ++r) {
      const int tok = 8 * r + (lane >> 3);
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(out + tok * 144 + 16 * (lane & 7));
      if (!FEW || tok0 + tok < left) *reinterpret_cast<u32x4_a2_t*>(y + (tok0 + tok) * pitch + at + 16 * (lane & 7)) = v;
    }
    asm volatile("" ::: "memory");
  };
#pragma unroll
  for (int j = 0; j < C::FT; ++j)
#pragma unroll
    for (int h = 0; h < 32 / TOK; ++h) {  // lanes of TOK tokens write, all read
      const bool mine = row / TOK == h;
      char* line = out + row % TOK * 144;
      if (a.y_bf16) {
        static_assert(C::FU % 2 == 0, "64 units a line");
#pragma unroll
        for (int i = 0; i < C::FU; i += 2) {
          if (mine) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const f32x16_t& v = acc[i + k][j];
                *reinterpret_cast<u32x2_t*>(line + 64 * k + 16 * q + 8 * half) =
                    u32x2_t{pack_bf16(v[4 * q], v[4 * q + 1]), pack_bf16(v[4 * q + 2], v[4 * q + 3])};
              }
          }
          flush(32 * j + TOK * h, 64 * i);
        }
      } else {
#pragma unroll
        for (int i = 0; i < C::FU; ++i) {
          if (mine) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const f32x16_t& v = acc[i][j];
              *reinterpret_cast<f32x4_t*>(line + 32 * q + 16 * half) =
                  f32x4_t{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
            }
          }
          flush(32 * j + TOK * h, 128 * i);
        }
      }
    }
}

// Needs at least BU units and BT tokens (without FEW). The last tile
// of a row or column of tiles is moved back to end with the matrix: what it
// shares with its neighbour is computed by both, to the same bits.
// HALF: the last stage has only 128 columns. ONE: there is one stage; loads run
// two ahead, so it is read again as a second, whose codes of w count as zeros
// (what it multiplies costs little, the product is bound by its stores then).
// FEW: fewer than BT tokens, one row of tiles; rows behind the last read the
// last one and are not stored.
template <class C, bool HALF, bool ONE, bool FEW>
__global__ __launch_bounds__(C::NT, C::OCC) void mx4_product_tiled(Mx4ProductArgs a, int tb, int ub) {
  __shared__ __attribute__((aligned(1024))) char smem[C::LDS];
  constexpr int FU = C::FU, FT = C::FT;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wu = wave / C::WT, wt = wave % C::WT;
  const int row = lane & 31, half = lane >> 5;
  const int cbytes = mx4_code_bytes(a.cols);
  const int KT = ONE ? 2 : (cbytes + 127) / 128;

  // This workgroup's tiles: every n-th (n workgroups on the XCD) of its XCD's run.
  const int64_t tiles = (int64_t)tb * ub;
  const int xcd = blockIdx.x % 8;
  const int64_t run = tiles / 8, extra = tiles % 8;
  const int64_t end = (xcd + 1) * run + min((int64_t)xcd + 1, extra);
  const int64_t stride = (gridDim.x + 7 - xcd) / 8;
  int64_t L = xcd * run + min((int64_t)xcd, extra) + blockIdx.x / 8;
  if (L >= end) return;

  // LDS: 16-byte piece p of row r lies at piece p ^ key(r), key = (r ^ r >> 3)
  // & 7 of r mod 32, so that eight consecutive rows' pieces (and sixteen's)
  // fall into different banks. A load covers 8 rows, lane l piece l & 7 of row
  // l >> 3; a wave's loads are 32 rows apart and share their keys.
  const int key = (row ^ (row >> 3)) & 7;
  const int lrow = 8 * wave + (lane >> 3);
  const int lpiece = (lane & 7) ^ ((lane >> 3) ^ wave);
  const uint32_t off = (uint32_t)(lrow * cbytes + 16 * lpiece);
  // the last stage's second half does not exist: read the first half again
  const uint32_t off_last = HALF ? (uint32_t)(lrow * cbytes + 16 * (lpiece & 3)) : off;
  uint32_t few[FEW ? C::TG : 1];  // FEW: rows of the token loads, held to the last one
  if constexpr (FEW) {
#pragma unroll
    for (int g = 0; g < C::TG; ++g) few[g] = (uint32_t)(min(lrow + 32 * g, (int)a.n - 1) * cbytes);
  }
  const uint32_t soff = 16u * lane;
  const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)(smem));

  struct Tile {
    const uint8_t *wq, *xq, *sc[C::SG];  // first rows of codes, and of this wave's scale loads
    int64_t t0;
    int u0;
  };
  auto tile_at = [&](int64_t l) {
    int t, u;
    tile_of(l, tb, ub, t, u);
    Tile r;
    r.t0 = FEW ? 0 : min((int64_t)t * C::BT, a.n - C::BT);
    r.u0 = min(u * C::BU, a.units - C::BU);
    r.wq = a.w_q + (int64_t)r.u0 * cbytes;
    r.xq = a.x_q + r.t0 * cbytes;
#pragma unroll
    for (int g = 0; g < C::SG; ++g) {
      const int first = (wave + 4 * g) % C::SROWS * 128;
      r.sc[g] = first < C::BU ? a.w_arr + (int64_t)(r.u0 + first) * 8 : a.x_arr + (r.t0 + first - C::BU) * 8;
    }
    return r;
  };
  int64_t sstep[C::SG];  // bytes from one stage's scales to the next's
#pragma unroll
  for (int g = 0; g < C::SG; ++g) sstep[g] = 8 * ((wave + 4 * g) % C::SROWS * 128 < C::BU ? (int64_t)a.units : mx4_arranged_rows(a.n));
  struct Stage {
    const uint8_t *wq, *xq, *sc[C::SG];
    uint32_t off;
  };
  auto stage_at = [&](const Tile& c, const Tile& n, int kt) {  // past c's last: of n
    const bool in = kt < KT;
    const int k = ONE ? 0 : in ? kt : kt - KT;
    Stage r;
    r.wq = (in ? c.wq : n.wq) + 128 * k;
    r.xq = (in ? c.xq : n.xq) + 128 * k;
#pragma unroll
    for (int g = 0; g < C::SG; ++g) r.sc[g] = (in ? c.sc[g] : n.sc[g]) + k * sstep[g];
    r.off = HALF && (ONE || k == KT - 1) ? off_last : off;
    return r;
  };
  auto issue = [&](const Stage& t, uint32_t buf, int g) {
    const uint32_t at = lds0 + buf * C::STAGE;
    if (g < C::UG)
      dma_16B(t.wq + (int64_t)(32 * g) * cbytes, t.off, at + (wave + 4 * g) * 1024);
    else if (FEW && g < C::UG + C::TG)
      dma_16B(t.xq, few[g - C::UG] + (t.off - (uint32_t)(lrow * cbytes)), at + C::BU * 128 + (wave + 4 * (g - C::UG)) * 1024);
    else if (g < C::UG + C::TG)
      dma_16B(t.xq + (int64_t)(32 * (g - C::UG)) * cbytes, t.off, at + C::BU * 128 + (wave + 4 * (g - C::UG)) * 1024);
    else
      dma_16B(t.sc[g - C::UG - C::TG], soff, at + C::CODES + (wave + 4 * (g - C::UG - C::TG)) % C::SROWS * 1024);
  };

  f32x16_t acc[FU][FT];
  u32x4_t av[4][FU], bv[4][FT];  // operands of a stage's four steps
  uint32_t sa[FU], sb[FT];
  int piece[4];
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) piece[ks] = row * 128 + ((2 * ks + half) ^ key) * 16;
  auto read_a = [&](int i, int ks, uint32_t buf) {
    return *reinterpret_cast<const u32x4_t*>(smem + buf * C::STAGE + (wu * FU + i) * 4096 + piece[ks]);
  };
  auto read_b = [&](int j, int ks, uint32_t buf) {
    return *reinterpret_cast<const u32x4_t*>(smem + buf * C::STAGE + C::BU * 128 + (wt * FT + j) * 4096 + piece[ks]);
  };
  // a row's scale codes of the steps' blocks `half`, step 0's lowest
  auto read_scale = [&](int r, uint32_t buf) {
    return *reinterpret_cast<const uint32_t*>(smem + buf * C::STAGE + C::CODES + r * 8 + 4 * half);
  };

  // Loads run two stages ahead, into the next tile at a tile's end; behind the
  // last tile they read it again, unused.
  Tile cur = tile_at(L);
  {
    const Stage s0 = stage_at(cur, cur, 0), s1 = stage_at(cur, cur, 1);
#pragma unroll
    for (int g = 0; g < C::LOADS; ++g) issue(s0, 0, g);
#pragma unroll
    for (int g = 0; g < C::LOADS; ++g) issue(s1, 1, g);
  }
  wait_vmcnt<C::LOADS>();
  lds_barrier();
#pragma unroll
  for (int i = 0; i < FU; ++i) {
    av[0][i] = read_a(i, 0, 0);
    sa[i] = read_scale((wu * FU + i) * 32 + row, 0);
  }
#pragma unroll
  for (int j = 0; j < FT; ++j) {
    bv[0][j] = read_b(j, 0, 0);
    sb[j] = read_scale(C::BU + (wt * FT + j) * 32 + row, 0);
  }

  uint32_t buf = 0, stores = 0;  // stores: the tile before has left some behind
  for (;;) {
    const bool more = L + stride < end;
    const Tile next = more ? tile_at(L + stride) : cur;
#pragma unroll
    for (int i = 0; i < FU; ++i)
#pragma unroll
      for (int j = 0; j < FT; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;

    for (int kt = 0; kt < KT; ++kt) {
      // Four steps of 64 columns. All operands of the stage are in registers
      // when the second step ends, so that its LDS can be filled again during
      // the third and fourth; the next stage's first operands are read in the
      // fourth. Loads are spread over two steps: a wave that issues them at
      // once waits for the address unit and keeps its matrix core waiting.
      const Stage ahead = stage_at(cur, next, kt + 2);
      // masks of this stage's last two steps, of its others, and of the next one's first
      const uint32_t last = HALF && (ONE || kt == KT - 1) ? 0u : ~0u;
      const uint32_t live = ONE && kt == 1 ? 0u : ~0u, live_next = ONE && kt == 0 ? 0u : ~0u;
      uint32_t na[FU], nb[FT];
      constexpr int OPS = FU + FT, M = FU * FT;  // operands and matrix instructions of a step
      // read r of the 3 OPS behind the first step's operands
      auto read = [&](int r) {
        const int ks = 1 + r / OPS, k = r % OPS;
        if (k < FU) {
          av[ks][k] = read_a(k, ks, buf);
          if (ONE || (HALF && ks >= 2)) av[ks][k] &= ks >= 2 ? last & live : live;
        } else {
          bv[ks][k - FU] = read_b(k - FU, ks, buf);
        }
      };
      auto read_next = [&](int r) {
        if (r < FU) {
          av[0][r] = read_a(r, 0, buf ^ 1);
          if (ONE) av[0][r] &= live_next;
        } else if (r < OPS) bv[0][r - FU] = read_b(r - FU, 0, buf ^ 1);
        else if (r < OPS + FU) na[r - OPS] = read_scale((wu * FU + r - OPS) * 32 + row, buf ^ 1);
        else nb[r - OPS - FU] = read_scale(C::BU + (wt * FT + r - OPS - FU) * 32 + row, buf ^ 1);
      };
      // Operation k of n that are dealt to slots [0, m): those of slot s.
      auto first_of = [](int s, int n, int m) { return s >= m ? n : s * n / m; };
      auto step = [&](auto KS) {
        constexpr int ks = decltype(KS)::value;
#pragma unroll
        for (int s = 0; s < M; ++s) {
          const int i = s / FT, j = s % FT;
          acc[i][j] = mfma<ks>(av[ks][i], bv[ks][j], acc[i][j], sa[i], sb[j]);
          if constexpr (ks < 2) {  // done half a step before the barrier
#pragma unroll
            for (int r = first_of(ks * M + s, 3 * OPS, M + M / 2); r < first_of(ks * M + s + 1, 3 * OPS, M + M / 2); ++r)
              read(r);
          } else {
#pragma unroll
            for (int g = first_of((ks - 2) * M + s, C::LOADS, 2 * M); g < first_of((ks - 2) * M + s + 1, C::LOADS, 2 * M); ++g)
              issue(ahead, buf, g);
          }
          if constexpr (ks == 3) {
#pragma unroll
            for (int r = first_of(s, 2 * OPS, M / 2 + 1); r < first_of(s + 1, 2 * OPS, M / 2 + 1); ++r) read_next(r);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      };
      step(std::integral_constant<int, 0>{});
      step(std::integral_constant<int, 1>{});
      lds_barrier();  // every wave has read all of this stage
      __builtin_amdgcn_sched_barrier(0);
      step(std::integral_constant<int, 2>{});
      // The next stage has landed once only this step's loads are pending, and
      // in a tile's first stage the stores of the tile before, which were
      // asked for later than it.
      wait_vmcnt_either<C::LOADS / 2 + C::MIN_STORES, C::LOADS / 2>(stores & (uint32_t)(kt == 0));
      lds_barrier();
      __builtin_amdgcn_sched_barrier(0);
      step(std::integral_constant<int, 3>{});
#pragma unroll
      for (int i = 0; i < FU; ++i) sa[i] = na[i];
#pragma unroll
      for (int j = 0; j < FT; ++j) sb[j] = nb[j];
      buf ^= 1;
    }

    store_tile<C, FEW>(a, acc, cur.t0 + wt * FT * 32, cur.u0 + wu * FU * 32, smem + 2 * C::STAGE + wave * C::OUT);
    if (!more) break;
    cur = next;
    L += stride;
    stores = FEW ? 0u : 1u;  // FEW: some have no token to store, and may not have been issued
  }
  wait_vmcnt<0>();  // no load may write to LDS behind the workgroup's end
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

template <class C, bool FEW>
hipError_t launch_tiled(const Mx4ProductArgs& a, hipStream_t s) {
  // a smaller matrix would be read in front of its first row
  if ((!FEW && a.n < C::BT) || (FEW && a.n >= C::BT) || a.units < C::BU || (FEW && a.cols <= 256))
    return hipErrorInvalidValue;
  const int tb = (int)((a.n + C::BT - 1) / C::BT), ub = (a.units + C::BU - 1) / C::BU;
  const int64_t tiles = (int64_t)tb * ub;
  const int64_t fit = 256 * C::OCC;  // workgroups that run at a time
  const dim3 grid((unsigned)(tiles < fit ? tiles : fit));
  auto go = [&](auto half, auto one) {
    TWELL_LAUNCH("mx4_product_tiled", (mx4_product_tiled<C, decltype(half)::value, decltype(one)::value, FEW>), grid,
                 C::NT, 0, s, a, tb, ub);
  };
  using No = std::false_type;
  using Yes = std::true_type;
  const bool half = mx4_code_bytes(a.cols) % 128 != 0;
  if (FEW || a.cols > 256) {
    if (half) go(Yes{}, No{});
    else go(No{}, No{});
  } else if constexpr (!FEW) {
    if (half) go(Yes{}, Yes{});
    else go(No{}, Yes{});
  }
  return hipGetLastError();
}

using Big = TileCfg<4, 4, 2, 2, 1>;
using Mid = TileCfg<2, 2, 2, 2, 2>;
static_assert(Big::BU == kMx4BigTile && Big::BT == kMx4BigTile && Mid::BU == kMx4MidTile && Mid::BT == kMx4MidTile,
              "the plan's tiles");

}  // namespace

hipError_t launch_mx4_product(Mx4Plan plan, const Mx4ProductArgs& a, hipStream_t s) {
  switch (plan) {
    case MX4_FUSED:
      // up to 4 tokens 16 units and 4 waves a workgroup, above twice of both: x
      // is quantised half as often (us at 1 and 8 x 4096 x 11008: 6.6 and 10.7
      // against 8.0 and 10.6; 16 x 2048 x 5632: 7.3 against 5.7); from 17 on 32
      // tokens (24 x 2048 x 5632 7.2, in tiles of 16 tokens 9.8, of 16 units 8.7)
      if (a.n <= 4) return a.x_bf16 ? launch_direct<X_BF16, 1, 1, 4>(a, s) : launch_direct<X_F32, 1, 1, 4>(a, s);
      if (a.n > 16) return a.x_bf16 ? launch_direct<X_BF16, 2, 2, 8>(a, s) : launch_direct<X_F32, 2, 2, 8>(a, s);
      return a.x_bf16 ? launch_direct<X_BF16, 2, 1, 8>(a, s) : launch_direct<X_F32, 2, 1, 8>(a, s);
    case MX4_BIG:
      return launch_tiled<Big, false>(a, s);
    case MX4_MID:
      return a.n < Mid::BT ? launch_tiled<Mid, true>(a, s) : launch_tiled<Mid, false>(a, s);
    default:
      switch (mx4_direct_tile(a.n, a.cols, a.units)) {
        case 1: return launch_direct<X_MX4, 1, 1, 4>(a, s);
        case 2: return launch_direct<X_MX4, 2, 2, 4>(a, s);
        default: return launch_direct<X_MX4, 4, 4, 4>(a, s);
      }
  }
}

}  // namespace twell
