// Products of many rows: out[i][u] = sum_k q(i, k) p(u, k) in bf16 on
// v_mfma_f32_32x32x16_bf16, tiles of BU units by BT rows through two LDS stages
// of 64 k. Lane l supplies k 8 (l >> 5) .. + 7 of line l & 31 of each operand;
// its results are elements 8 (v >> 2) + 4 (l >> 5) + (v & 3) of the first
// operand, line l & 31 of the second, so that the units, which are neighbours in
// memory, are the first.
//
// The matrix cores bound a large product (2.5 PFLOP/s): a stage's 64 matrix
// instructions a wave take 2048 cycles, in which it reads 32 KB from LDS and the
// workgroup loads 64 KB into it.
#pragma once

#include <utility>

#include "linear_device.h"
#include "../csrc/twell_trace.h"

namespace twell {

// Four waves, two by two, each FU x FT fragments of 32 x 32.
template <int FU_, int FT_, int OCC_>
struct LinearTile {
  static constexpr int FU = FU_, FT = FT_, OCC = OCC_;
  static constexpr int BU = 64 * FU, BT = 64 * FT;
  static constexpr int STAGE = (BU + BT) * 128;
  // a wave's results on their way out: TOK rows of 64 units in fp32, 16 bytes
  // more a row keep both sides' accesses on different banks
  static constexpr int TOK = OCC > 1 ? 8 : 16, LINE = 272, OUT = TOK * LINE;
  static constexpr int LDS = 2 * STAGE + 4 * OUT;
  static constexpr int UG = BU / 32, TG = BT / 32;  // 1 KB loads of a wave and stage
  static constexpr int LOADS = UG + TG;
  static constexpr int MIN_STORES = 2 * FU * FT;    // of a wave at the end of a whole tile: 16 bytes of bf16 a lane
  static_assert(LOADS / 2 + MIN_STORES <= 63, "vmcnt");
  static_assert(OCC * LDS <= 160 * 1024, "LDS of a compute unit");
};

// What a lane reads in place of k behind the last.
__device__ const u32x4_t linear_zeros = {0u, 0u, 0u, 0u};

// 16 bytes per lane into LDS, lane l's at lds + 16 l: from base + off, or from an
// address of its own. A load that takes M0 has to be one wait state behind its
// write; the compiler does not see to that inside a statement.
__device__ __forceinline__ void linear_dma(const char* base, uint32_t off, uint32_t lds) {
  const uint32_t m = __builtin_amdgcn_readfirstlane(lds);
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(m) : "memory");
}
__device__ __forceinline__ void linear_dma_at(const char* p, uint32_t lds) {
  const uint32_t m = __builtin_amdgcn_readfirstlane(lds);
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(p), "s"(m) : "memory");
}
// vmcnt(M) if `many` (uniform) is not 0, else vmcnt(N). The branch is inside
// the statement: one that the compiler sees would split the loop's body, and
// it then moves matrix instructions across.
template <int M, int N>
__device__ __forceinline__ void linear_wait_either(uint32_t many) {
  asm volatile(
      "s_cmp_eq_u32 %0, 0\n\ts_cbranch_scc1 .Lfew%=\n\ts_waitcnt vmcnt(%1)\n\ts_branch .Lend%=\n.Lfew%=:\n\t"
      "s_waitcnt vmcnt(%2)\n.Lend%=:" ::"s"(__builtin_amdgcn_readfirstlane(many)), "n"(M), "n"(N) : "memory", "scc");
}

// A pointer that is the same in all lanes, in scalar registers: the loads' base
// has to be there, and the compiler divides in vector registers.
__device__ __forceinline__ const char* linear_uniform(const void* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return reinterpret_cast<const char*>((uint64_t)hi << 32 | lo);
}

// One operand's side of a tile of B lines. KROWS: its lines are k with the
// side's elements neighbouring.
//
// LDS with k neighbouring: 128 bytes a line; 16-byte piece p of line r lies at
// piece p ^ key(r), key = (r ^ r >> 3) & 7 of r mod 32, so that eight
// consecutive lines' pieces (and sixteen's) fall into different banks. A load
// covers 8 lines, lane l piece l & 7 of line l >> 3; a wave's loads are 32 lines
// apart and share their keys.
//
// LDS with k lines: 2 B bytes a k; the 64 bytes of a fragment's 32 elements are
// moved to group g ^ (k & 3), so that the transposing read (ds_read_b64_tr_b16: 16
// lanes read 4 k of 16 elements, lane j gets element j of the four; checked
// with an in-bounds probe) of eight k by 64 bytes meets every bank twice, the
// least for its 512 bytes.
template <int B, int F, bool KROWS>
struct LinearSide {
  static constexpr int LOADS = B / 32;
  static constexpr int PER = KROWS ? 512 / B : 8;  // lines a load covers
  int line, col;     // this lane's line in a load of g = 0, and its bytes in the line
  uint32_t at[KROWS ? F : 4];  // LDS bytes of this lane's operands (fragments, or steps)
  uint32_t ld2;      // bytes of a line

  __device__ __forceinline__ LinearSide(const LinearOperand& o, int lane, int wave, int w) : ld2((uint32_t)(2 * o.ld)) {
    if constexpr (KROWS) {
      constexpr int SLOTS = 64 / PER;
      line = wave * PER + lane / SLOTS;
      const int slot = lane % SLOTS;
      col = 16 * ((((slot >> 2) ^ (line & 3)) << 2) + (slot & 3));
      const int i16 = lane & 15, k = 8 * (lane >> 5) + (i16 >> 2);
#pragma unroll
      for (int i = 0; i < F; ++i)
        at[i] = k * (2 * B) + (((w * F + i) ^ (i16 >> 2)) << 6) + 32 * ((lane >> 4) & 1) + 8 * (i16 & 3);
    } else {
      line = 8 * wave + (lane >> 3);
      col = 16 * ((lane & 7) ^ ((lane >> 3) ^ wave));
      const int row = lane & 31, key = (row ^ (row >> 3)) & 7;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) at[ks] = w * F * 4096 + row * 128 + ((2 * ks + (lane >> 5)) ^ key) * 16;
    }
  }
  // Load g of a stage from `base` (its first line and k): lines, or elements of a
  // line, behind `last` read that one. With TAIL k from `k_left` on are zeros.
  template <bool TAIL>
  __device__ __forceinline__ void issue(const char* base, int last, int k_left, int g, uint32_t lds, int wave) const {
    const uint32_t to = lds + (wave + 4 * g) * 1024;
    uint32_t off;
    bool in;
    if constexpr (KROWS) {
      base += (int64_t)(4 * PER * g) * ld2;
      off = (uint32_t)line * ld2 + (uint32_t)min(col, 2 * last - 14);
      in = line + 4 * PER * g < k_left;
    } else {
      off = (uint32_t)min(line + 32 * g, last) * ld2 + (uint32_t)col;
      in = col < 2 * k_left;
    }
    if constexpr (TAIL)
      linear_dma_at(in ? base + off : reinterpret_cast<const char*>(&linear_zeros), to);
    else
      linear_dma(base, off, to);
  }
  __device__ __forceinline__ u32x4_t read(const char* stage, int i, int ks) const {
    if constexpr (KROWS) {
      typedef short s16x4_t __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) s16x4_t* lds_t;
      const char* p = stage + at[i] + 16 * ks * (2 * B);
      const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t)(p));
      const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t)(p + 4 * (2 * B)));
      const u32x2_t a = __builtin_bit_cast(u32x2_t, lo), b = __builtin_bit_cast(u32x2_t, hi);
      return u32x4_t{a[0], a[1], b[0], b[1]};
    } else {
      return *reinterpret_cast<const u32x4_t*>(stage + at[ks] + 4096 * i);
    }
  }
};

// f(0), .. f(N - 1) with constants: the compiler gives up unrolling a loop of
// that much code, and results with a variable index would go to scratch memory.
template <typename F, int... I>
__device__ __forceinline__ void linear_each_of(F f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void linear_each(F f) {
  linear_each_of(f, std::make_integer_sequence<int, N>{});
}

// A wave's results to memory, through LDS, TOK rows by 64 units at a time, so
// that a store writes whole lines (8 rows, 128 bytes of bf16 each) and the
// epilogue reads the residual that way. Rows may begin at any element.
template <class C, int ACT>
__device__ __forceinline__ void linear_store(const LinearOut& o, const f32x16_t (&acc)[C::FU][C::FT], int64_t row0,
                                             int unit0, char* out) {
  const int lane = threadIdx.x & 63, row = lane & 31, half = lane >> 5;
  const int col = 8 * (lane & 7);
  constexpr int TOK = C::TOK, PASSES = TOK / 8;
  float bias[C::FU / 2][8];
#pragma unroll
  for (int i = 0; i < C::FU / 2; ++i) {
    const int unit = unit0 + 64 * i + col;
    if (o.bias != nullptr) {
      load_some<8>(o.bias, o.bias_bf16, unit, o.units - unit, bias[i]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) bias[i][k] = 0.f;
    }
  }
  linear_each<C::FT>([&](auto J) __attribute__((always_inline)) {
    linear_each<32 / TOK>([&](auto H) __attribute__((always_inline)) {  // lanes of TOK rows write, all read
      constexpr int j = decltype(J)::value, h = decltype(H)::value;
      const bool mine = row / TOK == h;
      char* line = out + row % TOK * C::LINE;
      const int64_t first = row0 + 32 * j + TOK * h + (lane >> 3);
      float res[C::FU / 2][PASSES][8];
#pragma unroll
      for (int i = 0; i < C::FU / 2; ++i)
#pragma unroll
        for (int r = 0; r < PASSES; ++r) {
          const int unit = unit0 + 64 * i + col;
          if (o.residual != nullptr && first + 8 * r < o.rows) {
            load_some<8>(o.residual, o.res_bf16, (first + 8 * r) * o.units + unit, o.units - unit, res[i][r]);
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) res[i][r][k] = 0.f;
          }
        }
      linear_each<C::FU / 2>([&](auto I) __attribute__((always_inline)) {
        constexpr int i = decltype(I)::value;
        if (mine) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const f32x16_t& v = acc[2 * i + k][j];
              *reinterpret_cast<f32x4_t*>(line + 128 * k + 32 * q + 16 * half) =
                  f32x4_t{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
            }
        }
        // A wave's LDS operations are done in their order; the statements around
        // the reads keep the compiler to it, which sees no lane's write of what
        // another reads.
        asm volatile("" ::: "memory");
#pragma unroll
        for (int r = 0; r < PASSES; ++r) {
          float z[8];
          const char* at = out + (8 * r + (lane >> 3)) * C::LINE + 4 * col;
#pragma unroll
          for (int k = 0; k < 8; k += 4) {
            const f32x4_t v = *reinterpret_cast<const f32x4_t*>(at + 4 * k);
#pragma unroll
            for (int e = 0; e < 4; ++e) z[k + e] = v[e];
          }
          const int unit = unit0 + 64 * i + col;
          if (first + 8 * r < o.rows && unit < o.units)
            finish_units<ACT, 8>(o, first + 8 * r, unit, o.units - unit, z, bias[i], res[i][r]);
        }
        asm volatile("" ::: "memory");
      });
    });
  });
}

// Workgroup -> tile: each XCD takes a contiguous run of tiles, walked in
// groups of 4 row blocks so that the tiles in flight share lines in L2.
__device__ __forceinline__ void linear_tile_of(int64_t L, int64_t tb, int ub, int64_t& t, int& u) {
  constexpr int kGroup = 4;
  const int64_t per = (int64_t)kGroup * ub, first = L / per * kGroup;
  const int g = (int)min(tb - first, (int64_t)kGroup), in = (int)(L % per);
  t = first + in % g;
  u = in / g;
}

// TAIL: k is not a whole number of stages, or there is one stage: loads run two
// ahead, and the second one's k are zeros then.
template <class C, bool PK, bool QK, bool TAIL, int ACT>
__global__ __launch_bounds__(256, C::OCC) void linear_tiled(LinearArgs a, int64_t tb, int ub) {
  __shared__ __attribute__((aligned(1024))) char smem[C::LDS];
  constexpr int FU = C::FU, FT = C::FT;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wu = wave >> 1, wt = wave & 1;
  const LinearSide<C::BU, FU, PK> P(a.p, lane, wave, wu);
  const LinearSide<C::BT, FT, QK> Q(a.q, lane, wave, wt);
  const int stages = (int)((a.k + 63) / 64);

  // This workgroup's items (tiles, for each split): every n-th (n workgroups on
  // the XCD) of its XCD's run.
  const int64_t tiles = tb * ub, items = tiles * a.splits;
  const int xcd = blockIdx.x % 8;
  const int64_t run = items / 8, extra = items % 8;
  const int64_t end = (xcd + 1) * run + min((int64_t)xcd + 1, extra);
  const int64_t stride = (gridDim.x + 7 - xcd) / 8;
  int64_t L = xcd * run + min((int64_t)xcd, extra) + blockIdx.x / 8;
  if (L >= end) return;

  struct Item {
    const char *p, *q;   // first line and k
    int p_last, q_last;  // lines (or elements of a line) that there are, less one
    int64_t row0, k0;
    int unit0, count, split;  // stages: two at least
  };
  auto item_at = [&](int64_t l) {
    Item r;
    r.split = __builtin_amdgcn_readfirstlane((int)(l / tiles));
    int64_t t;
    int u;
    linear_tile_of(l - r.split * tiles, tb, ub, t, u);
    r.row0 = t * C::BT;
    r.unit0 = u * C::BU;
    const int s0 = (int)((int64_t)r.split * stages / a.splits), s1 = (int)((int64_t)(r.split + 1) * stages / a.splits);
    r.k0 = (int64_t)s0 * 64;
    r.count = __builtin_amdgcn_readfirstlane(max(s1 - s0, 2));
    r.p = linear_uniform(a.p.p + (PK ? r.k0 * a.p.ld + r.unit0 : r.unit0 * a.p.ld + r.k0));
    r.q = linear_uniform(a.q.p + (QK ? r.k0 * a.q.ld + r.row0 : r.row0 * a.q.ld + r.k0));
    // with k lines whole 16 bytes are read: to the next multiple of 8
    r.p_last = PK ? ((min(C::BU, a.out.units - r.unit0) + 7) & ~7) - 1 : min(C::BU, a.out.units - r.unit0) - 1;
    const int rows = (int)min((int64_t)C::BT, a.out.rows - r.row0);
    r.q_last = QK ? ((rows + 7) & ~7) - 1 : rows - 1;
    return r;
  };
  struct Stage {
    const char *p, *q;
    int p_last, q_last, k_left;
  };
  auto stage_at = [&](const Item& c, const Item& n, int kt) {  // past c's last: of n
    const bool in = kt < c.count;
    const int64_t k = in ? kt : kt - c.count;
    Stage r;
    r.p = (in ? c.p : n.p) + 128 * k * (PK ? a.p.ld : 1);
    r.q = (in ? c.q : n.q) + 128 * k * (QK ? a.q.ld : 1);
    r.p_last = in ? c.p_last : n.p_last;
    r.q_last = in ? c.q_last : n.q_last;
    r.k_left = TAIL ? (int)min(a.k - (in ? c.k0 : n.k0) - 64 * k, (int64_t)64) : 64;
    return r;
  };
  const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)(smem));
  auto issue = [&](const Stage& s, uint32_t buf, int g) {
    const uint32_t at = lds0 + buf * C::STAGE;
    if (g < C::UG) P.template issue<TAIL>(s.p, s.p_last, s.k_left, g, at, wave);
    else Q.template issue<TAIL>(s.q, s.q_last, s.k_left, g - C::UG, at + C::BU * 128, wave);
  };

  f32x16_t acc[FU][FT];
  u32x4_t av[4][FU], bv[4][FT];  // operands of a stage's four steps
  auto read_a = [&](int i, int ks, uint32_t buf) { return P.read(smem + buf * C::STAGE, i, ks); };
  auto read_b = [&](int j, int ks, uint32_t buf) { return Q.read(smem + buf * C::STAGE + C::BU * 128, j, ks); };
  auto mfma = [](const u32x4_t& x, const u32x4_t& y, const f32x16_t& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, x), __builtin_bit_cast(bf16x8_t, y), c, 0, 0, 0);
  };

  // Loads run two stages ahead, into the next item at an item's end; behind the
  // last one they read it again, unused.
  Item cur = item_at(L);
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
  for (int i = 0; i < FU; ++i) av[0][i] = read_a(i, 0, 0);
#pragma unroll
  for (int j = 0; j < FT; ++j) bv[0][j] = read_b(j, 0, 0);

  uint32_t buf = 0, stores = 0;  // stores: the item before has left MIN_STORES behind
  for (;;) {
    const bool more = L + stride < end;
    const Item next = more ? item_at(L + stride) : cur;
#pragma unroll
    for (int i = 0; i < FU; ++i)
#pragma unroll
      for (int j = 0; j < FT; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;

    for (int kt = 0; kt < cur.count; ++kt) {
      // Four steps of 16 k. All operands of the stage are in registers when the
      // second step ends, so that its LDS can be filled again during the third
      // and fourth; the next stage's first operands are read in the fourth.
      // Loads are spread over two steps: a wave that issues them at once waits
      // for the address unit and keeps its matrix core waiting.
      const Stage ahead = stage_at(cur, next, kt + 2);
      constexpr int OPS = FU + FT, M = FU * FT;  // operands and matrix instructions of a step
      auto read = [&](int r) {  // read r of the 3 OPS behind the first step's operands
        const int ks = 1 + r / OPS, k = r % OPS;
        if (k < FU) av[ks][k] = read_a(k, ks, buf);
        else bv[ks][k - FU] = read_b(k - FU, ks, buf);
      };
      auto read_next = [&](int r) {
        if (r < FU) av[0][r] = read_a(r, 0, buf ^ 1);
        else bv[0][r - FU] = read_b(r - FU, 0, buf ^ 1);
      };
      // Operation k of n that are dealt to slots [0, m): those of slot s.
      auto first_of = [](int s, int n, int m) { return s >= m ? n : s * n / m; };
      auto step = [&](auto KS) {
        constexpr int ks = decltype(KS)::value;
#pragma unroll
        for (int s = 0; s < M; ++s) {
          const int i = s / FT, j = s % FT;
          acc[i][j] = mfma(av[ks][i], bv[ks][j], acc[i][j]);
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
            for (int r = first_of(s, OPS, M / 2 + 1); r < first_of(s + 1, OPS, M / 2 + 1); ++r) read_next(r);
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
      // in an item's first stage the stores of the one before, which were
      // asked for later than it.
      linear_wait_either<C::LOADS / 2 + C::MIN_STORES, C::LOADS / 2>(stores & (uint32_t)(kt == 0));
      lds_barrier();
      __builtin_amdgcn_sched_barrier(0);
      step(std::integral_constant<int, 3>{});
      buf ^= 1;
    }

    LinearOut o = a.out;
    if (a.splits > 1) {  // the sums as they are
      o.y = a.part + (int64_t)cur.split * a.out.rows * a.out.units;
      o.y_bf16 = 0;
    }
    const int64_t row0 = cur.row0 + wt * FT * 32;
    const int unit0 = cur.unit0 + wu * FU * 32;
    linear_store<C, ACT>(o, acc, row0, unit0, smem + 2 * C::STAGE + wave * C::OUT);
    if (!more) break;
    // at the result's edges some have nothing to store, and may not have been issued
    stores = row0 + FT * 32 <= a.out.rows && unit0 + FU * 32 <= a.out.units;
    cur = next;
    L += stride;
  }
  wait_vmcnt<0>();  // no load may write to LDS behind the workgroup's end
}

using LinearBig = LinearTile<4, 4, 1>;
using LinearMid = LinearTile<2, 2, 2>;

template <class C, bool PK, bool QK, int ACT>
hipError_t launch_linear_tile(const LinearArgs& a, hipStream_t s) {
  const int64_t tb = (a.out.rows + C::BT - 1) / C::BT;
  const int ub = (a.out.units + C::BU - 1) / C::BU;
  const int64_t items = tb * ub * a.splits, fit = 256 * C::OCC;  // workgroups that run at a time
  const dim3 grid((unsigned)(items < fit ? items : fit));
  if (a.k % 64 == 0 && a.k > 64)
    TWELL_LAUNCH("linear_tiled", (linear_tiled<C, PK, QK, false, ACT>), grid, 256, 0, s, a, tb, ub);
  else
    TWELL_LAUNCH("linear_tiled", (linear_tiled<C, PK, QK, true, ACT>), grid, 256, 0, s, a, tb, ub);
  return hipGetLastError();
}

}  // namespace twell
