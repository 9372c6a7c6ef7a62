// Backward of the join. With xh = r' * rho, yh = y * rho_y (or y itself) and m
// what dropout multiplies with (0 or one over the share that is kept):
//
//   G     = d_residual + rho * (d_out * w - xh * c)       c  = mean(d_out * w * xh)
//   dr    = alpha * G
//   dv    = G * gate * m
//   dy    = rho_y * (dv * post_w - yh * c2)               c2 = mean(dv * post_w * yh)
//   dw    = sum of d_out * xh,  dpost = sum of dv * yh,  dgate = sum of G * m * yh * post_w over the rows that share it
//
// (without the norm behind the block dy = dv and dgate sums G * m * y). c2 needs
// G, which needs c: it is taken apart into sums that do not,
//   sum(dv post_w yh) = sum((d_residual + rho d_out w) k yh) - rho c sum(xh k yh),  k = gate m post_w,
// so that a row is reduced once, three sums at a time.
//
// Bound by memory: one pass over d_out, d_residual, r' and y (8192 x 2048 52 us,
// 5.1 TB/s, 5 of them the second launch; 131 x 1000 8). A workgroup takes
// rows that share one row of the gate, or all rows of several rows of it, keeps
// its sums in registers (thread t owns the same columns in every row) and leaves
// partial rows; a second launch adds them in a fixed order.
#include "counter_rng.h"
#include "ops_kernels.h"
#include "../csrc/twell_trace.h"

namespace twell {
namespace {

// Eight elements of either type (uniform over the launch).
struct RawAny {
  u32x4_t v[2];
  template <int KIND>
  __device__ __forceinline__ void load(const void* base, int is_bf16, int64_t off, int i, int cols) {
    if (is_bf16) {
      Raw8<uint16_t> r;
      r.load<KIND>(static_cast<const uint16_t*>(base) + off, i, cols);
      v[0] = r.v;
    } else {
      Raw8<float> r;
      r.load<KIND>(static_cast<const float*>(base) + off, i, cols);
      v[0] = r.v[0];
      v[1] = r.v[1];
    }
  }
  __device__ __forceinline__ float get(int k, int is_bf16) const {
    const uint32_t b = k & 1 ? v[0][k >> 1] & 0xFFFF0000u : v[0][k >> 1] << 16;
    return __uint_as_float(is_bf16 ? b : v[k >> 2][k & 3]);
  }
};

// EACH: every row has a gate of its own, which is loaded with the row.
template <typename TR, typename TY, int NT, int T, int KIND, bool EACH>
__global__ __launch_bounds__(NT) void join_bwd_kernel(JoinBwdArgs a, int parts) {
  constexpr int C = 1;                // chunks of a thread
  constexpr int ROWS = NT / T;        // rows a workgroup takes at a time
  constexpr int G = T < 64 ? T : 64;  // lanes of a wave that share a row
  constexpr int WPR = T / G;          // waves of a row
  const int wave = threadIdx.x >> 6, t = threadIdx.x % T, side = threadIdx.x / T;
  const int cols = a.cols, b = blockIdx.x;
  const bool has_stream = a.d_residual != nullptr, has_post = a.post_w != nullptr, has_gate = a.gate != nullptr;
  const bool drops = a.drop != 0;

  struct Row {
    Raw8<TR> r[C], s[C];
    Raw8<TY> y[C];
    RawAny g[C], gate[EACH ? C : 1];
    float rho, rho_y;
  };
  auto fetch = [&](int64_t row, Row& x) {
    const int64_t off = row * cols;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      x.r[c].template load<KIND>(static_cast<const TR*>(a.residual) + off, t + T * c, cols);
      x.y[c].template load<KIND>(static_cast<const TY*>(a.y) + off, t + T * c, cols);
      x.g[c].template load<KIND>(a.d_out, a.g_bf16, off, t + T * c, cols);
      if constexpr (EACH) x.gate[c].template load<KIND>(a.gate, a.gate_bf16, off, t + T * c, cols);
    }
    // zeros without a gradient of the stream, and below ones without a weight or
    // gate: branches over whole rows would keep their terms in registers
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (has_stream) x.s[c].template load<KIND>(static_cast<const TR*>(a.d_residual) + off, t + T * c, cols);
      else x.s[c] = {};
    }
    x.rho = a.rstd[row];
    x.rho_y = has_post ? a.post_rstd[row] : 1.f;
  };

  float w[C][8], post[C][8], gate[EACH ? 1 : C][8];
  load_weight<T, C, KIND>(a.w, a.w_bf16, t, cols, w);
  if (has_post) {
    load_weight<T, C, KIND>(a.post_w, a.post_bf16, t, cols, post);
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) post[c][k] = 1.f;
  }
  float dw[C][8], dpost[C][8], dgate[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[c][k] = dpost[c][k] = dgate[c][k] = 0.f;

  // The sums of the rows taken side by side, added in their order, to `to`.
  __shared__ float acc[ROWS > 1 ? ROWS : 1][ROWS > 1 ? 8 : 1][ROWS > 1 ? T : 1];
  auto put = [&](float (&sum)[C][8], float* to) {
    if constexpr (ROWS > 1) {
      __syncthreads();  // what was put before has been read
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[side][k][t] = sum[0][k];
      __syncthreads();
      if (side > 0) return;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        for (int i = 1; i < ROWS; ++i) sum[0][k] += acc[i][k][t];
    }
#pragma unroll
    for (int c = 0; c < C; ++c) store8<KIND>(to, t + T * c, cols, sum[c]);
  };

  const DropArgs drop_args{a.rng, a.site, a.drop, a.drop_scale};
  DropBits bits = drops ? DropBits(drop_args) : DropBits();
  __shared__ float red[2][3][ROWS][WPR];
  int flip = 0;
  // Rows of the gate of this workgroup; with EACH rows are dealt as they are.
  const int64_t per = EACH ? a.rows : a.rows / a.gates;
  const int64_t gates = EACH ? 1 : a.gates;
  const bool shared = EACH || parts > 1;  // several workgroups for one row of the gate
  const int n = EACH ? (int)gridDim.x : parts;
  const int64_t first_gate = shared ? b / n : b * gates / gridDim.x;
  const int64_t end_gate = shared ? first_gate + 1 : (b + 1) * gates / gridDim.x;
  const int64_t slice = shared ? b % n : 0, slices = shared ? n : 1;
  for (int64_t gr = first_gate; gr < end_gate; ++gr) {
    const int64_t r0 = gr * per + slice * per / slices, r1 = gr * per + (slice + 1) * per / slices;
    int64_t row = r0 + side;
    Row now, next;
    if (row < r1) fetch(row, now);
    if constexpr (!EACH) {
      if (has_gate) {
        load_weight<T, C, KIND>(static_cast<const char*>(a.gate) + gr * cols * (a.gate_bf16 ? 2 : 4), a.gate_bf16, t,
                                cols, gate);
      } else {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int k = 0; k < 8; ++k) gate[c][k] = 1.f;
      }
    }
    for (int64_t first = r0; first < r1; first += ROWS, row += ROWS) {  // the same number of times in every wave
      const bool here = row < r1;
      if (row + ROWS < r1) fetch(row + ROWS, next);
      uint32_t keep[C];
#pragma unroll
      for (int c = 0; c < C; ++c) keep[c] = drops ? bits.template chunk<KIND>((uint32_t)row, t + T * c, cols) : 0xFFu;
      auto gate_at = [&](int c, int k) {
        if constexpr (EACH) return now.gate[c].get(k, a.gate_bf16);
        else return gate[c][k];
      };
      float s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float xh = now.r[c].get(k) * now.rho, g = now.g[c].get(k, a.g_bf16), u = g * w[c][k];
          if (here) dw[c][k] = fmaf(g, xh, dw[c][k]);
          const bool counts = chunk_counts<KIND>(t + T * c, k, cols);
          const float base = fmaf(now.rho, u, now.s[c].get(k));
          const float kyh = keep[c] >> k & 1 ? gate_at(c, k) * a.drop_scale * post[c][k] * (now.y[c].get(k) * now.rho_y) : 0.f;
          if (counts) {
            s1 = fmaf(u, xh, s1);
            s2 = fmaf(base, kyh, s2);
            s3 = fmaf(xh, kyh, s3);
          }
        }
      s1 = group_sum<G>(s1);
      s2 = group_sum<G>(s2);
      s3 = group_sum<G>(s3);
      if constexpr (WPR > 1) {
        // two buffers: a wave may write the next row's sums while another still
        // reads this row's
        if ((threadIdx.x & 63) == 0) {
          red[flip][0][side][wave % WPR] = s1;
          red[flip][1][side][wave % WPR] = s2;
          red[flip][2][side][wave % WPR] = s3;
        }
        lds_barrier();
        s1 = s2 = s3 = 0.f;
#pragma unroll
        for (int i = 0; i < WPR; ++i) {
          s1 += red[flip][0][side][i];
          s2 += red[flip][1][side][i];
          s3 += red[flip][2][side][i];
        }
        flip ^= 1;
      }
      const float c1 = s1 / (float)cols, c2 = (s2 - now.rho * c1 * s3) / (float)cols;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float dr[8], dy[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float xh = now.r[c].get(k) * now.rho;
          const float d = fmaf(now.rho, now.g[c].get(k, a.g_bf16) * w[c][k] - xh * c1, now.s[c].get(k));
          dr[k] = a.alpha * d;
          const float yh = now.y[c].get(k) * now.rho_y;  // y itself without the norm: rho_y is 1 then
          const bool kept = keep[c] >> k & 1;
          const float dm = kept ? d * a.drop_scale : 0.f, dv = dm * gate_at(c, k);
          const float u = kept ? yh * post[c][k] : 0.f;
          if constexpr (EACH) {
            dgate[c][k] = dm * u;
          } else {
            if (here) dgate[c][k] = fmaf(dm, u, dgate[c][k]);
          }
          if (here) dpost[c][k] = fmaf(dv, yh, dpost[c][k]);
          dy[k] = now.rho_y * (dv * post[c][k] - (has_post ? yh * c2 : 0.f));  // dv without the norm, whatever y holds
        }
        if (here) {
          store8<KIND>(static_cast<TR*>(a.dr) + row * cols, t + T * c, cols, dr);
          store8<KIND>(static_cast<TY*>(a.dy) + row * cols, t + T * c, cols, dy);
          if constexpr (EACH) store8<KIND>(a.dgate + row * cols, t + T * c, cols, dgate[c]);
        }
      }
      now = next;
    }
    if (!EACH && has_gate) {
      const bool part = parts > 1;
      put(dgate, part ? a.part + ((int64_t)gridDim.x * (has_post ? 2 : 1) + b) * cols : a.dgate + gr * cols);
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k) dgate[c][k] = 0.f;
    }
  }
  const bool alone = gridDim.x == 1;
  put(dw, alone ? a.dw : a.part + (int64_t)b * cols);
  if (has_post) put(dpost, alone ? a.dpost : a.part + ((int64_t)gridDim.x + b) * cols);
}

// Rows of more than 4096 elements: 512 threads a row, C chunks each, one chunk at a
// time. Only the sums are kept; a chunk's operands and weights are read for the
// row's sums, and again, from L2 then, for what follows them (kept in registers
// they went to scratch memory: 2000 x 8192 122 us, 1000 x 16384 352). A chunk's
// loads wait for the chunk before by a dependence of their addresses, without
// which the compiler still hoists them all into scratch memory; with four chunks
// two of the sums lie in LDS. 2000 x 8192 114 -> 80 us, 1000 x 16384 278 -> 89.
template <typename TR, typename TY, int C, int KIND>
__global__ __launch_bounds__(512) void join_bwd_wide_kernel(JoinBwdArgs a, int parts, int each) {
  constexpr int T = 512, WAVES = T / 64;
  const int wave = threadIdx.x >> 6, t = threadIdx.x, cols = a.cols, b = blockIdx.x;
  const bool has_stream = a.d_residual != nullptr, has_post = a.post_w != nullptr, has_gate = a.gate != nullptr;
  const bool drops = a.drop != 0;
  float dgate[C][8];
  // two of the three sums: registers, or LDS where they would not fit; a thread
  // touches only its own
  constexpr bool LDS = C > 2;
  __shared__ float lds_sum[LDS ? 2 : 1][LDS ? C * 8 : 1][LDS ? T : 1];
  float reg_sum[2][LDS ? 1 : C][8];
  auto sum_at = [&](int which, int c, int k) -> float& {
    if constexpr (LDS) return lds_sum[which][c * 8 + k][t];
    else return reg_sum[which][c][k];
  };
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int k = 0; k < 8; ++k) sum_at(0, c, k) = sum_at(1, c, k) = dgate[c][k] = 0.f;
  const DropArgs drop_args{a.rng, a.site, a.drop, a.drop_scale};
  const DropBits bits = drops ? DropBits(drop_args) : DropBits();
  __shared__ float red[2][3][WAVES];
  int flip = 0;
  // rows of the gate of this workgroup, as in join_bwd_kernel
  const int64_t per = each ? a.rows : a.rows / a.gates, gates = each ? 1 : a.gates;
  const bool shared = each || parts > 1;
  const int n = each ? (int)gridDim.x : parts;
  const int64_t first_gate = shared ? b / n : b * gates / gridDim.x;
  const int64_t end_gate = shared ? first_gate + 1 : (b + 1) * gates / gridDim.x;
  const int64_t slice = shared ? b % n : 0, slices = shared ? n : 1;
  for (int64_t gr = first_gate; gr < end_gate; ++gr) {
    const int64_t r0 = gr * per + slice * per / slices, r1 = gr * per + (slice + 1) * per / slices;
    for (int64_t row = r0; row < r1; ++row) {
      const int64_t off = row * cols, gate_off = (each ? row : gr) * cols;
      const float rho = a.rstd[row], rho_y = has_post ? a.post_rstd[row] : 1.f;
      struct Operands {
        Raw8<TR> r, s;
        Raw8<TY> y;
        RawAny g, w, post, gate;
        uint32_t keep;
      };
      // `after`: a result of the chunk before, without which this one's loads do
      // not begin
      auto fetch = [&](int c, Operands& x, float after) {
        int i = t + T * c;
        asm volatile("" : "+v"(i) : "v"(after));
        x.r.template load<KIND>(static_cast<const TR*>(a.residual) + off, i, cols);
        x.y.template load<KIND>(static_cast<const TY*>(a.y) + off, i, cols);
        x.g.template load<KIND>(a.d_out, a.g_bf16, off, i, cols);
        if (has_stream) x.s.template load<KIND>(static_cast<const TR*>(a.d_residual) + off, i, cols);
        else x.s = {};
        x.w.template load<KIND>(a.w, a.w_bf16, 0, i, cols);
        if (has_post) x.post.template load<KIND>(a.post_w, a.post_bf16, 0, i, cols);
        if (has_gate) x.gate.template load<KIND>(a.gate, a.gate_bf16, gate_off, i, cols);
        x.keep = drops ? bits.template chunk<KIND>((uint32_t)row, i, cols) : 0xFFu;
      };
      float s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        Operands x;
        fetch(c, x, s3);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float xh = x.r.get(k) * rho, g = x.g.get(k, a.g_bf16), u = g * x.w.get(k, a.w_bf16);
          const float post = has_post ? x.post.get(k, a.post_bf16) : 1.f, gate = has_gate ? x.gate.get(k, a.gate_bf16) : 1.f;
          sum_at(0, c, k) = fmaf(g, xh, sum_at(0, c, k));
          const float base = fmaf(rho, u, x.s.get(k));
          const float kyh = x.keep >> k & 1 ? gate * a.drop_scale * post * (x.y.get(k) * rho_y) : 0.f;
          if (chunk_counts<KIND>(t + T * c, k, cols)) {
            s1 = fmaf(u, xh, s1);
            s2 = fmaf(base, kyh, s2);
            s3 = fmaf(xh, kyh, s3);
          }
        }
        __builtin_amdgcn_sched_barrier(0);  // one chunk at a time
      }
      s1 = group_sum<64>(s1);
      s2 = group_sum<64>(s2);
      s3 = group_sum<64>(s3);
      if ((t & 63) == 0) {
        red[flip][0][wave] = s1;
        red[flip][1][wave] = s2;
        red[flip][2][wave] = s3;
      }
      lds_barrier();
      s1 = s2 = s3 = 0.f;
#pragma unroll
      for (int i = 0; i < WAVES; ++i) {
        s1 += red[flip][0][i];
        s2 += red[flip][1][i];
        s3 += red[flip][2][i];
      }
      flip ^= 1;
      const float c1 = s1 / (float)cols, c2 = (s2 - rho * c1 * s3) / (float)cols;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        Operands x;
        fetch(c, x, c == 0 ? c2 : dgate[c - 1][7]);
        float dr[8], dy[8], dg[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float post = has_post ? x.post.get(k, a.post_bf16) : 1.f, gate = has_gate ? x.gate.get(k, a.gate_bf16) : 1.f;
          const float xh = x.r.get(k) * rho;
          const float d = fmaf(rho, x.g.get(k, a.g_bf16) * x.w.get(k, a.w_bf16) - xh * c1, x.s.get(k));
          dr[k] = a.alpha * d;
          const float yh = x.y.get(k) * rho_y;
          const bool kept = x.keep >> k & 1;
          const float dm = kept ? d * a.drop_scale : 0.f, dv = dm * gate, u = kept ? yh * post : 0.f;
          dg[k] = dm * u;
          dgate[c][k] += dg[k];
          sum_at(1, c, k) = fmaf(dv, yh, sum_at(1, c, k));
          dy[k] = rho_y * (dv * post - (has_post ? yh * c2 : 0.f));
        }
        store8<KIND>(static_cast<TR*>(a.dr) + off, t + T * c, cols, dr);
        store8<KIND>(static_cast<TY*>(a.dy) + off, t + T * c, cols, dy);
        if (each) store8<KIND>(a.dgate + off, t + T * c, cols, dg);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (!each && has_gate) {
      float* to = parts > 1 ? a.part + ((int64_t)gridDim.x * (has_post ? 2 : 1) + b) * cols : a.dgate + gr * cols;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        store8<KIND>(to, t + T * c, cols, dgate[c]);
#pragma unroll
        for (int k = 0; k < 8; ++k) dgate[c][k] = 0.f;
      }
    }
  }
  const bool alone = gridDim.x == 1;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if (which == 1 && !has_post) break;
    float* to = which == 0 ? (alone ? a.dw : a.part + (int64_t)b * cols) : alone ? a.dpost : a.part + ((int64_t)gridDim.x + b) * cols;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = sum_at(which, c, k);
      store8<KIND>(to, t + T * c, cols, v);
    }
  }
}

// Sums of partial rows: a workgroup takes 64 columns of one of them, each of its
// 16 waves every 16th row in ascending order, then the 16 sums in order. Sum 0 is
// dw, then dpost if it is there, then the rows of the gate, `parts` rows each.
__global__ __launch_bounds__(1024) void join_bwd_sum(JoinBwdArgs a, int groups, int parts) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + lane, whole = a.post_w != nullptr ? 2 : 1, which = blockIdx.y;
  const int rows = which < whole ? groups : parts;
  const float* part = a.part + (which < whole ? (int64_t)which * groups : (int64_t)whole * groups + (int64_t)(which - whole) * parts) * a.cols;
  float* out = which == 0 ? a.dw : which < whole ? a.dpost : a.dgate + (int64_t)(which - whole) * a.cols;
  float s = 0.f;
  if (col < a.cols) {
#pragma unroll 8
    for (int g = wave; g < rows; g += 16) s += part[(int64_t)g * a.cols + col];
  }
  red[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && col < a.cols) {
    for (int i = 1; i < 16; ++i) s += red[i][lane];
    out[col] = s;
  }
}

template <typename TR, typename TY, int NT, int T, int C>
hipError_t launch_cfg(const JoinBwdArgs& a, hipStream_t s) {
  const JoinBwdPlan p = join_bwd_plan(a.rows, a.cols, a.gates);
  const bool each = a.gate != nullptr && a.gates == a.rows && a.rows > 1;
  row_kind(a.cols, [&](auto kind) {
    constexpr int KIND = decltype(kind)::value;
    if constexpr (C > 1) {
      if constexpr (KIND != ROWS_SHORT)
        TWELL_LAUNCH("join_rms_norm_bwd", (join_bwd_wide_kernel<TR, TY, C, KIND>), dim3(p.groups), NT, 0, s, a, p.parts, each);
    } else if constexpr (KIND != ROWS_SHORT || T == 16) {
      if (each)
        TWELL_LAUNCH("join_rms_norm_bwd", (join_bwd_kernel<TR, TY, NT, T, KIND, true>), dim3(p.groups), NT, 0, s, a, p.parts);
      else
        TWELL_LAUNCH("join_rms_norm_bwd", (join_bwd_kernel<TR, TY, NT, T, KIND, false>), dim3(p.groups), NT, 0, s, a, p.parts);
    }
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.groups == 1) return e;
  const int sums = (a.post_w != nullptr ? 2 : 1) + (a.gate != nullptr && p.parts > 1 ? (int)a.gates : 0);
  TWELL_LAUNCH("join_bwd_sum", join_bwd_sum, dim3((a.cols + 63) / 64, sums), 1024, 0, s, a, p.groups, p.parts);
  return hipGetLastError();
}

template <typename TR, typename TY>
hipError_t launch_typed(const JoinBwdArgs& a, hipStream_t s) {
  if (a.cols <= 128) return launch_cfg<TR, TY, 512, 16, 1>(a, s);
  if (a.cols <= 256) return launch_cfg<TR, TY, 512, 32, 1>(a, s);
  if (a.cols <= 512) return launch_cfg<TR, TY, 512, 64, 1>(a, s);
  if (a.cols <= 1024) return launch_cfg<TR, TY, 512, 128, 1>(a, s);
  if (a.cols <= 2048) return launch_cfg<TR, TY, 512, 256, 1>(a, s);
  if (a.cols <= 4096) return launch_cfg<TR, TY, 512, 512, 1>(a, s);
  if (a.cols <= 8192) return launch_cfg<TR, TY, 512, 512, 2>(a, s);
  return launch_cfg<TR, TY, 512, 512, 4>(a, s);
}

}  // namespace

hipError_t launch_join_rms_norm_bwd(const JoinBwdArgs& a, hipStream_t s) {
  if (a.res_bf16) return a.y_bf16 ? launch_typed<uint16_t, uint16_t>(a, s) : launch_typed<uint16_t, float>(a, s);
  return a.y_bf16 ? launch_typed<float, uint16_t>(a, s) : launch_typed<float, float>(a, s);
}

}  // namespace twell
