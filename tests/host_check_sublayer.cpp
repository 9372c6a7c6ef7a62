// Host-side check of the linear layer, the join and dropout (linear_api.hip,
// join_api.hip), built with g++ under AddressSanitizer and
// UndefinedBehaviorSanitizer: the buffers, extents and checks of
// host_check.cpp, whose driver is left aside, with stand-ins for the operators'
// launch functions. Every entry point is called with buffers of exactly the
// sizes that the queries and the header give, and every array handed to a
// kernel is checked to lie inside one of them.
#define main host_check_block_main
#include "host_check.cpp"
#undef main

#include "ops_kernels.h"

namespace twell {

hipError_t launch_join_rms_norm(const JoinArgs& a, hipStream_t) {
  const size_t n = (size_t)a.rows * a.cols;
  extent(a.residual, n * (a.res_bf16 ? 2 : 4), "residual");
  extent(a.y, n * (a.y_bf16 ? 2 : 4), "y");
  extent(a.w, (size_t)a.cols * (a.w_bf16 ? 2 : 4), "weight");
  if (a.post_w) extent(a.post_w, (size_t)a.cols * (a.post_bf16 ? 2 : 4), "post_weight");
  CHECK(a.per_gate >= 1, "rows of a gate");
  if (a.gate) extent(a.gate, ((size_t)(a.rows - 1) / a.per_gate + 1) * a.cols * (a.gate_bf16 ? 2 : 4), "gate");
  if (a.drop) extent(a.rng, 16, "rng");
  if (a.residual_out) extent(a.residual_out, n * (a.res_bf16 ? 2 : 4), "residual_out");
  if (a.out) extent(a.out, n * (a.out_bf16 ? 2 : 4), "out");
  if (a.q) extent(a.q, n, "q");
  if (a.q) extent(a.q_scale, (size_t)a.rows * 4, "q_scale");
  if (a.rstd) extent(a.rstd, (size_t)a.rows * 4, "rstd");
  if (a.post_rstd) extent(a.post_rstd, (size_t)a.rows * 4, "post_rstd");
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_join_rms_norm_bwd(const JoinBwdArgs& a, hipStream_t) {
  const size_t n = (size_t)a.rows * a.cols, er = a.res_bf16 ? 2 : 4, ey = a.y_bf16 ? 2 : 4;
  extent(a.d_out, n * (a.g_bf16 ? 2 : 4), "d_out");
  if (a.d_residual) extent(a.d_residual, n * er, "d_residual");
  extent(a.residual, n * er, "residual");
  extent(a.rstd, (size_t)a.rows * 4, "rstd");
  extent(a.y, n * ey, "y");
  extent(a.w, (size_t)a.cols * (a.w_bf16 ? 2 : 4), "weight");
  if (a.post_w) extent(a.post_w, (size_t)a.cols * (a.post_bf16 ? 2 : 4), "post_weight");
  if (a.post_w) extent(a.post_rstd, (size_t)a.rows * 4, "post_rstd");
  if (a.gate) extent(a.gate, (size_t)a.gates * a.cols * (a.gate_bf16 ? 2 : 4), "gate");
  if (a.drop) extent(a.rng, 16, "rng");
  extent(a.dr, n * er, "dr");
  extent(a.dy, n * ey, "dy");
  extent(a.dw, (size_t)a.cols * 4, "dw");
  if (a.post_w) extent(a.dpost, (size_t)a.cols * 4, "dpost");
  if (a.gate) extent(a.dgate, (size_t)a.gates * a.cols * 4, "dgate");
  const JoinBwdPlan p = join_bwd_plan(a.rows, a.cols, a.gates);
  CHECK(p.groups >= 1 && p.groups <= kJoinBwdGroups && p.parts >= 1, "%d groups, %d parts", p.groups, p.parts);
  CHECK(p.parts == 1 || (int64_t)p.groups == (int64_t)a.gates * p.parts, "%d groups of %d parts", p.groups, p.parts);
  // every workgroup has rows, and a launch of the sums has one row of workgroups for each
  if (a.rows > 0) CHECK((int64_t)p.groups <= a.rows && (p.parts == 1 || (int64_t)p.parts * a.gates <= a.rows), "groups without rows");
  const size_t sums = p.groups > 1 ? (size_t)p.groups * (a.post_w ? 2 : 1) : 0;
  extent(a.part, (sums + (a.gate && p.parts > 1 ? p.groups : 0)) * a.cols * 4, "ws.part");
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_dropout(const DropoutArgs& a, hipStream_t) {
  const size_t n = (size_t)a.rows * a.cols * (a.bf16 ? 2 : 4);
  extent(a.x, n, "x");
  extent(a.out, n, "out");
  extent(a.rng, 16, "rng");
  ++g_launches;
  return hipSuccess;
}

static int g_tiles[6], g_splits, g_any, g_pads;
hipError_t launch_linear(LinearLayout layout, const LinearPlan& plan, const LinearArgs& a, hipStream_t) {
  const LinearOut& o = a.out;
  ++g_tiles[plan.tile];
  g_splits += plan.splits > 1;
  g_any += a.any;
  const bool direct = plan.tile == LINEAR_DIRECT;
  CHECK(!direct || (layout == LINEAR_ROWS && plan.splits == 1), "straight from memory");
  CHECK(!(a.any && plan.tile >= LINEAR_TALL), "no registers");
  CHECK(plan.tile != LINEAR_TALL || layout == LINEAR_COLS, "a tile of one layout");
  // lines: of the side (p: units, q: rows) with k neighbouring, or k lines; read in whole 16 bytes unless at any element
  auto operand = [&](const LinearOperand& p, bool k_lines, bool any, int64_t side, const char* what) {
    const int64_t lines = k_lines ? a.k : side, line = k_lines ? side : a.k;
    CHECK(p.ld >= line, "%s: lines overlap", what);
    if (!any && !direct) {
      CHECK(p.ld % 8 == 0 && (reinterpret_cast<uintptr_t>(p.p) & 15) == 0, "%s: lines of part of 16 bytes", what);
      CHECK(p.ld >= linear_pad(line), "%s: a line's end", what);
    }
    if (any) CHECK(line >= 8 && !direct, "%s: short lines", what);
    extent(p.p, (size_t)((lines - 1) * p.ld + (any || direct ? line : linear_pad(line))) * 2, what);
  };
  operand(a.p, layout != LINEAR_ROWS, a.any, o.units, "p");
  operand(a.q, layout == LINEAR_COLS, a.any && layout == LINEAR_ROWS, o.rows, "q");
  const size_t n = (size_t)o.rows * o.units;
  extent(o.y, n * (o.y_bf16 ? 2 : 4), "y");
  if (o.pre) extent(o.pre, n * 2, "pre");
  if (o.residual) extent(o.residual, n * (o.res_bf16 ? 2 : 4), "residual");
  if (o.bias) extent(o.bias, (size_t)o.units * (o.bias_bf16 ? 2 : 4), "bias");
  const int64_t stages = (a.k + kLinearStage - 1) / kLinearStage;
  CHECK(plan.splits == 1 || plan.splits * (a.any ? 3 : 2) <= stages, "%d splits of %lld stages", plan.splits, (long long)stages);
  if (plan.splits > 1) extent(a.part, n * 4 * plan.splits, "ws.part");
  ++g_launches;
  return hipSuccess;
}
static int g_pairs;
hipError_t launch_linear_pair(const LinearArgs& dx, const LinearArgs& dw, hipStream_t s) {
  const int64_t tiles = (dx.out.units + 127) / 128 * ((dx.out.rows + 63) / 64 + (dw.out.rows + 63) / 64);
  CHECK(tiles <= 512 && dx.out.units == dw.out.units && dx.any == dw.any && dx.splits == 1 && dw.splits == 1, "pair");
  const LinearPlan few{LINEAR_FEW, 1, false, 0};
  ++g_pairs;
  launch_linear(LINEAR_MIXED, few, dx, s);
  return launch_linear(LINEAR_COLS, few, dw, s);
}
hipError_t launch_linear_zero(const LinearOut& o, hipStream_t) {
  extent(o.y, (size_t)o.rows * o.units * (o.y_bf16 ? 2 : 4), "dw");
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_linear_pad(const void* in, int64_t rows, int cols, void* out, int64_t ld, hipStream_t) {
  extent(in, (size_t)rows * cols * 2, "lines to copy");
  CHECK(ld % 8 == 0 && ld >= cols, "lines of %lld", (long long)ld);
  extent(out, (size_t)rows * ld * 2, "copied lines");
  ++g_pads;
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_linear_dz(const LinearDzArgs& a, hipStream_t) {
  const size_t n = (size_t)a.rows * a.units;
  extent(a.d_out, n * (a.g_bf16 ? 2 : 4), "d_out");
  if (a.act != TWELL_ACT_NONE) extent(a.pre, n * 2, "pre");
  if (a.dz) CHECK(a.ld % 8 == 0 && a.ld >= a.units, "lines of dz");
  if (a.dz) extent(a.dz, (size_t)a.rows * a.ld * 2, "dz");
  if (a.db) extent(a.db, (size_t)a.units * 4, "db");
  const int parts = linear_db_parts(a.rows, a.units);
  CHECK(parts >= 1 && parts <= 64, "%d parts", parts);
  if (a.db && parts > 1) extent(a.part, (size_t)parts * a.units * 4, "ws.db");
  ++g_launches;
  return hipSuccess;
}

}  // namespace twell

namespace {

size_t esz(twell_dtype t) { return t == TWELL_BF16 ? 2 : 4; }

void join_case(int64_t rows, int cols, int64_t gates, bool post, twell_dtype rt, twell_dtype yt) {
  g_where = "join " + std::to_string(rows) + "x" + std::to_string(cols) + " gates " + std::to_string(gates);
  const size_t n = (size_t)rows * cols;
  void *r = alloc(n * esz(rt), "r"), *y = alloc(n * esz(yt), "y"), *w = alloc(cols * esz(yt), "w");
  void *ro = alloc(n * esz(rt), "r_out"), *o = alloc(n * esz(yt), "out");
  uint8_t* q = (uint8_t*)alloc(n, "q");
  float *qs = (float*)alloc(rows * 4, "q_scale"), *rs = (float*)alloc(rows * 4, "rstd"), *ps = (float*)alloc(rows * 4, "post_rstd");
  twell_join j{};
  j.alpha = 1.f;
  j.p = 0.25f;
  j.rng = (const uint64_t*)alloc(16, "rng");
  j.post_weight = post ? alloc(cols * esz(rt), "post_weight") : nullptr;
  j.post_weight_dtype = rt;
  j.gate = gates ? alloc((size_t)gates * cols * esz(yt), "gate") : nullptr;
  j.gate_dtype = yt;
  j.gate_rows = gates;
  auto fwd = [&](void* out_r, void* out, uint8_t* codes, float* rstd, float* pr) {
    return twell_join_rms_norm(rows, cols, rt, r, yt, y, yt, w, &j, 1e-6f, out_r, yt, out, codes, codes ? qs : nullptr, rstd, pr,
                               nullptr);
  };
  CHECK(fwd(ro, o, q, rs, post ? ps : nullptr) == TWELL_OK, "%s", twell_last_error());
  CHECK(fwd(r, o, nullptr, nullptr, nullptr) == TWELL_OK, "in place: %s", twell_last_error());
  if (rows > 0) CHECK(fwd(nullptr, nullptr, nullptr, nullptr, nullptr) == TWELL_ERR_INVALID_ARG, "no output accepted");
  if (rows > 0 && !post) CHECK(fwd(ro, o, nullptr, nullptr, ps) == TWELL_ERR_INVALID_ARG, "post_rstd without its norm accepted");
  size_t need = 1;
  CHECK(twell_join_rms_norm_bwd_ws(rows, cols, post, gates, &need) == TWELL_OK, "%s", twell_last_error());
  void *ws = alloc(need, "bwd ws"), *dr = alloc(n * esz(rt), "dr"), *dy = alloc(n * esz(yt), "dy");
  float *dw = (float*)alloc(cols * 4, "dw"), *dp = post ? (float*)alloc(cols * 4, "dpost") : nullptr;
  float* dg = gates ? (float*)alloc((size_t)gates * cols * 4, "dgate") : nullptr;
  auto bwd = [&](void* ds, size_t have) {
    return twell_join_rms_norm_bwd(rows, cols, yt, o, rt, ds, ro, rs, yt, y, post ? ps : nullptr, yt, w, &j, dr, dy, dw, dp, dg,
                                   ws, have, nullptr);
  };
  CHECK(bwd(nullptr, need) == TWELL_OK && bwd(r, need) == TWELL_OK, "%s", twell_last_error());
  const int mark = g_launches;
  if (need > 0) CHECK(bwd(nullptr, need - 1) == TWELL_ERR_WORKSPACE, "short workspace accepted");
  CHECK(g_launches == mark, "an invalid call reached a launch");
  CHECK(twell_dropout(rows, cols, rt, r, 0.5f, j.rng, 0, ro, nullptr) == TWELL_OK, "%s", twell_last_error());
  free_all();
}

void linear_case(int64_t n, int cols, int units, int act, twell_dtype a, twell_dtype b) {
  g_where = "linear " + std::to_string(n) + "x" + std::to_string(cols) + "x" + std::to_string(units);
  const size_t results = (size_t)n * units;
  void *x = alloc((size_t)n * cols * 2, "x"), *w = alloc((size_t)units * cols * 2, "w"), *y = alloc(results * esz(a), "y");
  void *bias = alloc(units * esz(b), "bias"), *res = alloc(results * esz(b), "residual"), *pre = alloc(results * 2, "pre");
  size_t need = 1;
  CHECK(twell_linear_ws(n, cols, units, &need) == TWELL_OK, "%s", twell_last_error());
  void* ws = alloc(need, "ws");
  CHECK(twell_linear(n, cols, units, x, w, b, bias, act, b, res, pre, a, y, ws, need, nullptr) == TWELL_OK, "%s", twell_last_error());
  CHECK(twell_linear(n, cols, units, x, w, b, nullptr, act, b, nullptr, nullptr, a, y, ws, need, nullptr) == TWELL_OK, "%s",
        twell_last_error());
  int mark = g_launches;
  if (need > 0)
    CHECK(twell_linear(n, cols, units, x, w, b, bias, act, b, res, pre, a, y, ws, need - 1, nullptr) == TWELL_ERR_WORKSPACE, "short");
  CHECK(g_launches == mark, "an invalid call reached a launch");
  void *g = alloc(results * esz(b), "d_out"), *dx = alloc((size_t)n * cols * esz(a), "dx"), *dw = alloc((size_t)units * cols * esz(b), "dw");
  float* db = (float*)alloc(units * 4, "db");
  for (uint32_t want = 1; want < 8; ++want) {
    size_t nb = 1;
    CHECK(twell_linear_bwd_ws(n, cols, units, b, act, want, &nb) == TWELL_OK, "%s", twell_last_error());
    void* wb = alloc(nb, "bwd ws");
    auto bwd = [&](size_t have) {
      return twell_linear_bwd(n, cols, units, b, g, act, act ? pre : nullptr, want & TWELL_LINEAR_DW ? x : nullptr,
                              want & TWELL_LINEAR_DX ? w : nullptr, a, want & TWELL_LINEAR_DX ? dx : nullptr, b,
                              want & TWELL_LINEAR_DW ? dw : nullptr, want & TWELL_LINEAR_DB ? db : nullptr, wb, have, nullptr);
    };
    CHECK(bwd(nb) == TWELL_OK, "%s", twell_last_error());
    mark = g_launches;
    if (nb > 0 && n > 0) CHECK(bwd(nb - 1) == TWELL_ERR_WORKSPACE, "short workspace accepted");
    CHECK(g_launches == mark, "an invalid call reached a launch");
  }
  free_all();
}

}  // namespace

int main() {
  for (int64_t rows : {0, 1, 2, 12, 96, 513, 516, 3000})
    for (int cols : {1, 7, 95, 128, 256, 500, 1000, 1999, 4096, 8200, 16384}) {
      if (rows * cols > 4000000) continue;
      for (int64_t gates : {(int64_t)0, (int64_t)1, (int64_t)3, (int64_t)12, rows / 2, rows}) {
        if (gates > 0 && rows % gates != 0) continue;
        join_case(rows, cols, gates, true, TWELL_BF16, TWELL_F32);
        join_case(rows, cols, gates, false, TWELL_F32, TWELL_BF16);
      }
    }
  for (int64_t n : {0, 1, 8, 24, 33, 64, 100, 257, 1000, 4100})
    for (int cols : {1, 7, 8, 63, 100, 129, 1990, 4096})
      for (int units : {1, 5, 64, 100, 129, 515, 2048, 4100}) {
        if (n * units > 5000000 || n * cols > 5000000 || units * cols > 5000000) continue;
        linear_case(n, cols, units, TWELL_ACT_NONE, TWELL_BF16, TWELL_BF16);
        linear_case(n, cols, units, TWELL_ACT_GELU, TWELL_F32, TWELL_F32);
      }
  linear_case(1500, 200, 4104, TWELL_ACT_NONE, TWELL_BF16, TWELL_BF16);
  linear_case(4100, 200, 3000, TWELL_ACT_NONE, TWELL_BF16, TWELL_F32);
  linear_case(300, 8192, 4000, TWELL_ACT_SILU, TWELL_F32, TWELL_BF16);
  linear_case(3000, 2001, 4105, TWELL_ACT_RELU, TWELL_BF16, TWELL_F32);
  g_where = "plans";
  for (int p = 0; p < 6; ++p) CHECK(twell::g_tiles[p] > 0, "tile %d was not reached", p);
  CHECK(twell::g_splits > 0 && twell::g_any > 0 && twell::g_pads > 0, "splits, lines at any element, copies");

  g_where = "pairs";  // tokens, columns, units of test_gpu_linear_variants.py's
  const int pairs[][3] = {{1, 8, 1}, {33, 100, 100}, {64, 128, 64}, {65, 129, 63}, {1, 4096, 500}, {500, 1000, 9},
                          {509, 1000, 1021}, {509, 1021, 1000}, {2049, 264, 500}, {2000, 1001, 2000}, {2048, 1024, 2048}};
  for (const auto& p : pairs) {
    const int before = twell::g_pairs;
    linear_case(p[0], p[1], p[2], TWELL_ACT_NONE, TWELL_BF16, TWELL_BF16);
    CHECK(twell::g_pairs > before, "%d x %d x %d in two launches", p[0], p[1], p[2]);
  }

  g_where = "tiles of a launch";
  for (int64_t n : {0x7FFFFFFFll, (1ll << 30) + 1, 1ll << 24, 1ll << 20})
    for (int units : {1, 8, 15, 100, 129, 2304, 1 << 20})
      for (int64_t k : {8ll, 64ll, 100000ll})
        for (bool any : {false, true})
          for (int layout = 0; layout < 3; ++layout) {
            if (n * ((units + 7) / 8) >= (1ll << 32) - 256) continue;
            const twell::LinearPlan p = twell::linear_plan((twell::LinearLayout)layout, n, k, units, any);
            CHECK(p.tile != twell::LINEAR_DIRECT && twell::linear_tiles(p.tile, n, units) * p.splits < twell::kLinearMaxItems,
                  "%lld x %lld x %d", (long long)n, (long long)k, units);
          }

  g_where = "limits";
  size_t b = 0;
  CHECK(twell_linear_ws(1, 1 << 20, 1 << 20, &b) == TWELL_OK, "%s", twell_last_error());
  CHECK(twell_linear_ws(1, (1 << 20) + 1, 8, &b) == TWELL_ERR_UNSUPPORTED, "too many columns accepted");
  CHECK(twell_linear_ws(0x7FFFFFFFll, 64, 64, &b) == TWELL_ERR_UNSUPPORTED, "too many pieces accepted");
  CHECK(twell_join_rms_norm_bwd_ws(0x7FFFFFFFll, 16384, 1, 0x7FFFFFFFll, &b) == TWELL_OK, "%s", twell_last_error());
  if (g_failures) {
    std::fprintf(stderr, "%d check(s) failed\n", g_failures);
    return 1;
  }
  std::printf("host check ok: %d launches checked\n", g_launches);
  return 0;
}
