// Host-side check of the operators around the block (ops_api.hip), built with
// g++ under AddressSanitizer and UndefinedBehaviorSanitizer: the buffers,
// extents and checks of host_check.cpp, whose driver is left aside, with
// stand-ins for the operators' launch functions. Every entry point is called
// with buffers of exactly the sizes that the queries and the header give, and
// every array handed to a kernel is checked to lie inside one of them.
#define main host_check_block_main
#include "host_check.cpp"
#undef main

#include "ops_kernels.h"

namespace twell {

hipError_t launch_add_rms_norm(const NormArgs& a, hipStream_t) {
  const size_t n = (size_t)a.rows * a.cols, er = a.res_bf16 ? 2 : 4;
  extent(a.residual, n * er, "residual");
  if (a.delta) extent(a.delta, n * (a.delta_bf16 ? 2 : 4), "delta");
  extent(a.w, (size_t)a.cols * (a.w_bf16 ? 2 : 4), "weight");
  if (a.residual_out) extent(a.residual_out, n * er, "residual_out");
  if (a.out) extent(a.out, n * (a.out_bf16 ? 2 : 4), "out");
  if (a.q) extent(a.q, n, "q");
  if (a.q) extent(a.q_scale, (size_t)a.rows * 4, "q_scale");
  if (a.rstd) extent(a.rstd, (size_t)a.rows * 4, "rstd");
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_add_rms_norm_bwd(const NormBwdArgs& a, hipStream_t) {
  const size_t n = (size_t)a.rows * a.cols, er = a.res_bf16 ? 2 : 4;
  extent(a.d_out, n * (a.g_bf16 ? 2 : 4), "d_out");
  if (a.d_residual) extent(a.d_residual, n * er, "d_residual");
  extent(a.residual, n * er, "residual");
  extent(a.rstd, (size_t)a.rows * 4, "rstd");
  extent(a.w, (size_t)a.cols * (a.w_bf16 ? 2 : 4), "weight");
  extent(a.dr, n * er, "dr");
  extent(a.dw, (size_t)a.cols * 4, "dw");
  const int groups = norm_bwd_groups(a.rows, a.cols);
  CHECK(groups >= 1 && (int64_t)(groups - 1) * norm_bwd_rows(a.cols) < (a.rows > 0 ? a.rows : 1), "%d groups", groups);
  if (groups > 1) extent(a.part, (size_t)groups * a.cols * 4, "ws.part");
  ++g_launches;
  return hipSuccess;
}
static void arranged_extents(const Mx4Arrange& r, int cols) {
  extent(r.scale, (size_t)r.rows * mx4_scale_bytes(cols), "scales to arrange");
  CHECK(r.pitch >= r.rows, "pitch %lld of %lld rows", (long long)r.pitch, (long long)r.rows);
  extent(r.out, mx4_arranged_bytes(r.pitch, cols), "arranged scales");
}
hipError_t launch_quantize_mx4(const void* in, int is_bf16, int64_t rows, int cols, uint8_t* q, uint8_t* scale,
                               uint8_t* arranged, int64_t pitch, const Mx4Arrange* also, hipStream_t) {
  extent(in, (size_t)rows * cols * (is_bf16 ? 2 : 4), "in");
  extent(q, (size_t)rows * mx4_code_bytes(cols), "q");
  CHECK((scale == nullptr) != (arranged == nullptr), "one place for the scales");
  if (scale) extent(scale, (size_t)rows * mx4_scale_bytes(cols), "scale");
  if (arranged) {
    CHECK(pitch >= rows, "pitch below the rows");
    extent(arranged, mx4_arranged_bytes(pitch, cols), "arranged");
  }
  if (also) arranged_extents(*also, cols);
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_mx4_arrange(const Mx4Arrange& a, const Mx4Arrange& b, int cols, hipStream_t) {
  arranged_extents(a, cols);
  arranged_extents(b, cols);
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_dequantize_mx4(const uint8_t* q, const uint8_t* scale, int64_t rows, int cols, int out_bf16,
                                 void* out, hipStream_t) {
  extent(q, (size_t)rows * mx4_code_bytes(cols), "q");
  extent(scale, (size_t)rows * mx4_scale_bytes(cols), "scale");
  extent(out, (size_t)rows * cols * (out_bf16 ? 2 : 4), "out");
  ++g_launches;
  return hipSuccess;
}
static int g_plans[4];
hipError_t launch_mx4_product(Mx4Plan plan, const Mx4ProductArgs& a, hipStream_t) {
  ++g_plans[plan];
  extent(a.w_q, (size_t)a.units * mx4_code_bytes(a.cols), "w_q");
  extent(a.y, (size_t)a.n * a.units * (a.y_bf16 ? 2 : 4), "y");
  if (plan == MX4_FUSED) {
    extent(a.x, (size_t)a.n * a.cols * (a.x_bf16 ? 2 : 4), "x");
    // the kernel holds a tile's rows of x in this many blocks of shared memory
    CHECK((a.n < 32 ? a.n : 32) * ((a.cols + 255) / 256) * 8 <= kMx4FusedBlocks, "x does not fit");
  } else {
    extent(a.x_q, (size_t)a.n * mx4_code_bytes(a.cols), "x_q");
  }
  if (mx4_tiled(plan)) {
    const int tile = plan == MX4_BIG ? kMx4BigTile : kMx4MidTile;
    CHECK(a.units >= tile && (a.n >= tile || (plan == MX4_MID && a.cols > 256)), "a tile larger than the operands");
    extent(a.x_arr, mx4_arranged_bytes(mx4_arranged_rows(a.n), a.cols), "arranged x scales");
    extent(a.w_arr, mx4_arranged_bytes(a.units, a.cols), "arranged w scales");
  } else {
    extent(a.w_scale, (size_t)a.units * mx4_scale_bytes(a.cols), "w_scale");
    if (plan == MX4_DIRECT) extent(a.x_scale, (size_t)a.n * mx4_scale_bytes(a.cols), "x_scale");
  }
  ++g_launches;
  return hipSuccess;
}

}  // namespace twell

namespace {

size_t esz(twell_dtype t) { return t == TWELL_BF16 ? 2 : 4; }

void norm_case(int64_t rows, int cols, twell_dtype rt, twell_dtype dt, twell_dtype ot) {
  g_where = "norm " + std::to_string(rows) + "x" + std::to_string(cols);
  const size_t n = (size_t)rows * cols;
  void *r = alloc(n * esz(rt), "r"), *d = alloc(n * esz(dt), "delta"), *w = alloc(cols * esz(ot), "w");
  void *ro = alloc(n * esz(rt), "r_out"), *o = alloc(n * esz(ot), "out");
  uint8_t* q = (uint8_t*)alloc(n, "q");
  float *qs = (float*)alloc(rows * 4, "q_scale"), *rs = (float*)alloc(rows * 4, "rstd");
  auto fwd = [&](void* delta, void* out_r, void* out, uint8_t* codes, float* rstd) {
    return twell_add_rms_norm(rows, cols, rt, r, dt, delta, ot, w, 1e-6f, out_r, ot, out, codes, codes ? qs : nullptr,
                              rstd, nullptr);
  };
  CHECK(fwd(d, ro, o, q, rs) == TWELL_OK, "%s", twell_last_error());
  CHECK(fwd(d, r, o, nullptr, nullptr) == TWELL_OK, "in place: %s", twell_last_error());
  CHECK(fwd(nullptr, nullptr, nullptr, q, nullptr) == TWELL_OK, "codes alone: %s", twell_last_error());
  if (rows > 0) CHECK(fwd(d, nullptr, nullptr, nullptr, nullptr) == TWELL_ERR_INVALID_ARG, "no output accepted");
  size_t need = 1;
  CHECK(twell_add_rms_norm_bwd_ws(rows, cols, &need) == TWELL_OK, "%s", twell_last_error());
  void* ws = alloc(need, "bwd ws");
  void *dr = alloc(n * esz(rt), "dr"), *g = alloc(n * esz(ot), "d_out");
  float* dw = (float*)alloc(cols * 4, "dw");
  for (void* ds : {static_cast<void*>(nullptr), r})
    CHECK(twell_add_rms_norm_bwd(rows, cols, ot, g, rt, ds, ro, rs, ot, w, dr, dw, ws, need, nullptr) == TWELL_OK, "%s",
          twell_last_error());
  const int mark = g_launches;
  if (need > 0)
    CHECK(twell_add_rms_norm_bwd(rows, cols, ot, g, rt, nullptr, ro, rs, ot, w, dr, dw, ws, need - 1, nullptr) ==
              TWELL_ERR_WORKSPACE,
          "short workspace accepted");
  CHECK(g_launches == mark, "an invalid call reached a launch");
  free_all();
}

void mx4_case(int64_t n, int cols, int units, twell_dtype xt, twell_dtype yt) {
  g_where = "mx4 " + std::to_string(n) + "x" + std::to_string(cols) + "x" + std::to_string(units);
  size_t xqb, xsb, wqb, wsb;
  CHECK(twell_mx4_sizes(n, cols, &xqb, &xsb) == TWELL_OK && twell_mx4_sizes(units, cols, &wqb, &wsb) == TWELL_OK, "%s",
        twell_last_error());
  void *x = alloc((size_t)n * cols * esz(xt), "x"), *y = alloc((size_t)n * units * esz(yt), "y");
  uint8_t *xq = (uint8_t*)alloc(xqb, "xq"), *xs = (uint8_t*)alloc(xsb, "xs");
  uint8_t *wq = (uint8_t*)alloc(wqb, "wq"), *wsc = (uint8_t*)alloc(wsb, "ws");
  CHECK(twell_quantize_mx4(n, cols, xt, x, xq, xs, nullptr) == TWELL_OK, "%s", twell_last_error());
  CHECK(twell_dequantize_mx4(n, cols, xq, xs, xt, x, nullptr) == TWELL_OK, "%s", twell_last_error());
  size_t lin = 0, mat = 0;
  CHECK(twell_linear_mx4_ws(n, cols, units, &lin) == TWELL_OK, "%s", twell_last_error());
  CHECK(twell_matmul_mx4_ws(n, cols, units, &mat) == TWELL_OK, "%s", twell_last_error());
  void *wl = alloc(lin, "linear ws"), *wm = alloc(mat, "matmul ws");
  CHECK(twell_linear_mx4(n, cols, units, xt, x, wq, wsc, yt, y, wl, lin, nullptr) == TWELL_OK, "%s", twell_last_error());
  CHECK(twell_matmul_mx4(n, cols, units, xq, xs, wq, wsc, yt, y, wm, mat, nullptr) == TWELL_OK, "%s",
        twell_last_error());
  const int mark = g_launches;
  if (lin > 0)
    CHECK(twell_linear_mx4(n, cols, units, xt, x, wq, wsc, yt, y, wl, lin - 1, nullptr) == TWELL_ERR_WORKSPACE, "short");
  if (mat > 0)
    CHECK(twell_matmul_mx4(n, cols, units, xq, xs, wq, wsc, yt, y, wm, mat - 1, nullptr) == TWELL_ERR_WORKSPACE, "short");
  CHECK(g_launches == mark, "an invalid call reached a launch");
  free_all();
}

}  // namespace

int main() {
  for (int64_t rows : {0, 1, 3, 16, 17, 513, 3000})
    for (int cols : {1, 8, 95, 128, 129, 256, 512, 1000, 1024, 1999, 2048, 2050, 4096, 8192, 16384}) {
      if (rows * cols > 9000000) continue;
      norm_case(rows, cols, TWELL_BF16, TWELL_F32, TWELL_BF16);
      norm_case(rows, cols, TWELL_F32, TWELL_BF16, TWELL_F32);
    }
  for (int64_t n : {0, 1, 4, 5, 16, 17, 100, 127, 128, 255, 256, 1003, 4100})
    for (int cols : {1, 32, 127, 256, 257, 512, 1990, 4096})
      for (int units : {1, 16, 127, 128, 255, 256, 2048, 8100}) {
        if (n * units > 9000000 || n * cols > 9000000) continue;
        mx4_case(n, cols, units, TWELL_BF16, TWELL_F32);
        mx4_case(n, cols, units, TWELL_F32, TWELL_BF16);
      }
  mx4_case(5000, 300, 4000, TWELL_BF16, TWELL_BF16);
  mx4_case(5000, 100, 4000, TWELL_F32, TWELL_F32);
  g_where = "plans";
  for (int p = 0; p < 4; ++p) CHECK(twell::g_plans[p] > 0, "plan %d was not reached", p);

  g_where = "limits";
  size_t b = 0;
  CHECK(twell_mx4_sizes(1ll << 27, 512, &b, &b) == TWELL_OK, "%s", twell_last_error());
  CHECK(twell_mx4_sizes((1ll << 27) + 1, 512, &b, &b) == TWELL_ERR_UNSUPPORTED, "too many pieces accepted");
  CHECK(twell_linear_mx4_ws(1, 1 << 20, 1 << 17, &b) == TWELL_ERR_UNSUPPORTED, "too large a weight accepted");
  CHECK(twell_linear_mx4_ws(1 << 26, 64, 1024, &b) == TWELL_ERR_UNSUPPORTED, "too many tiles accepted");
  if (g_failures) {
    std::fprintf(stderr, "%d check(s) failed\n", g_failures);
    return 1;
  }
  std::printf("host check ok: %d launches checked\n", g_launches);
  return 0;
}
