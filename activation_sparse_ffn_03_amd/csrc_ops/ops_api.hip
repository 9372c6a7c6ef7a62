// C ABI of the operators around the block: host-side validation, then kernel
// launches on the caller's stream. See include/twell.h for the contract of
// every call.
#include "ops_check.h"
#include "ops_kernels.h"

using namespace twell::check;

namespace {

twell_status check_norm_shape(int64_t rows, int32_t cols) {
  if (rows < 0 || cols <= 0) return fail(TWELL_ERR_INVALID_ARG, "rows must be >= 0 and cols > 0");
  if (rows > 0x7FFFFFFFll) return fail(TWELL_ERR_UNSUPPORTED, "rows above 2^31 - 1");
  if (cols > twell::kNormMaxCols) return fail(TWELL_ERR_UNSUPPORTED, "cols above 16384");
  return TWELL_OK;
}

size_t norm_bwd_ws_bytes(int64_t rows, int32_t cols) {
  const int g = twell::norm_bwd_groups(rows, cols);
  return g == 1 ? 0 : (size_t)g * cols * 4;
}

twell_status check_mx4_shape(int64_t rows, int32_t cols) {
  if (rows < 0 || cols <= 0) return fail(TWELL_ERR_INVALID_ARG, "rows must be >= 0 and cols > 0");
  if (rows > 0x7FFFFFFFll) return fail(TWELL_ERR_UNSUPPORTED, "rows above 2^31 - 1");
  if (cols > twell::kMx4MaxCols) return fail(TWELL_ERR_UNSUPPORTED, "cols above 2^20");
  // one launch: 16 threads a piece of 512 columns, less than 2^32 threads
  if (rows * ((cols + 511) / 512) > (1ll << 27)) return fail(TWELL_ERR_UNSUPPORTED, "more than 2^27 pieces of 512 columns");
  return TWELL_OK;
}

size_t mx4_codes(int64_t rows, int32_t cols) { return (size_t)rows * twell::mx4_code_bytes(cols); }
size_t mx4_scales(int64_t rows, int32_t cols) { return (size_t)rows * twell::mx4_scale_bytes(cols); }

twell_status check_mx4_dims(int64_t n, int32_t cols, int32_t units) {
  twell_status st = check_mx4_shape(n, cols);
  if (st != TWELL_OK) return st;
  if (units <= 0) return fail(TWELL_ERR_INVALID_ARG, "units must be > 0");
  if (units > (1 << 24)) return fail(TWELL_ERR_UNSUPPORTED, "units above 2^24");
  if ((st = check_mx4_shape(units, cols)) != TWELL_OK) return st;
  // one launch: a workgroup of 256 threads a tile of 64 x 64, less than 2^32 threads
  if (((n + 63) / 64) * ((units + 63) / 64) >= (1ll << 24))
    return fail(TWELL_ERR_UNSUPPORTED, "2^24 output tiles of 64 x 64 or more");
  return TWELL_OK;
}

// Shape, weights and output shared by the products.
twell_status check_mx4_product(int64_t n, int32_t cols, int32_t units, const uint8_t* w_q, const uint8_t* w_scale,
                               twell_dtype y_dtype, void* y, twell::Mx4ProductArgs* a) {
  const twell_status st = check_mx4_dims(n, cols, units);
  if (st != TWELL_OK) return st;
  if (bad_dtype(y_dtype)) return fail(TWELL_ERR_INVALID_ARG, "dtypes must be bf16 or fp32");
  OPS_CHECK_PTR(w_q, mx4_codes(units, cols), "w_q");
  OPS_CHECK_PTR(w_scale, mx4_scales(units, cols), "w_scale");
  OPS_CHECK_PTR(y, (size_t)n * units * size_of(y_dtype), "y");
  a->n = n;
  a->cols = cols;
  a->units = units;
  a->w_q = w_q;
  a->w_scale = w_scale;
  a->y = y;
  a->y_bf16 = y_dtype == TWELL_BF16;
  return TWELL_OK;
}

// Workspaces: the arranged scales of w and x (tiled plans), and in front of
// them, for the product that quantises x, its MX4 rows (their scales only where
// they are not arranged at once).
struct ProductLayout {
  size_t x_q, x_scale, w_arr, x_arr, total;
};
ProductLayout product_layout(twell::Mx4Plan plan, int64_t n, int32_t cols, int32_t units, bool quantise) {
  const bool tiled = twell::mx4_tiled(plan);
  ProductLayout L{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t off = at;
    at += (bytes + 15) / 16 * 16;
    return off;
  };
  const bool rows = quantise && plan != twell::MX4_FUSED;
  L.x_q = take(rows ? mx4_codes(n, cols) : 0);
  L.x_scale = take(rows && !tiled ? mx4_scales(n, cols) : 0);
  L.w_arr = take(tiled ? twell::mx4_arranged_bytes(units, cols) : 0);
  L.x_arr = take(tiled ? twell::mx4_arranged_bytes(twell::mx4_arranged_rows(n), cols) : 0);
  L.total = at;
  return L;
}

twell_status product_ws(int64_t n, int32_t cols, int32_t units, bool quantise, size_t* ws_bytes) {
  const twell_status st = check_mx4_dims(n, cols, units);
  if (st != TWELL_OK) return st;
  if (ws_bytes == nullptr) return fail(TWELL_ERR_INVALID_ARG, "ws_bytes is NULL");
  *ws_bytes = n == 0 ? 0 : product_layout(twell::mx4_plan(n, cols, units, !quantise), n, cols, units, quantise).total;
  twell::set_error(TWELL_OK, "");
  return TWELL_OK;
}

}  // namespace

extern "C" {

twell_status twell_add_rms_norm(int64_t rows, int32_t cols, twell_dtype res_dtype, const void* residual,
                                twell_dtype delta_dtype, const void* delta, twell_dtype weight_dtype,
                                const void* weight, float eps, void* residual_out, twell_dtype out_dtype, void* out,
                                uint8_t* q, float* q_scale, float* rstd, void* stream) {
  const twell_status st = check_norm_shape(rows, cols);
  if (st != TWELL_OK) return st;
  if (bad_dtype(res_dtype) || bad_dtype(weight_dtype) || bad_dtype(out_dtype) ||
      (delta != nullptr && bad_dtype(delta_dtype)))
    return fail(TWELL_ERR_INVALID_ARG, "dtypes must be bf16 or fp32");
  if (!(eps > 0.f) || eps - eps != 0.f) return fail(TWELL_ERR_INVALID_ARG, "eps must be positive and finite");
  const size_t n = (size_t)rows * cols;
  OPS_CHECK_PTR(residual, n * size_of(res_dtype), "residual");
  OPS_CHECK_OPT(delta, n * size_of(delta_dtype), "delta");
  OPS_CHECK_PTR(weight, (size_t)cols * size_of(weight_dtype), "weight");
  OPS_CHECK_OPT(residual_out, n * size_of(res_dtype), "residual_out");
  OPS_CHECK_OPT(out, n * size_of(out_dtype), "out");
  OPS_CHECK_OPT(q, n, "q");
  if (q != nullptr) OPS_CHECK_PTR(q_scale, (size_t)rows * 4, "q_scale");
  OPS_CHECK_OPT(rstd, (size_t)rows * 4, "rstd");
  if (residual_out == nullptr && out == nullptr && q == nullptr && rstd == nullptr && rows > 0)
    return fail(TWELL_ERR_INVALID_ARG, "no output is given");
  if (rows == 0) return ok();
  twell::NormArgs a{};
  a.rows = rows;
  a.cols = cols;
  a.res_bf16 = res_dtype == TWELL_BF16;
  a.delta_bf16 = delta_dtype == TWELL_BF16;
  a.w_bf16 = weight_dtype == TWELL_BF16;
  a.out_bf16 = out_dtype == TWELL_BF16;
  a.residual = residual;
  a.delta = delta;
  a.w = weight;
  a.eps = eps;
  a.residual_out = residual_out;
  a.out = out;
  a.q = q;
  a.q_scale = q_scale;
  a.rstd = rstd;
  ok();
  return hip_status(twell::launch_add_rms_norm(a, (hipStream_t)stream), "twell_add_rms_norm");
}

twell_status twell_add_rms_norm_bwd_ws(int64_t rows, int32_t cols, size_t* ws_bytes) {
  const twell_status st = check_norm_shape(rows, cols);
  if (st != TWELL_OK) return st;
  if (ws_bytes == nullptr) return fail(TWELL_ERR_INVALID_ARG, "ws_bytes is NULL");
  *ws_bytes = norm_bwd_ws_bytes(rows, cols);
  return ok();
}

twell_status twell_add_rms_norm_bwd(int64_t rows, int32_t cols, twell_dtype d_out_dtype, const void* d_out,
                                    twell_dtype res_dtype, const void* d_residual, const void* residual,
                                    const float* rstd, twell_dtype weight_dtype, const void* weight, void* dr,
                                    float* dw, void* ws, size_t ws_bytes, void* stream) {
  const twell_status st = check_norm_shape(rows, cols);
  if (st != TWELL_OK) return st;
  if (bad_dtype(d_out_dtype) || bad_dtype(res_dtype) || bad_dtype(weight_dtype))
    return fail(TWELL_ERR_INVALID_ARG, "dtypes must be bf16 or fp32");
  const size_t n = (size_t)rows * cols;
  OPS_CHECK_PTR(d_out, n * size_of(d_out_dtype), "d_out");
  OPS_CHECK_OPT(d_residual, n * size_of(res_dtype), "d_residual");
  OPS_CHECK_PTR(residual, n * size_of(res_dtype), "residual");
  OPS_CHECK_PTR(rstd, (size_t)rows * 4, "rstd");
  OPS_CHECK_PTR(weight, (size_t)cols * size_of(weight_dtype), "weight");
  OPS_CHECK_PTR(dr, n * size_of(res_dtype), "dr");
  OPS_CHECK_PTR(dw, (size_t)cols * 4, "dw");
  const size_t need = norm_bwd_ws_bytes(rows, cols);
  if (ws_bytes < need) return fail(TWELL_ERR_WORKSPACE, "workspace smaller than twell_add_rms_norm_bwd_ws says");
  if (twell::bad_ptr(ws, need)) return fail(TWELL_ERR_WORKSPACE, "workspace is NULL or not 16-byte aligned");
  twell::NormBwdArgs a{};
  a.rows = rows;
  a.cols = cols;
  a.g_bf16 = d_out_dtype == TWELL_BF16;
  a.res_bf16 = res_dtype == TWELL_BF16;
  a.w_bf16 = weight_dtype == TWELL_BF16;
  a.d_out = d_out;
  a.d_residual = d_residual;
  a.residual = residual;
  a.rstd = rstd;
  a.w = weight;
  a.dr = dr;
  a.dw = dw;
  a.part = static_cast<float*>(ws);
  ok();
  return hip_status(twell::launch_add_rms_norm_bwd(a, (hipStream_t)stream), "twell_add_rms_norm_bwd");
}

twell_status twell_mx4_sizes(int64_t rows, int32_t cols, size_t* q_bytes, size_t* scale_bytes) {
  const twell_status st = check_mx4_shape(rows, cols);
  if (st != TWELL_OK) return st;
  if (q_bytes == nullptr || scale_bytes == nullptr) return fail(TWELL_ERR_INVALID_ARG, "q_bytes or scale_bytes is NULL");
  *q_bytes = mx4_codes(rows, cols);
  *scale_bytes = mx4_scales(rows, cols);
  return ok();
}

twell_status twell_quantize_mx4(int64_t rows, int32_t cols, twell_dtype dtype, const void* in, uint8_t* q,
                                uint8_t* scale, void* stream) {
  const twell_status st = check_mx4_shape(rows, cols);
  if (st != TWELL_OK) return st;
  if (bad_dtype(dtype)) return fail(TWELL_ERR_INVALID_ARG, "dtypes must be bf16 or fp32");
  OPS_CHECK_PTR(in, (size_t)rows * cols * size_of(dtype), "in");
  OPS_CHECK_PTR(q, mx4_codes(rows, cols), "q");
  OPS_CHECK_PTR(scale, mx4_scales(rows, cols), "scale");
  ok();
  if (rows == 0) return TWELL_OK;
  return hip_status(twell::launch_quantize_mx4(in, dtype == TWELL_BF16, rows, cols, q, scale, nullptr, 0, nullptr,
                                               (hipStream_t)stream),
                    "twell_quantize_mx4");
}

twell_status twell_dequantize_mx4(int64_t rows, int32_t cols, const uint8_t* q, const uint8_t* scale,
                                  twell_dtype dtype, void* out, void* stream) {
  const twell_status st = check_mx4_shape(rows, cols);
  if (st != TWELL_OK) return st;
  if (bad_dtype(dtype)) return fail(TWELL_ERR_INVALID_ARG, "dtypes must be bf16 or fp32");
  OPS_CHECK_PTR(q, mx4_codes(rows, cols), "q");
  OPS_CHECK_PTR(scale, mx4_scales(rows, cols), "scale");
  OPS_CHECK_PTR(out, (size_t)rows * cols * size_of(dtype), "out");
  ok();
  if (rows == 0) return TWELL_OK;
  return hip_status(twell::launch_dequantize_mx4(q, scale, rows, cols, dtype == TWELL_BF16, out, (hipStream_t)stream),
                    "twell_dequantize_mx4");
}

twell_status twell_matmul_mx4_ws(int64_t n, int32_t cols, int32_t units, size_t* ws_bytes) {
  return product_ws(n, cols, units, false, ws_bytes);
}

twell_status twell_matmul_mx4(int64_t n, int32_t cols, int32_t units, const uint8_t* x_q, const uint8_t* x_scale,
                              const uint8_t* w_q, const uint8_t* w_scale, twell_dtype y_dtype, void* y, void* ws,
                              size_t ws_bytes, void* stream) {
  twell::Mx4ProductArgs a{};
  twell_status st = check_mx4_product(n, cols, units, w_q, w_scale, y_dtype, y, &a);
  if (st != TWELL_OK) return st;
  OPS_CHECK_PTR(x_q, mx4_codes(n, cols), "x_q");
  OPS_CHECK_PTR(x_scale, mx4_scales(n, cols), "x_scale");
  if (n == 0) return ok();
  const twell::Mx4Plan plan = twell::mx4_plan(n, cols, units, true);
  const ProductLayout L = product_layout(plan, n, cols, units, false);
  if ((st = check_ws(ws, ws_bytes, L.total, "workspace smaller than twell_matmul_mx4_ws says")) != TWELL_OK) return st;
  ok();
  a.x_q = x_q;
  a.x_scale = x_scale;
  if (twell::mx4_tiled(plan)) {
    uint8_t* base = static_cast<uint8_t*>(ws);
    const twell::Mx4Arrange w{w_scale, base + L.w_arr, units, units};
    const twell::Mx4Arrange x{x_scale, base + L.x_arr, n, twell::mx4_arranged_rows(n)};
    const hipError_t e = twell::launch_mx4_arrange(w, x, cols, (hipStream_t)stream);
    if (e != hipSuccess) return hip_status(e, "twell_matmul_mx4");
    a.w_arr = w.out;
    a.x_arr = x.out;
  }
  return hip_status(twell::launch_mx4_product(plan, a, (hipStream_t)stream), "twell_matmul_mx4");
}

twell_status twell_linear_mx4_ws(int64_t n, int32_t cols, int32_t units, size_t* ws_bytes) {
  return product_ws(n, cols, units, true, ws_bytes);
}

twell_status twell_linear_mx4(int64_t n, int32_t cols, int32_t units, twell_dtype x_dtype, const void* x,
                              const uint8_t* w_q, const uint8_t* w_scale, twell_dtype y_dtype, void* y, void* ws,
                              size_t ws_bytes, void* stream) {
  twell::Mx4ProductArgs a{};
  twell_status st = check_mx4_product(n, cols, units, w_q, w_scale, y_dtype, y, &a);
  if (st != TWELL_OK) return st;
  if (bad_dtype(x_dtype)) return fail(TWELL_ERR_INVALID_ARG, "dtypes must be bf16 or fp32");
  OPS_CHECK_PTR(x, (size_t)n * cols * size_of(x_dtype), "x");
  if (n == 0) return ok();
  const twell::Mx4Plan plan = twell::mx4_plan(n, cols, units, false);
  const ProductLayout L = product_layout(plan, n, cols, units, true);
  if ((st = check_ws(ws, ws_bytes, L.total, "workspace smaller than twell_linear_mx4_ws says")) != TWELL_OK) return st;
  ok();
  const int x_bf16 = x_dtype == TWELL_BF16;
  if (plan == twell::MX4_FUSED) {
    a.x = x;
    a.x_bf16 = x_bf16;
  } else {
    uint8_t* base = static_cast<uint8_t*>(ws);
    const bool tiled = twell::mx4_tiled(plan);
    uint8_t* const x_arr = tiled ? base + L.x_arr : nullptr;
    const twell::Mx4Arrange w{w_scale, base + L.w_arr, units, units};
    const hipError_t e =
        twell::launch_quantize_mx4(x, x_bf16, n, cols, base + L.x_q, tiled ? nullptr : base + L.x_scale, x_arr,
                                   twell::mx4_arranged_rows(n), tiled ? &w : nullptr, (hipStream_t)stream);
    if (e != hipSuccess) return hip_status(e, "twell_linear_mx4");
    a.x_q = base + L.x_q;
    a.x_scale = base + L.x_scale;
    a.w_arr = w.out;
    a.x_arr = x_arr;
  }
  return hip_status(twell::launch_mx4_product(plan, a, (hipStream_t)stream), "twell_linear_mx4");
}

}  // extern "C"
