// C ABI of the operators around the block: host-side validation, then kernel
// launches on the caller's stream. See include/twell.h for the contract of
// every call.
#include <string>

#include "../csrc/twell_host.h"
#include "../csrc/twell_internal.h"
#include "ops_kernels.h"

namespace {

twell_status fail(twell_status st, const char* why) { return twell::set_error(st, why); }

twell_status hip_status(hipError_t e, const char* where) {
  if (e == hipSuccess) return TWELL_OK;
  return twell::set_error(TWELL_ERR_HIP, (std::string(where) + ": " + hipGetErrorString(e)).c_str());
}

twell_status ok() {
  twell::set_error(TWELL_OK, "");
  return TWELL_OK;
}

bool bad_dtype(twell_dtype t) { return t != TWELL_BF16 && t != TWELL_F32; }
size_t size_of(twell_dtype t) { return t == TWELL_BF16 ? 2 : 4; }

#define OPS_CHECK_PTR(p, bytes, name)                                                            \
  do {                                                                                           \
    if (twell::bad_ptr((p), (bytes)))                                                            \
      return fail(TWELL_ERR_INVALID_ARG, name " is NULL or not 16-byte aligned");                \
  } while (0)
#define OPS_CHECK_OPT(p, bytes, name)                                                            \
  do {                                                                                           \
    if ((p) != nullptr) OPS_CHECK_PTR(p, bytes, name);                                           \
  } while (0)

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

}  // extern "C"
