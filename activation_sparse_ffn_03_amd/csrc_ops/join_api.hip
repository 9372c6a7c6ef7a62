// C ABI of the join of a block's output to the stream, its backward and
// dropout: host-side validation, then kernel launches on the caller's stream.
// See include/twell.h for the contract of every call.
#include <cmath>

#include "ops_check.h"
#include "ops_kernels.h"

using namespace twell::check;

namespace {

// The dropped share in 1/65536 and what is kept is multiplied with.
struct Drop {
  uint32_t drop;
  float scale;
};
twell_status check_drop(float p, const uint64_t* rng, Drop* out) {
  if (!(p >= 0.f && p <= 1.f)) return fail(TWELL_ERR_INVALID_ARG, "p must be from 0 to 1");
  out->drop = (uint32_t)std::lrint((double)p * 65536.0);
  out->scale = out->drop == 65536 ? 0.f : (float)(65536.0 / (65536.0 - out->drop));
  if (out->drop != 0) OPS_CHECK_PTR(rng, 16, "rng");
  return TWELL_OK;
}

twell_status check_shape(int64_t rows, int32_t cols) {
  if (rows < 0 || cols <= 0) return fail(TWELL_ERR_INVALID_ARG, "rows must be >= 0 and cols > 0");
  if (rows > 0x7FFFFFFFll) return fail(TWELL_ERR_UNSUPPORTED, "rows above 2^31 - 1");
  return TWELL_OK;
}

twell_status check_join_shape(int64_t rows, int32_t cols, bool gate, int64_t gate_rows) {
  const twell_status st = check_shape(rows, cols);
  if (st != TWELL_OK) return st;
  if (cols > twell::kNormMaxCols) return fail(TWELL_ERR_UNSUPPORTED, "cols above 16384");
  if (gate && (gate_rows < 1 || rows % gate_rows != 0))
    return fail(TWELL_ERR_INVALID_ARG, "gate_rows must be at least 1 and divide rows");
  if (gate && gate_rows > 0x7FFFFFFFll) return fail(TWELL_ERR_UNSUPPORTED, "gate_rows above 2^31 - 1");
  return TWELL_OK;
}

// Shape and options that both directions take.
twell_status check_join(int64_t rows, int32_t cols, const twell_join* j, Drop* drop) {
  if (j == nullptr) return fail(TWELL_ERR_INVALID_ARG, "join is NULL");
  twell_status st = check_join_shape(rows, cols, j->gate != nullptr, j->gate_rows);
  if (st != TWELL_OK) return st;
  if ((j->post_weight != nullptr && bad_dtype(j->post_weight_dtype)) || (j->gate != nullptr && bad_dtype(j->gate_dtype)))
    return fail(TWELL_ERR_INVALID_ARG, "dtypes must be bf16 or fp32");
  if (j->alpha - j->alpha != 0.f) return fail(TWELL_ERR_INVALID_ARG, "alpha must be finite");
  OPS_CHECK_OPT(j->post_weight, (size_t)cols * size_of(j->post_weight_dtype), "post_weight");
  OPS_CHECK_OPT(j->gate, (size_t)j->gate_rows * cols * size_of(j->gate_dtype), "gate");
  return check_drop(j->p, j->rng, drop);
}

}  // namespace

extern "C" {

twell_status twell_join_rms_norm(int64_t rows, int32_t cols, twell_dtype res_dtype, const void* residual,
                                 twell_dtype y_dtype, const void* y, twell_dtype weight_dtype, const void* weight,
                                 const twell_join* join, float eps, void* residual_out, twell_dtype out_dtype,
                                 void* out, uint8_t* q, float* q_scale, float* rstd, float* post_rstd, void* stream) {
  Drop drop;
  twell_status st = check_join(rows, cols, join, &drop);
  if (st != TWELL_OK) return st;
  if (bad_dtype(res_dtype) || bad_dtype(y_dtype) || bad_dtype(weight_dtype) || bad_dtype(out_dtype))
    return fail(TWELL_ERR_INVALID_ARG, "dtypes must be bf16 or fp32");
  if (!(eps > 0.f) || eps - eps != 0.f) return fail(TWELL_ERR_INVALID_ARG, "eps must be positive and finite");
  const size_t n = (size_t)rows * cols;
  OPS_CHECK_PTR(residual, n * size_of(res_dtype), "residual");
  OPS_CHECK_PTR(y, n * size_of(y_dtype), "y");
  OPS_CHECK_PTR(weight, (size_t)cols * size_of(weight_dtype), "weight");
  OPS_CHECK_OPT(residual_out, n * size_of(res_dtype), "residual_out");
  OPS_CHECK_OPT(out, n * size_of(out_dtype), "out");
  OPS_CHECK_OPT(q, n, "q");
  if (q != nullptr) OPS_CHECK_PTR(q_scale, (size_t)rows * 4, "q_scale");
  OPS_CHECK_OPT(rstd, (size_t)rows * 4, "rstd");
  OPS_CHECK_OPT(post_rstd, (size_t)rows * 4, "post_rstd");
  if (post_rstd != nullptr && join->post_weight == nullptr)
    return fail(TWELL_ERR_INVALID_ARG, "post_rstd is given without post_weight");
  if (residual_out == nullptr && out == nullptr && q == nullptr && rstd == nullptr && post_rstd == nullptr && rows > 0)
    return fail(TWELL_ERR_INVALID_ARG, "no output is given");
  if (rows == 0) return ok();
  st = check_apart({{residual_out, n * size_of(res_dtype)}, {out, n * size_of(out_dtype)}, {q, n},
                    {q != nullptr ? q_scale : nullptr, (size_t)rows * 4}, {rstd, (size_t)rows * 4}, {post_rstd, (size_t)rows * 4}},
                   {{residual == residual_out ? nullptr : residual, n * size_of(res_dtype)}, {y, n * size_of(y_dtype)},
                    {weight, (size_t)cols * size_of(weight_dtype)},
                    {join->post_weight, (size_t)cols * size_of(join->post_weight_dtype)},
                    {join->gate, (size_t)join->gate_rows * cols * size_of(join->gate_dtype)}, {drop.drop != 0 ? join->rng : nullptr, 16}});
  if (st != TWELL_OK) return st;
  twell::JoinArgs a{};
  a.rows = rows;
  a.cols = cols;
  a.res_bf16 = res_dtype == TWELL_BF16;
  a.y_bf16 = y_dtype == TWELL_BF16;
  a.w_bf16 = weight_dtype == TWELL_BF16;
  a.post_bf16 = join->post_weight_dtype == TWELL_BF16;
  a.gate_bf16 = join->gate_dtype == TWELL_BF16;
  a.out_bf16 = out_dtype == TWELL_BF16;
  a.residual = residual;
  a.y = y;
  a.w = weight;
  a.post_w = join->post_weight;
  a.gate = join->gate;
  a.per_gate = join->gate != nullptr ? (uint32_t)(rows / join->gate_rows) : 1u;
  a.alpha = join->alpha;
  a.eps = eps;
  a.rng = join->rng;
  a.site = join->site;
  a.drop = drop.drop;
  a.drop_scale = drop.scale;
  a.residual_out = residual_out;
  a.out = out;
  a.q = q;
  a.q_scale = q_scale;
  a.rstd = rstd;
  a.post_rstd = post_rstd;
  ok();
  return hip_status(twell::launch_join_rms_norm(a, (hipStream_t)stream), "twell_join_rms_norm");
}

twell_status twell_join_rms_norm_bwd_ws(int64_t rows, int32_t cols, int32_t post, int64_t gate_rows, size_t* ws_bytes) {
  if (gate_rows < 0) return fail(TWELL_ERR_INVALID_ARG, "gate_rows must be >= 0");
  const twell_status st = check_join_shape(rows, cols, gate_rows > 0, gate_rows);
  if (st != TWELL_OK) return st;
  if (ws_bytes == nullptr) return fail(TWELL_ERR_INVALID_ARG, "ws_bytes is NULL");
  *ws_bytes = 4 * twell::join_bwd_ws_floats(rows, cols, gate_rows > 0 ? (uint32_t)gate_rows : 1u, post != 0, gate_rows > 0);
  return ok();
}

twell_status twell_join_rms_norm_bwd(int64_t rows, int32_t cols, twell_dtype d_out_dtype, const void* d_out,
                                     twell_dtype res_dtype, const void* d_residual, const void* residual,
                                     const float* rstd, twell_dtype y_dtype, const void* y, const float* post_rstd,
                                     twell_dtype weight_dtype, const void* weight, const twell_join* join, void* dr,
                                     void* dy, float* dw, float* dpost, float* dgate, void* ws, size_t ws_bytes,
                                     void* stream) {
  Drop drop;
  twell_status st = check_join(rows, cols, join, &drop);
  if (st != TWELL_OK) return st;
  if (bad_dtype(d_out_dtype) || bad_dtype(res_dtype) || bad_dtype(y_dtype) || bad_dtype(weight_dtype))
    return fail(TWELL_ERR_INVALID_ARG, "dtypes must be bf16 or fp32");
  const size_t n = (size_t)rows * cols;
  const bool post = join->post_weight != nullptr, gate = join->gate != nullptr;
  const uint32_t gates = gate ? (uint32_t)join->gate_rows : 1u;
  OPS_CHECK_PTR(d_out, n * size_of(d_out_dtype), "d_out");
  OPS_CHECK_OPT(d_residual, n * size_of(res_dtype), "d_residual");
  OPS_CHECK_PTR(residual, n * size_of(res_dtype), "residual");
  OPS_CHECK_PTR(rstd, (size_t)rows * 4, "rstd");
  OPS_CHECK_PTR(y, n * size_of(y_dtype), "y");
  if (post) OPS_CHECK_PTR(post_rstd, (size_t)rows * 4, "post_rstd");
  OPS_CHECK_PTR(weight, (size_t)cols * size_of(weight_dtype), "weight");
  OPS_CHECK_PTR(dr, n * size_of(res_dtype), "dr");
  OPS_CHECK_PTR(dy, n * size_of(y_dtype), "dy");
  OPS_CHECK_PTR(dw, (size_t)cols * 4, "dw");
  if (post) OPS_CHECK_PTR(dpost, (size_t)cols * 4, "dpost");
  if (gate) OPS_CHECK_PTR(dgate, (size_t)gates * cols * 4, "dgate");
  const size_t need = 4 * twell::join_bwd_ws_floats(rows, cols, gates, post, gate);
  if ((st = check_ws(ws, ws_bytes, need, "workspace smaller than twell_join_rms_norm_bwd_ws says")) != TWELL_OK) return st;
  st = check_apart({{dr, n * size_of(res_dtype)}, {dy, n * size_of(y_dtype)}, {dw, (size_t)cols * 4},
                    {post ? dpost : nullptr, (size_t)cols * 4}, {gate ? dgate : nullptr, (size_t)gates * cols * 4}, {ws, need}},
                   {{d_out, n * size_of(d_out_dtype)}, {d_residual, n * size_of(res_dtype)}, {residual, n * size_of(res_dtype)},
                    {rstd, (size_t)rows * 4}, {y, n * size_of(y_dtype)}, {post ? post_rstd : nullptr, (size_t)rows * 4},
                    {weight, (size_t)cols * size_of(weight_dtype)},
                    {join->post_weight, (size_t)cols * size_of(join->post_weight_dtype)},
                    {join->gate, (size_t)gates * cols * size_of(join->gate_dtype)}, {drop.drop != 0 ? join->rng : nullptr, 16}});
  if (st != TWELL_OK) return st;
  twell::JoinBwdArgs a{};
  a.rows = rows;
  a.cols = cols;
  a.g_bf16 = d_out_dtype == TWELL_BF16;
  a.res_bf16 = res_dtype == TWELL_BF16;
  a.y_bf16 = y_dtype == TWELL_BF16;
  a.w_bf16 = weight_dtype == TWELL_BF16;
  a.post_bf16 = join->post_weight_dtype == TWELL_BF16;
  a.gate_bf16 = join->gate_dtype == TWELL_BF16;
  a.d_out = d_out;
  a.d_residual = d_residual;
  a.residual = residual;
  a.rstd = rstd;
  a.y = y;
  a.post_rstd = post_rstd;
  a.w = weight;
  a.post_w = join->post_weight;
  a.gate = join->gate;
  a.gates = gates;
  a.alpha = join->alpha;
  a.rng = join->rng;
  a.site = join->site;
  a.drop = drop.drop;
  a.drop_scale = drop.scale;
  a.dr = dr;
  a.dy = dy;
  a.dw = dw;
  a.dpost = dpost;
  a.dgate = dgate;
  a.part = static_cast<float*>(ws);
  ok();
  return hip_status(twell::launch_join_rms_norm_bwd(a, (hipStream_t)stream), "twell_join_rms_norm_bwd");
}

twell_status twell_dropout(int64_t rows, int32_t cols, twell_dtype dtype, const void* x, float p, const uint64_t* rng,
                           uint32_t site, void* out, void* stream) {
  twell_status st = check_shape(rows, cols);
  if (st != TWELL_OK) return st;
  if (cols > twell::kDropoutMaxCols) return fail(TWELL_ERR_UNSUPPORTED, "cols above 2^30");
  if (bad_dtype(dtype)) return fail(TWELL_ERR_INVALID_ARG, "dtypes must be bf16 or fp32");
  Drop drop;
  if ((st = check_drop(p, rng, &drop)) != TWELL_OK) return st;
  OPS_CHECK_PTR(rng, 16, "rng");
  const size_t bytes = (size_t)rows * cols * size_of(dtype);
  OPS_CHECK_PTR(x, bytes, "x");
  OPS_CHECK_PTR(out, bytes, "out");
  if (rows == 0) return ok();
  st = check_apart({{out, bytes}}, {{x == out ? nullptr : x, bytes}, {rng, 16}});
  if (st != TWELL_OK) return st;
  twell::DropoutArgs a{};
  a.rows = rows;
  a.cols = cols;
  a.bf16 = dtype == TWELL_BF16;
  a.x = x;
  a.out = out;
  a.rng = rng;
  a.site = site;
  a.drop = drop.drop;
  a.drop_scale = drop.scale;
  ok();
  return hip_status(twell::launch_dropout(a, (hipStream_t)stream), "twell_dropout");
}

}  // extern "C"
