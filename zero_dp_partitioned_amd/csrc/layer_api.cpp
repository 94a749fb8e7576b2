// Host side of a layer's operators (include/zero_dp.h): argument checks and launches.
#include <float.h>
#include <hip/hip_runtime.h>
#include <math.h>

#include <initializer_list>

#include "api_common.h"
#include "layer_internal.h"

using namespace zdp;

namespace {

bool valid_dt(int32_t dt) { return dt == ZERO_DT_F32 || dt == ZERO_DT_F16 || dt == ZERO_DT_BF16; }
int64_t dt_bytes(int32_t dt) { return dt == ZERO_DT_F32 ? 4 : 2; }

// rows x cols values of dt, ld from row to row, of which `p` may be null if there are none.
int check_rows(const char* what, const void* p, int32_t dt, int64_t rows, int64_t cols, int64_t ld) {
  if (ld < cols)
    return fail(ZERO_ERR_INVALID_ARG, "%s: %lld elements from row to row, fewer than a row's %lld", what, (long long)ld,
                (long long)cols);
  int64_t t;
  if (__builtin_mul_overflow(rows, ld, &t) || __builtin_mul_overflow(t, dt_bytes(dt), &t))
    return fail(ZERO_ERR_INVALID_ARG, "%s: extent overflows int64", what);
  if (rows == 0 || cols == 0) return ZERO_OK;
  if (!p) return fail(ZERO_ERR_INVALID_ARG, "%s is NULL", what);
  if (!aligned(p, static_cast<uintptr_t>(dt_bytes(dt))))
    return fail(ZERO_ERR_ALIGNMENT, "%s is not aligned to its elements", what);
  return ZERO_OK;
}

int check_dt(const char* what, int32_t dt) {
  return valid_dt(dt) ? ZERO_OK : fail(ZERO_ERR_INVALID_ARG, "%s: dtype %d is not f32/f16/bf16", what, dt);
}

int check_norm(int32_t dt, int32_t w_dt, int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0) return fail(ZERO_ERR_INVALID_ARG, "rows or cols < 0");
  if (int rc = check_dt("x", dt)) return rc;
  if (w_dt != dt && w_dt != ZERO_DT_F32)
    return fail(ZERO_ERR_INVALID_ARG, "weight: dtype %d is neither x's %d nor f32", w_dt, dt);
  if (cols > kMaxNormCols) return fail(ZERO_ERR_UNSUPPORTED, "%lld columns, more than %d", (long long)cols, kMaxNormCols);
  return ZERO_OK;
}

int check_vector(const char* what, const void* p, int32_t dt, bool wanted) {
  if (!p && wanted) return fail(ZERO_ERR_INVALID_ARG, "%s is NULL", what);
  if (!aligned(p, static_cast<uintptr_t>(dt_bytes(dt))))
    return fail(ZERO_ERR_ALIGNMENT, "%s is not aligned to its elements", what);
  return ZERO_OK;
}

int check_gated(int32_t dt, int64_t m, int64_t d, int64_t f, int32_t act) {
  if (m < 0 || d < 0 || f < 0) return fail(ZERO_ERR_INVALID_ARG, "m, d or f < 0");
  if (dt != ZERO_DT_F16 && dt != ZERO_DT_BF16) return fail(ZERO_ERR_INVALID_ARG, "x: dtype %d is not f16/bf16", dt);
  if (act < ZERO_ACT_SILU || act > ZERO_ACT_SIGMOID) return fail(ZERO_ERR_INVALID_ARG, "act = %d", act);
  if (m > INT32_MAX || d > INT32_MAX || f > INT32_MAX)
    return fail(ZERO_ERR_UNSUPPORTED, "more than 2^31 - 1 rows or columns");
  return ZERO_OK;
}

int check_strides(std::initializer_list<int64_t> lds) {
  for (int64_t ld : lds)
    if (ld > kMaxRowStride)
      return fail(ZERO_ERR_UNSUPPORTED, "rows more than %lld elements apart", (long long)kMaxRowStride);
  return ZERO_OK;
}

int launched(hipError_t e, const char* what) {
  if (e == hipErrorInvalidConfiguration) return fail(ZERO_ERR_UNSUPPORTED, "more output tiles than a launch holds");
  return e == hipSuccess ? ZERO_OK : hip_fail(e, what);
}

}  // namespace

extern "C" {

int zero_layer_norm(const void* x, int32_t dt, int64_t rows, int64_t cols, int64_t x_ld, const void* weight,
                    const void* bias, int32_t w_dt, double eps, void* y, int64_t y_ld, float* mean, float* rstd,
                    void* stream) {
  if (int rc = check_norm(dt, w_dt, rows, cols)) return rc;
  if (!(eps >= 0) || !(eps <= FLT_MAX)) return fail(ZERO_ERR_INVALID_ARG, "eps = %g", eps);
  // what the kernels add: not 0 for a smaller eps, which would make a row without spread NaN
  const float eps32 = eps > 0 && eps < FLT_TRUE_MIN ? FLT_TRUE_MIN : static_cast<float>(eps);
  if (int rc = check_rows("x", x, dt, rows, cols, x_ld)) return rc;
  if (int rc = check_rows("y", y, dt, rows, cols, y_ld)) return rc;
  if ((mean == nullptr) != (rstd == nullptr)) return fail(ZERO_ERR_INVALID_ARG, "mean and rstd must be given together");
  if (rows == 0 || cols == 0) return ZERO_OK;
  if (int rc = check_vector("weight", weight, w_dt, true)) return rc;
  if (int rc = check_vector("bias", bias, w_dt, false)) return rc;
  if (int rc = check_vector("mean", mean, ZERO_DT_F32, false)) return rc;
  if (int rc = check_vector("rstd", rstd, ZERO_DT_F32, false)) return rc;
  if (int rc = check_device()) return rc;
  NormArgs N;
  N.x = {x, x_ld};
  N.y = {y, y_ld};
  N.rows = rows;
  N.cols = static_cast<int32_t>(cols);
  N.weight = weight;
  N.bias = bias;
  N.w_dt = w_dt;
  N.eps = eps32;
  N.inv = 1.0f / static_cast<float>(cols);
  N.scale = ldexpf(1.0f, ilogbf(N.inv) - 1);  // (one power to spare for the sum's roundings)
  N.unscale = N.inv / N.scale;
  N.mean = mean;
  N.rstd = rstd;
  hipError_t e = launch_norm(N, dt, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ZERO_OK : hip_fail(e, "layer norm launch");
}

int zero_layer_norm_backward(const void* dy, int64_t dy_ld, const void* x, int64_t x_ld, int32_t dt, int64_t rows,
                             int64_t cols, const void* weight, int32_t w_dt, const float* mean, const float* rstd,
                             const void* dresidual, int64_t dresidual_ld, void* dx, int64_t dx_ld, void* dweight,
                             void* dbias, int32_t dw_dt, int32_t accumulate, void* workspace, size_t workspace_bytes,
                             void* stream) {
  if (int rc = check_norm(dt, w_dt, rows, cols)) return rc;
  if (int rc = check_rows("dy", dy, dt, rows, cols, dy_ld)) return rc;
  if (int rc = check_rows("x", x, dt, rows, cols, x_ld)) return rc;
  if (int rc = check_rows("dx", dx, dt, rows, cols, dx_ld)) return rc;
  if (dresidual)
    if (int rc = check_rows("dresidual", dresidual, dt, rows, cols, dresidual_ld)) return rc;
  const bool sums = dweight || dbias;
  if (sums) {
    if (int rc = check_dt("dweight", dw_dt)) return rc;
    if (int rc = check_vector("dweight", dweight, dw_dt, false)) return rc;
    if (int rc = check_vector("dbias", dbias, dw_dt, false)) return rc;
    if (int rc = check_workspace(workspace, workspace_bytes)) return rc;
  }
  if (cols == 0 || (rows == 0 && !sums)) return ZERO_OK;
  if (int rc = check_vector("weight", weight, w_dt, rows > 0)) return rc;
  if (int rc = check_vector("mean", mean, ZERO_DT_F32, rows > 0)) return rc;
  if (int rc = check_vector("rstd", rstd, ZERO_DT_F32, rows > 0)) return rc;
  if (int rc = check_device()) return rc;
  NormGradArgs N;
  N.dy = {dy, dy_ld};
  N.x = {x, x_ld};
  N.dresidual = {dresidual, dresidual_ld};
  N.dx = {dx, dx_ld};
  N.rows = rows;
  N.cols = static_cast<int32_t>(cols);
  N.weight = weight;
  N.w_dt = w_dt;
  N.mean = mean;
  N.rstd = rstd;
  N.dweight = dweight;
  N.dbias = dbias;
  N.dw_dt = dw_dt;
  N.accumulate = accumulate != 0;
  N.partials = sums ? reinterpret_cast<float*>(scratch_of(workspace)) : nullptr;
  hipError_t e = launch_norm_grad(N, dt, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ZERO_OK : hip_fail(e, "layer norm gradient launch");
}

int zero_dropout(const void* x, int32_t dt, int64_t rows, int64_t cols, int64_t x_ld, const void* residual,
                 int64_t residual_ld, void* y, int64_t y_ld, double p, uint64_t seed, uint64_t offset,
                 const int64_t* counter, int64_t first, void* stream) {
  if (rows < 0 || cols < 0) return fail(ZERO_ERR_INVALID_ARG, "rows or cols < 0");
  if (int rc = check_dt("x", dt)) return rc;
  const double limit = nearbyint(p * 4294967296.0);
  if (!(p >= 0) || !(limit < 4294967296.0)) return fail(ZERO_ERR_INVALID_ARG, "p = %g is not in [0, 1)", p);
  if (int rc = check_rows("x", x, dt, rows, cols, x_ld)) return rc;
  if (int rc = check_rows("y", y, dt, rows, cols, y_ld)) return rc;
  if (residual)
    if (int rc = check_rows("residual", residual, dt, rows, cols, residual_ld)) return rc;
  int64_t end;
  if (first < 0 || __builtin_mul_overflow(rows, cols, &end) || __builtin_add_overflow(first, end, &end))
    return fail(ZERO_ERR_INVALID_ARG, "first = %lld: elements [first, first + rows * cols) are not int64",
                (long long)first);
  if (!aligned(counter, 8)) return fail(ZERO_ERR_ALIGNMENT, "counter is not 8-byte aligned");
  if (rows == 0 || cols == 0) return ZERO_OK;
  if (int rc = check_device()) return rc;
  DropoutArgs D;
  D.x = {x, x_ld};
  D.residual = {residual, residual_ld};
  D.y = {y, y_ld};
  D.rows = rows;
  D.cols = cols;
  D.scale = static_cast<float>(1.0 / (1.0 - p));
  D.threshold = static_cast<uint32_t>(limit);
  D.seed = seed;
  D.offset = offset;
  D.first = static_cast<uint64_t>(first);
  D.counter = counter;
  hipError_t e = launch_dropout(D, dt, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ZERO_OK : hip_fail(e, "dropout launch");
}

int zero_gated_product(const void* x, int32_t dt, int64_t m, int64_t d, int64_t x_ld, const void* w_gate,
                       const void* w_up, int64_t f, int64_t w_ld, int32_t act, void* h, int64_t h_ld, void* gate,
                       void* up, int64_t pre_ld, void* stream) {
  if (int rc = check_gated(dt, m, d, f, act)) return rc;
  if (int rc = check_rows("x", x, dt, m, d, x_ld)) return rc;
  if (int rc = check_rows("w_gate", w_gate, dt, f, d, w_ld)) return rc;
  if (int rc = check_rows("w_up", w_up, dt, f, d, w_ld)) return rc;
  if (int rc = check_rows("h", h, dt, m, f, h_ld)) return rc;
  if ((gate == nullptr) != (up == nullptr)) return fail(ZERO_ERR_INVALID_ARG, "gate and up must be given together");
  if (gate) {
    if (int rc = check_rows("gate", gate, dt, m, f, pre_ld)) return rc;
    if (int rc = check_rows("up", up, dt, m, f, pre_ld)) return rc;
  }
  if (m == 0 || f == 0) return ZERO_OK;
  if (int rc = check_strides({x_ld, w_ld})) return rc;
  if (int rc = check_device()) return rc;
  GatedArgs G;
  G.x = {x, x_ld};
  G.w[0] = {w_gate, w_ld};
  G.w[1] = {w_up, w_ld};
  G.m = m;
  G.d = d;
  G.f = f;
  G.act = act;
  G.out[0] = {h, h_ld};
  G.out[1] = {gate, pre_ld};
  G.out[2] = {up, pre_ld};
  return launched(launch_gated(G, dt, static_cast<hipStream_t>(stream)), "gated product launch");
}

int zero_gated_product_backward(const void* dh, int64_t dh_ld, const void* x, int32_t dt, int64_t m, int64_t d,
                                int64_t x_ld, const void* w_gate, const void* w_up, int64_t f, int64_t w_ld, int32_t act,
                                const void* gate, const void* up, int64_t pre_ld, void* dgate, void* dup,
                                int64_t dpre_ld, void* dx, int64_t dx_ld, void* dw_gate, void* dw_up, int64_t dw_ld,
                                int32_t dw_dt, int32_t accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  if (int rc = check_gated(dt, m, d, f, act)) return rc;
  if (int rc = check_rows("dh", dh, dt, m, f, dh_ld)) return rc;
  if (int rc = check_rows("gate", gate, dt, m, f, pre_ld)) return rc;
  if (int rc = check_rows("up", up, dt, m, f, pre_ld)) return rc;
  if (int rc = check_rows("dgate", dgate, dt, m, f, dpre_ld)) return rc;
  if (int rc = check_rows("dup", dup, dt, m, f, dpre_ld)) return rc;
  if (dx) {
    if (int rc = check_rows("dx", dx, dt, m, d, dx_ld)) return rc;
    if (int rc = check_rows("w_gate", w_gate, dt, f, d, w_ld)) return rc;
    if (int rc = check_rows("w_up", w_up, dt, f, d, w_ld)) return rc;
    if (int rc = check_strides({w_ld})) return rc;
  }
  if ((dw_gate == nullptr) != (dw_up == nullptr))
    return fail(ZERO_ERR_INVALID_ARG, "dw_gate and dw_up must be given together");
  if (dw_gate) {
    if (dw_dt != dt && dw_dt != ZERO_DT_F32)
      return fail(ZERO_ERR_INVALID_ARG, "dw_gate: dtype %d is neither x's %d nor f32", dw_dt, dt);
    if (int rc = check_rows("x", x, dt, m, d, x_ld)) return rc;
    if (int rc = check_rows("dw_gate", dw_gate, dw_dt, f, d, dw_ld)) return rc;
    if (int rc = check_rows("dw_up", dw_up, dw_dt, f, d, dw_ld)) return rc;
    if (int rc = check_strides({x_ld})) return rc;
  }
  if (int rc = check_strides({dpre_ld})) return rc;
  if (int rc = check_workspace(workspace, workspace_bytes)) return rc;
  if (int rc = check_device()) return rc;
  GatedGradArgs G;
  G.dh = {dh, dh_ld};
  G.x = {x, x_ld};
  G.w[0] = {w_gate, w_ld};
  G.w[1] = {w_up, w_ld};
  G.pre[0] = {gate, pre_ld};
  G.pre[1] = {up, pre_ld};
  G.m = m;
  G.d = d;
  G.f = f;
  G.act = act;
  G.dpre[0] = {dgate, dpre_ld};
  G.dpre[1] = {dup, dpre_ld};
  G.dx = {dx, dx_ld};
  G.dw[0] = {dw_gate, dw_ld};
  G.dw[1] = {dw_up, dw_ld};
  G.dw_dt = dw_dt;
  G.accumulate = accumulate != 0;
  G.scratch = reinterpret_cast<float*>(scratch_of(workspace));
  return launched(launch_gated_grad(G, dt, static_cast<hipStream_t>(stream)), "gated product gradient launch");
}

}  // extern "C"
