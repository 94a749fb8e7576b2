// Host side of a layer's operators (include/zero_dp.h): argument checks and launches.
#include <hip/hip_runtime.h>
#include <math.h>

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

}  // namespace

extern "C" {

int zero_layer_norm(const void* x, int32_t dt, int64_t rows, int64_t cols, int64_t x_ld, const void* weight,
                    const void* bias, int32_t w_dt, double eps, void* y, int64_t y_ld, float* mean, float* rstd,
                    void* stream) {
  if (int rc = check_norm(dt, w_dt, rows, cols)) return rc;
  if (!(eps >= 0) || !isfinite(eps)) return fail(ZERO_ERR_INVALID_ARG, "eps = %g", eps);
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
  N.eps = static_cast<float>(eps);
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

}  // extern "C"
