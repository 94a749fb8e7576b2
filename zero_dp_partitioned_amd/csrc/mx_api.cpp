// Host side of the microscaled 4-bit calls (include/zero_dp.h): argument checks
// and launches.
#include <hip/hip_runtime.h>
#include <string.h>

#include "api_common.h"
#include "mx_internal.h"

using namespace zdp;

namespace {

bool valid_mx_dt(int32_t dt) { return dt == ZERO_DT_F32 || dt == ZERO_DT_F16 || dt == ZERO_DT_BF16; }
uintptr_t dt_bytes(int32_t dt) { return dt == ZERO_DT_F32 ? 4 : 2; }

// rows * stride elements of `bytes` each must have an int64 byte count.
bool extent_ok(int64_t rows, int64_t stride, int64_t bytes) {
  int64_t t;
  return !__builtin_mul_overflow(rows, stride, &t) && !__builtin_mul_overflow(t, bytes, &t);
}

// A 4-bit matrix of `rows` rows of `blocks` blocks.
int check_mx(const char* what, const void* codes, const void* scales, int64_t rows, int64_t blocks, int64_t ld) {
  if (ld < blocks)
    return fail(ZERO_ERR_INVALID_ARG, "%s: ld = %lld blocks, fewer than a row's %lld", what, (long long)ld,
                (long long)blocks);
  if (!extent_ok(rows, ld, kMxCodeBytes)) return fail(ZERO_ERR_INVALID_ARG, "%s: extent overflows int64", what);
  if (rows == 0 || blocks == 0) return ZERO_OK;
  if (!codes || !scales) return fail(ZERO_ERR_INVALID_ARG, "%s: codes or scales is NULL", what);
  if (!aligned(codes, kMxCodeBytes)) return fail(ZERO_ERR_ALIGNMENT, "%s: codes are not 16-byte aligned", what);
  return ZERO_OK;
}

// A rows x cols array of dt.
int check_values(const char* what, const void* p, int32_t dt, int64_t rows, int64_t cols, int64_t ld) {
  if (!valid_mx_dt(dt)) return fail(ZERO_ERR_INVALID_ARG, "%s: dtype %d is not f32/f16/bf16", what, dt);
  if (ld < cols)
    return fail(ZERO_ERR_INVALID_ARG, "%s: %lld elements from row to row, fewer than a row's %lld", what, (long long)ld,
                (long long)cols);
  if (!extent_ok(rows, ld, static_cast<int64_t>(dt_bytes(dt))))
    return fail(ZERO_ERR_INVALID_ARG, "%s: extent overflows int64", what);
  if (rows == 0 || cols == 0) return ZERO_OK;
  if (!p) return fail(ZERO_ERR_INVALID_ARG, "%s is NULL", what);
  if (!aligned(p, dt_bytes(dt))) return fail(ZERO_ERR_ALIGNMENT, "%s is not aligned to its elements", what);
  return ZERO_OK;
}

// The copies' pointers; more than the inline table holds must be equally spaced.
int make_copies(const void* const* codes, const void* const* scales, int32_t n_d, int64_t n, MxCopies* S) {
  memset(S, 0, sizeof *S);
  if (!codes || !scales) return fail(ZERO_ERR_INVALID_ARG, "codes or scales pointer array is NULL");
  if (n_d < 1) return fail(ZERO_ERR_INVALID_ARG, "n_d = %d < 1", n_d);
  if (n_d > ZERO_MAX_REPLICAS) return fail(ZERO_ERR_UNSUPPORTED, "n_d = %d > %d", n_d, ZERO_MAX_REPLICAS);
  S->n_d = n_d;
  S->nd = static_cast<float>(n_d);
  S->inv_nd = (n_d & (n_d - 1)) == 0 ? 1.0f / static_cast<float>(n_d) : 0.0f;
  if (n == 0) return ZERO_OK;
  for (int32_t r = 0; r < n_d; ++r) {
    if (!codes[r] || !scales[r]) return fail(ZERO_ERR_INVALID_ARG, "copy %d: codes or scales is NULL", r);
    if (!aligned(codes[r], kMxCodeBytes)) return fail(ZERO_ERR_ALIGNMENT, "copy %d: codes are not 16-byte aligned", r);
  }
  if (n_d <= kInlineReplicas) {
    for (int32_t r = 0; r < n_d; ++r) {
      S->codes[r] = static_cast<const uint8_t*>(codes[r]);
      S->scales[r] = static_cast<const uint8_t*>(scales[r]);
    }
    return ZERO_OK;
  }
  const uint8_t* c0 = static_cast<const uint8_t*>(codes[0]);
  const uint8_t* s0 = static_cast<const uint8_t*>(scales[0]);
  S->code_stride = static_cast<const uint8_t*>(codes[1]) - c0;
  S->scale_stride = static_cast<const uint8_t*>(scales[1]) - s0;
  for (int32_t r = 0; r < n_d; ++r)
    if (static_cast<const uint8_t*>(codes[r]) - c0 != r * S->code_stride ||
        static_cast<const uint8_t*>(scales[r]) - s0 != r * S->scale_stride)
      return fail(ZERO_ERR_UNSUPPORTED, "n_d > %d needs equally spaced copies", kInlineReplicas);
  S->codes[0] = c0;
  S->scales[0] = s0;
  S->strided = 1;
  return ZERO_OK;
}

}  // namespace

extern "C" {

int zero_mx_cast_writeback(const float* master, int64_t n, void* codes, void* scales, int64_t offset, void* stream) {
  if (n < 0) return fail(ZERO_ERR_INVALID_ARG, "n < 0");
  if (offset < 0 || offset % kMxBlock)
    return fail(ZERO_ERR_INVALID_ARG, "offset = %lld is not a multiple of %d", (long long)offset, kMxBlock);
  if (n == 0) return ZERO_OK;  // nothing to write
  if (!codes || !scales) return fail(ZERO_ERR_INVALID_ARG, "codes or scales is NULL");
  uint8_t* c = static_cast<uint8_t*>(codes) + offset / kMxBlock * kMxCodeBytes;
  uint8_t* s = static_cast<uint8_t*>(scales) + offset / kMxBlock;
  return zero_mx_quantize(master, ZERO_DT_F32, 1, n, n, c, s, mx_blocks(n), nullptr, nullptr, 0, stream);
}

int zero_mx_quantize(const void* src, int32_t src_dt, int64_t rows, int64_t cols, int64_t src_ld, void* codes,
                     void* scales, int64_t ld, void* codes_t, void* scales_t, int64_t ld_t, void* stream) {
  if (rows < 0 || cols < 0) return fail(ZERO_ERR_INVALID_ARG, "rows or cols < 0");
  if (int rc = check_values("src", src, src_dt, rows, cols, src_ld)) return rc;
  if ((codes == nullptr) != (scales == nullptr) || (codes_t == nullptr) != (scales_t == nullptr))
    return fail(ZERO_ERR_INVALID_ARG, "codes and scales must be given together");
  if (rows == 0 || cols == 0) return ZERO_OK;  // no blocks
  if (!codes && !codes_t) return fail(ZERO_ERR_INVALID_ARG, "no output");
  if (codes)
    if (int rc = check_mx("output", codes, scales, rows, mx_blocks(cols), ld)) return rc;
  if (codes_t)
    if (int rc = check_mx("transposed output", codes_t, scales_t, cols, mx_blocks(rows), ld_t)) return rc;
  if (int rc = check_device()) return rc;
  MxQuantArgs Q;
  Q.src = src;
  Q.rows = rows;
  Q.cols = cols;
  Q.src_ld = src_ld;
  Q.codes = static_cast<uint8_t*>(codes);
  Q.scales = static_cast<uint8_t*>(scales);
  Q.ld = ld;
  Q.codes_t = static_cast<uint8_t*>(codes_t);
  Q.scales_t = static_cast<uint8_t*>(scales_t);
  Q.ld_t = ld_t;
  hipError_t e = launch_mx_quantize(Q, src_dt, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ZERO_OK : hip_fail(e, "quantise launch");
}

int zero_mx_dequantize(const void* codes, const void* scales, int64_t rows, int64_t cols, int64_t ld, void* out,
                       int32_t out_dt, int64_t out_ld, void* stream) {
  if (rows < 0 || cols < 0) return fail(ZERO_ERR_INVALID_ARG, "rows or cols < 0");
  if (int rc = check_values("out", out, out_dt, rows, cols, out_ld)) return rc;
  if (int rc = check_mx("input", codes, scales, rows, mx_blocks(cols), ld)) return rc;
  if (rows == 0 || cols == 0) return ZERO_OK;
  if (int rc = check_device()) return rc;
  MxWidenArgs W;
  W.codes = static_cast<const uint8_t*>(codes);
  W.scales = static_cast<const uint8_t*>(scales);
  W.rows = rows;
  W.cols = cols;
  W.ld = ld;
  W.out = out;
  W.out_ld = out_ld;
  hipError_t e = launch_mx_widen(W, out_dt, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ZERO_OK : hip_fail(e, "widen launch");
}

int zero_mx_reduce_grad_segment(const void* const* codes, const void* const* scales, int32_t n_d, int64_t n,
                                float* avg_out, void* workspace, size_t workspace_bytes, int32_t group,
                                const zero_step_state* state, void* stream) {
  if (n < 0) return fail(ZERO_ERR_INVALID_ARG, "n < 0");
  if (!avg_out && n > 0) return fail(ZERO_ERR_INVALID_ARG, "avg_out is NULL");
  if (!aligned(avg_out, 4)) return fail(ZERO_ERR_ALIGNMENT, "avg_out is not 4-byte aligned");
  if (!state) return fail(ZERO_ERR_INVALID_ARG, "state is NULL");
  if (int rc = check_workspace(workspace, workspace_bytes)) return rc;
  if (group < 0 || group >= ZERO_MAX_GROUPS) return fail(ZERO_ERR_WORKSPACE, "group %d out of range", group);
  MxReduceArgs R;
  if (int rc = make_copies(codes, scales, n_d, n, &R.src)) return rc;
  if (int rc = check_device()) return rc;
  R.n = n;
  R.avg_out = avg_out;
  R.state = state;
  R.partials = scratch_of(workspace);
  R.level2 = level2_of(workspace, group);
  hipStream_t s = static_cast<hipStream_t>(stream);
  int blocks = 0;
  hipError_t e = launch_mx_reduce(R, s, &blocks);
  if (e != hipSuccess) return hip_fail(e, "4-bit average launch");
  e = fold_into(workspace, group, blocks, s);
  return e == hipSuccess ? ZERO_OK : hip_fail(e, "fold launch");
}

int zero_mx_product(const void* a_codes, const void* a_scales, int64_t lda, const void* b_codes, const void* b_scales,
                    int64_t ldb, int64_t m, int64_t n, int64_t k_blocks, void* out, int32_t out_dt, int64_t ldo,
                    void* stream) {
  if (m < 0 || n < 0 || k_blocks < 0) return fail(ZERO_ERR_INVALID_ARG, "m, n or k_blocks < 0");
  if (m > INT32_MAX || n > INT32_MAX) return fail(ZERO_ERR_UNSUPPORTED, "more than 2^31 - 1 rows");
  if (int rc = check_mx("A", a_codes, a_scales, m, k_blocks, lda)) return rc;
  if (int rc = check_mx("B", b_codes, b_scales, n, k_blocks, ldb)) return rc;
  if (int rc = check_values("out", out, out_dt, m, n, ldo)) return rc;
  if (m == 0 || n == 0) return ZERO_OK;
  if (lda > kMxMaxLd || ldb > kMxMaxLd)
    return fail(ZERO_ERR_UNSUPPORTED, "rows more than %lld blocks apart", (long long)kMxMaxLd);
  if (int rc = check_device()) return rc;
  MxProductArgs P;
  P.a_codes = static_cast<const uint8_t*>(a_codes);
  P.a_scales = static_cast<const uint8_t*>(a_scales);
  P.lda = lda;
  P.b_codes = static_cast<const uint8_t*>(b_codes);
  P.b_scales = static_cast<const uint8_t*>(b_scales);
  P.ldb = ldb;
  P.m = m;
  P.n = n;
  P.kb = k_blocks;
  P.out = out;
  P.ldo = ldo;
  hipError_t e = launch_mx_product(P, out_dt, static_cast<hipStream_t>(stream));
  if (e == hipErrorInvalidConfiguration) return fail(ZERO_ERR_UNSUPPORTED, "more output tiles than a launch holds");
  return e == hipSuccess ? ZERO_OK : hip_fail(e, "product launch");
}

}  // extern "C"
