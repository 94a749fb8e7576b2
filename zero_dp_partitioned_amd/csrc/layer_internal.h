// Internal interface between the host side of a layer's operators (layer_api.cpp)
// and their kernels (layer_norm.hip, dropout.hip, gated_product.hip).
#pragma once

#include "zero_dp_internal.h"

namespace zdp {

inline int64_t ceil_div(int64_t n, int64_t size) { return n / size + (n % size != 0); }

// rows x cols values, `ld` values from row to row.
struct Rows {
  const void* p;
  int64_t ld;
};
struct RowsOut {
  void* p;
  int64_t ld;
};

constexpr int32_t kMaxNormCols = 1 << 20;

struct NormArgs {
  Rows x;
  RowsOut y;
  int64_t rows;
  int32_t cols;
  const void* weight;
  const void* bias;  // or null
  int32_t w_dt;      // of weight and bias: x's type or F32
  float eps;
  float inv;      // 1 / cols
  float scale;    // a power of two below it
  float unscale;  // what makes a sum of values times `scale` the mean
  float* mean;    // one a row, or null (both)
  float* rstd;
};

struct NormGradArgs {
  Rows dy, x, dresidual;  // dresidual.p may be null
  RowsOut dx;
  int64_t rows;
  int32_t cols;
  const void* weight;
  int32_t w_dt;
  const float* mean;
  const float* rstd;
  void* dweight;  // or null
  void* dbias;    // or null
  int32_t dw_dt;  // of dweight and dbias
  int32_t accumulate;
  float* partials;  // of the column sums: a row of `cols` for dy * xhat and one for dy, per block
};

struct DropoutArgs {
  Rows x, residual;  // residual.p may be null
  RowsOut y;
  int64_t rows, cols;
  float scale;          // 1 / (1 - p)
  uint32_t threshold;   // words below it drop their element
  uint64_t seed, offset, first;
  const int64_t* counter;  // added to offset, or null
};

// h = act(x wg^T) * (x wu^T): x m x d, wg and wu f x d.
struct GatedArgs {
  Rows x, w[2];
  int64_t m, d, f;
  int32_t act;
  RowsOut out[3];  // h, and the two products (or null)
};

// dg = dh act'(g) u, du = dh act(g); dx = dg wg + du wu, dw = {dg^T x, du^T x}.
struct GatedGradArgs {
  Rows dh, x, w[2], pre[2];  // pre: g and u
  int64_t m, d, f;
  int32_t act;
  RowsOut dpre[2];  // dg and du
  RowsOut dx;       // or null
  RowsOut dw[2];    // or null (both)
  int32_t dw_dt;
  int32_t accumulate;
  float* scratch;  // partial sums of products that few tiles would compute
};

// Values from row to row of a product's operand: byte offsets inside a tile of
// 256 rows are 32-bit.
constexpr int64_t kMaxRowStride = 4194303;
static_assert(256 * kMaxRowStride * 2 < (int64_t{1} << 32), "offsets of a tile");

hipError_t launch_norm(const NormArgs& a, int32_t dt, hipStream_t s);
hipError_t launch_norm_grad(const NormGradArgs& a, int32_t dt, hipStream_t s);
hipError_t launch_dropout(const DropoutArgs& a, int32_t dt, hipStream_t s);
hipError_t launch_gated(const GatedArgs& a, int32_t dt, hipStream_t s);
hipError_t launch_gated_grad(const GatedGradArgs& a, int32_t dt, hipStream_t s);

}  // namespace zdp
