// Internal interface between the host side of the microscaled 4-bit calls
// (mx_api.cpp) and their kernels (mx_quant.hip, mx_product.hip).
//
// The format (declared in include/zero_dp.h): blocks of kMxBlock values share
// one biased power-of-two exponent byte; a value is a 4-bit E2M1 code, two
// codes a byte, the even element in the low nibble. Codes and scales are
// separate arrays: block b has its 16 bytes of codes at codes + 16 * b and its
// scale at scales[b]. A matrix has `ld` blocks from one row to the next.
#pragma once

#include "zero_dp_internal.h"

namespace zdp {

constexpr int kMxBlock = 32;       // values that share a scale
constexpr int kMxCodeBytes = 16;   // bytes of codes in a block
constexpr int kMxNaN = 255;        // the scale byte of a block that holds inf or NaN

// Blocks from row to row of a product's operand: the byte offsets inside a tile
// of 256 rows are 32-bit.
constexpr int64_t kMxMaxLd = ZERO_MX_MAX_LD;
static_assert((256 * kMxMaxLd) * kMxCodeBytes < (int64_t{1} << 32), "offsets of a tile");

inline int64_t mx_blocks(int64_t values) { return values / kMxBlock + (values % kMxBlock != 0); }
inline int64_t mx_tiles(int64_t n, int64_t size) { return n / size + (n % size != 0); }

struct MxQuantArgs {
  const void* src;  // rows x cols values of src_dt, `src_ld` values from row to row
  int64_t rows, cols, src_ld;
  uint8_t* codes;   // along the rows (null: not wanted)
  uint8_t* scales;
  int64_t ld;
  uint8_t* codes_t;  // of the transpose (null: not wanted)
  uint8_t* scales_t;
  int64_t ld_t;
};

struct MxWidenArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t rows, cols, ld;
  void* out;  // rows x cols values of out_dt, `out_ld` values from row to row
  int64_t out_ld;
};

// N_d copies of a shard in 4 bits: copy r at codes[r] / scales[r], or (strided)
// at codes[0] + r * code_stride / scales[0] + r * scale_stride.
struct MxCopies {
  const uint8_t* codes[kInlineReplicas];
  const uint8_t* scales[kInlineReplicas];
  int64_t code_stride, scale_stride;
  int32_t n_d, strided;
  float inv_nd;  // as GradSource
  float nd;
};

struct MxReduceArgs {
  MxCopies src;
  int64_t n;
  float* avg_out;
  const zero_step_state* state;
  double* partials;
  double* level2;    // as ReduceArgs
  int32_t fill = 0;  // as ReduceArgs
};

struct MxProductArgs {
  const uint8_t* a_codes;
  const uint8_t* a_scales;
  int64_t lda;
  const uint8_t* b_codes;
  const uint8_t* b_scales;
  int64_t ldb;
  int64_t m, n, kb;  // kb: blocks along the contraction
  void* out;         // m x n values of out_dt, `ldo` values from row to row
  int64_t ldo;
};

hipError_t launch_mx_quantize(const MxQuantArgs& a, int32_t src_dt, hipStream_t s);
hipError_t launch_mx_widen(const MxWidenArgs& a, int32_t out_dt, hipStream_t s);
hipError_t launch_mx_reduce(const MxReduceArgs& a, hipStream_t s, int* blocks);
hipError_t launch_mx_product(const MxProductArgs& a, int32_t out_dt, hipStream_t s);

}  // namespace zdp
