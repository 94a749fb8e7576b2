// Device helpers of the microscaled 4-bit kernels.
#pragma once

#include "device_common.h"
#include "mx_internal.h"

namespace zdp {
namespace {

typedef float f2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));

// Lanes of a quad that share a 32-value block: lane l ^ 1 and lane l ^ 2.
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
  const uint32_t a = __builtin_amdgcn_update_dpp(0, x, 0xB1, 0xF, 0xF, true);  // lanes 1,0,3,2
  x = x > a ? x : a;
  const uint32_t b = __builtin_amdgcn_update_dpp(0, x, 0x4E, 0xF, 0xF, true);  // lanes 2,3,0,1
  return x > b ? x : b;
}

// The scale byte of a block from the bits of its largest magnitude: the
// exponent field of max |v| less 2 (E2M1's largest exponent), at least 0; a
// zero or subnormal maximum has field 0 and gets 0 as well. Infinity and NaN
// have field 255 and make the block a NaN block. Magnitudes compare as their
// bits, so the maximum needs no floating compare and carries NaN along.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 23;
  return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}

// The conversions take the scale as an fp32 whose exponent field is the byte.
__device__ __forceinline__ float scale_operand(uint32_t byte) { return __uint_as_float(byte << 23); }

// Eight values divided by the block's scale and rounded to E2M1 codes (nearest
// even, saturating at +-6), element 0 in the low nibble. A NaN block's codes
// are 0.
__device__ __forceinline__ uint32_t encode8(const float v[8], uint32_t byte) {
  const float s = scale_operand(byte);
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], s, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], s, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], s, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], s, 3);
  return byte == 255u ? 0u : c;
}

// Eight codes times the block's scale, in fp32 (exact; NaN for a NaN block).
__device__ __forceinline__ void decode8(uint32_t c, float s, float v[8]) {
  const f2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0);
  const f2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1);
  const f2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 2);
  const f2 e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 3);
  v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
  v[4] = d.x; v[5] = d.y; v[6] = e.x; v[7] = e.y;
}

}  // namespace
}  // namespace zdp
