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

// Eight values in their own type DT (ZERO_DT_F32 / F16 / BF16), as they lie in memory.
template <int DT>
struct Raw8 {
  static constexpr int kWords = DT == ZERO_DT_F32 ? 8 : 4;
  uint32_t w[kWords];
};

// The bits, in fp32, of the largest magnitude. 16-bit magnitudes compare as
// their bits too, two at a time.
template <int DT>
__device__ __forceinline__ uint32_t max_bits(const uint32_t* w, int words) {
  uint32_t m = 0;
  if constexpr (DT == ZERO_DT_F32) {
#pragma unroll
    for (int q = 0; q < words; ++q) {
      const uint32_t b = w[q] & 0x7FFFFFFFu;
      m = b > m ? b : m;
    }
    return m;
  } else {
    typedef unsigned short us2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int q = 0; q < words; ++q)
      m = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(us2, m),
                                                                 __builtin_bit_cast(us2, w[q] & 0x7FFF7FFFu)));
    const uint32_t top = (m >> 16) > (m & 0xFFFFu) ? m >> 16 : m & 0xFFFFu;
    return __float_as_uint(decode16<DT == ZERO_DT_BF16 ? kSrcBF16 : kSrcF16>(top));
  }
}

// Two values (fp32 words lo and hi, or the two halves of one 16-bit word `lo`)
// divided by the scale s and rounded to E2M1 codes (nearest even, saturating at
// +-6), into byte SEL of c.
template <int DT, int SEL>
__device__ __forceinline__ uint32_t encode2(uint32_t c, uint32_t lo, uint32_t hi, float s) {
  if constexpr (DT == ZERO_DT_F32)
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(lo), __uint_as_float(hi), s, SEL);
  else if constexpr (DT == ZERO_DT_BF16)
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf2, lo), s, SEL);
  else
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(h2, lo), s, SEL);
}

// Eight values' codes, element 0 in the low nibble. A NaN block's are 0.
template <int DT>
__device__ __forceinline__ uint32_t encode8(const uint32_t* w, uint32_t byte) {
  constexpr int K = DT == ZERO_DT_F32 ? 2 : 1;  // words per pair
  const float s = scale_operand(byte);
  uint32_t c = 0;
  c = encode2<DT, 0>(c, w[0], w[K - 1], s);
  c = encode2<DT, 1>(c, w[K], w[2 * K - 1], s);
  c = encode2<DT, 2>(c, w[2 * K], w[3 * K - 1], s);
  c = encode2<DT, 3>(c, w[3 * K], w[4 * K - 1], s);
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
