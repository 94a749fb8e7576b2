// Device helpers of the microscaled 4-bit kernels. The first part (encodings,
// norm partials) repeats what the step's kernels (kernels.hip) keep to
// themselves: the traffic measured for the step is recorded with that file's
// text, which therefore stays as it was.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "mx_internal.h"

#pragma clang fp contract(off)

namespace zdp {
namespace {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef unsigned u2 __attribute__((ext_vector_type(2)));
typedef unsigned u4 __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------------
// Streaming accesses: the non-temporal hint.
// ------------------------------------------------------------------------

template <typename T>
__device__ __forceinline__ T ld_stream(const T* p) {
  return __builtin_nontemporal_load(p);
}

template <typename T>
__device__ __forceinline__ void st_stream(T* p, T x) {
  __builtin_nontemporal_store(x, p);
}

// 16 bytes at any alignment of a smaller type.
typedef u4 u4_any __attribute__((aligned(2)));

// ------------------------------------------------------------------------
// 16-bit encodings
// ------------------------------------------------------------------------

template <int DT>
__device__ __forceinline__ float decode16(uint32_t h) {
  if constexpr (DT == kSrcBF16) {
    return __uint_as_float(h << 16);
  } else {
    const _Float16 x = __builtin_bit_cast(_Float16, static_cast<uint16_t>(h));
    return static_cast<float>(x);
  }
}

// fp32 -> 16 bits, round to nearest even, NaN -> canonical quiet NaN.
__device__ __forceinline__ uint32_t encode16(float x, int dt) {
  if (__builtin_isnan(x)) return dt == ZERO_DT_BF16 ? 0x7FC0u : 0x7E00u;
  if (dt == ZERO_DT_BF16) {
    uint32_t u = __float_as_uint(x);
    u += 0x7FFFu + ((u >> 16) & 1u);
    return u >> 16;
  }
  const _Float16 h = static_cast<_Float16>(x);
  return __builtin_bit_cast(uint16_t, h);
}

// ------------------------------------------------------------------------
// Norm and overflow partials, as the step's kernels write them
// ------------------------------------------------------------------------

// Norm / overflow contribution of one averaged gradient.
__device__ __forceinline__ void account(float a, float g, double& sumsq, int& bad) {
  bad |= !__builtin_isfinite(a);
  const double gd = static_cast<double>(g);
  sumsq = __builtin_fma(gd, gd, sumsq);
}

// One fp64 partial per block: wavefront butterfly, then the block's four
// wavefronts through LDS in a fixed order. NaN marks a non-finite gradient.
// With fill > gridDim.x (a small launch writing a group's level-2 partials
// directly) the blocks also zero the slots [gridDim.x, fill), each once.
__device__ __forceinline__ void write_block_partial(double s, int bad, double* out, int fill) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off, 64);
  const int any_bad = __any(bad);
  __shared__ double ws[kBlock / 64];
  __shared__ int wf[kBlock / 64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  if (lane == 0) {
    ws[w] = s;
    wf[w] = any_bad;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    double t = 0.0;
    int f = 0;
#pragma unroll
    for (int k = 0; k < kBlock / 64; ++k) {
      t += ws[k];
      f |= wf[k];
    }
    out[blockIdx.x] = f ? __builtin_nan("") : t;
    for (int k = blockIdx.x + gridDim.x; k < fill; k += gridDim.x) out[k] = 0.0;
  }
}

// A launch of at most kFoldBlocks blocks with the group's level-2 partials at
// hand writes them itself: block b's partial into slot b, zeros into the
// slots past its grid. That is what the fold would write: with one partial
// per slot, its sums only add zeros, which changes no bit (a partial, a sum
// of squares from +0, is never -0). *blocks = 0 then tells the caller that
// nothing is left to fold; otherwise it is the grid.
template <typename Args>
Args route_partials(const Args& a, int grid, int* blocks) {
  Args b = a;
  b.fill = 0;
  *blocks = grid;
  if (a.level2 && a.partials && grid <= kFoldBlocks) {
    b.partials = a.level2;
    b.fill = kFoldBlocks;
    *blocks = 0;
  }
  return b;
}

typedef float f2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));

// The largest of 4 or 8 neighbouring lanes.
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t x) {
  static_assert(LANES == 4 || LANES == 8, "");
  const uint32_t a = __builtin_amdgcn_update_dpp(0, x, 0xB1, 0xF, 0xF, true);  // lanes 1,0,3,2
  x = x > a ? x : a;
  const uint32_t b = __builtin_amdgcn_update_dpp(0, x, 0x4E, 0xF, 0xF, true);  // lanes 2,3,0,1
  x = x > b ? x : b;
  if constexpr (LANES == 8) {
    const uint32_t c = __builtin_amdgcn_update_dpp(0, x, 0x141, 0xF, 0xF, true);  // 7,6,5,4,3,2,1,0 of eight
    x = x > c ? x : c;
  }
  return x;
}

// Four lanes' a[0..3], transposed: lane l's a[k] becomes lane k's a[l].
__device__ __forceinline__ void quad_transpose(uint32_t a[4], int lane) {
  const bool odd = lane & 1, high = lane & 2;
#pragma unroll
  for (int k = 0; k < 4; k += 2) {
    const uint32_t t = __builtin_amdgcn_update_dpp(0, odd ? a[k] : a[k + 1], 0xB1, 0xF, 0xF, true);
    a[k] = odd ? t : a[k];
    a[k + 1] = odd ? a[k + 1] : t;
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t t = __builtin_amdgcn_update_dpp(0, high ? a[k] : a[k + 2], 0x4E, 0xF, 0xF, true);
    a[k] = high ? t : a[k];
    a[k + 2] = high ? a[k + 2] : t;
  }
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

// 16 bytes of values of type DT (ZERO_DT_F32 / F16 / BF16), as they lie in memory.
template <int DT>
struct Raw {
  static constexpr int kElem = DT == ZERO_DT_F32 ? 4 : 2;
  static constexpr int kVals = 16 / kElem;
  static constexpr int kLanes = kMxBlock / kVals;  // that share a block
  using Codes = typename std::conditional<DT == ZERO_DT_F32, uint16_t, uint32_t>::type;  // of kVals values
  uint32_t w[4];
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

// The codes of Raw<DT>::kVals values, element 0 in the low nibble. A NaN block's are 0.
template <int DT>
__device__ __forceinline__ uint32_t encode(const uint32_t* w, uint32_t byte) {
  const float s = scale_operand(byte);
  uint32_t c = 0;
  if constexpr (DT == ZERO_DT_F32) {
    c = encode2<DT, 0>(c, w[0], w[1], s);
    c = encode2<DT, 1>(c, w[2], w[3], s);
  } else {
    c = encode2<DT, 0>(c, w[0], 0, s);
    c = encode2<DT, 1>(c, w[1], 0, s);
    c = encode2<DT, 2>(c, w[2], 0, s);
    c = encode2<DT, 3>(c, w[3], 0, s);
  }
  return byte == 255u ? 0u : c;
}

// Four codes (the low 16 bits of c) times the scale s, in fp32 (exact; NaN for the scale of a NaN block).
__device__ __forceinline__ f4 decode4(uint32_t c, float s) {
  const f2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0);
  const f2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1);
  return (f4){a.x, a.y, b.x, b.y};
}

}  // namespace
}  // namespace zdp
