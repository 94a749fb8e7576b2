// Device code that the library's kernels share: streaming accesses, the 16-bit
// encodings, and the norm / overflow partials of a launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zero_dp_internal.h"

#pragma clang fp contract(off)

namespace zdp {
namespace {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef unsigned u2 __attribute__((ext_vector_type(2)));
typedef unsigned u4 __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------------
// Streaming accesses. Every byte a step touches is read once and written
// once, so the vector loads and stores of the quad paths carry the
// non-temporal hint: on gfx950 the read-modify-write of the fp32 state then
// sustains a few per cent more HBM bandwidth than with the default policy.
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
// Norm and overflow partials
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

}  // namespace
}  // namespace zdp
