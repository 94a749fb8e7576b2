// gfx950 kernels of the product of two microscaled 4-bit matrices,
//   out[i][j] = sum_k A[i][k] * B[j][k],
// on the scaled matrix instruction v_mfma_scale_f32_32x32x64 with both operands
// in E2M1: lane l of a wave gives row l & 31 of either operand and its 32-value
// block l >> 5 of the instruction's two, so a lane's operand is exactly one
// block (16 bytes of codes) and its scale byte. The instruction multiplies by
// both scales, and sums in fp32.
#include "mx_device.h"

namespace zdp {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));

constexpr int kE2M1 = 4;  // the instruction's format code for both operands

__device__ __forceinline__ v16f mfma(v4i a, uint32_t sa, v4i b, uint32_t sb, v16f c) {
  const v8i A = {a.x, a.y, a.z, a.w, 0, 0, 0, 0}, B = {b.x, b.y, b.z, b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(A, B, c, kE2M1, kE2M1, 0, static_cast<int>(sa), 0,
                                                         static_cast<int>(sb));
}

template <int DT>
__device__ __forceinline__ void store_value(void* out, int64_t at, float x) {
  if constexpr (DT == ZERO_DT_F32) static_cast<float*>(out)[at] = x;
  else static_cast<uint16_t*>(out)[at] = static_cast<uint16_t>(encode16(x, DT));
}

// One wave per 32 x 32 tile of the output.
template <int DT>
__global__ void __launch_bounds__(64) mx_product_kernel(const MxProductArgs P) {
  const int r = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int64_t nt = (P.n + 31) / 32;
  const int64_t m0 = blockIdx.x / nt * 32, n0 = blockIdx.x % nt * 32;
  const int64_t i = m0 + r < P.m ? m0 + r : P.m - 1, j = n0 + r < P.n ? n0 + r : P.n - 1;
  v16f c = {};
  for (int64_t k = 0; k < P.kb; k += 2) {
    v4i a = {}, b = {};
    uint32_t sa = 0, sb = 0;
    if (k + g < P.kb) {
      a = reinterpret_cast<const v4i*>(P.a_codes)[i * P.lda + k + g];
      b = reinterpret_cast<const v4i*>(P.b_codes)[j * P.ldb + k + g];
      sa = P.a_scales[i * P.lda + k + g];
      sb = P.b_scales[j * P.ldb + k + g];
    }
    c = mfma(a, sa, b, sb, c);
  }
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    const int64_t row = m0 + (q >> 2) * 8 + g * 4 + (q & 3), col = n0 + r;
    if (row < P.m && col < P.n) store_value<DT>(P.out, row * P.ldo + col, c[q]);
  }
}

}  // namespace

hipError_t launch_mx_product(const MxProductArgs& a, int32_t dt, hipStream_t s) {
  const int64_t tiles = (a.m + 31) / 32 * ((a.n + 31) / 32);
  const dim3 grid(static_cast<uint32_t>(tiles));
  if (dt == ZERO_DT_F32) hipLaunchKernelGGL(mx_product_kernel<ZERO_DT_F32>, grid, dim3(64), 0, s, a);
  else if (dt == ZERO_DT_F16) hipLaunchKernelGGL(mx_product_kernel<ZERO_DT_F16>, grid, dim3(64), 0, s, a);
  else if (dt == ZERO_DT_BF16) hipLaunchKernelGGL(mx_product_kernel<ZERO_DT_BF16>, grid, dim3(64), 0, s, a);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

}  // namespace zdp
