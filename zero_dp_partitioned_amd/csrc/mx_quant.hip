// gfx950 kernels that write and read the microscaled 4-bit format: quantise,
// widen, and the average of a shard's N_d copies.
//
// All three are streaming passes. A lane handles 8 consecutive values, so four
// lanes share a 32-value block: the block's maximum is two quad permutes, a
// wave's codes are one contiguous 256-byte run, and the wide side of the pass
// (16-bit or fp32 values) moves 16 or 32 bytes a lane.
#include "mx_device.h"

namespace zdp {
namespace {

constexpr int kLane = 8;                   // values a lane handles
constexpr int kMxGroups = 4;               // groups of 8 a lane has in flight
constexpr int kLanesPerBlock = kMxBlock / kLane;

// Values e .. e+7 of a row of which `left` values from e on exist; the missing
// ones are 0. DT: ZERO_DT_F32 / F16 / BF16, any alignment of the type.
template <int DT>
__device__ __forceinline__ void load8(const void* row, int64_t e, int64_t left, float v[8]) {
  if constexpr (DT == ZERO_DT_F32) {
    const float* p = static_cast<const float*>(row) + e;
    if (left >= 8) {
      f4 a, b;
      __builtin_memcpy(&a, p, 16);
      __builtin_memcpy(&b, p + 4, 16);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = q < left ? p[q] : 0.0f;
    }
  } else {
    constexpr int K = DT == ZERO_DT_BF16 ? kSrcBF16 : kSrcF16;
    const uint16_t* p = static_cast<const uint16_t*>(row) + e;
    if (left >= 8) {
      u4 a;
      __builtin_memcpy(&a, p, 16);
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[2 * q] = decode16<K>(w[q] & 0xFFFFu);
        v[2 * q + 1] = decode16<K>(w[q] >> 16);
      }
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = q < left ? decode16<K>(p[q]) : 0.0f;
    }
  }
}

__device__ __forceinline__ uint32_t max_bits8(const float v[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const uint32_t b = __float_as_uint(v[q]) & 0x7FFFFFFFu;
    m = b > m ? b : m;
  }
  return m;
}

// ------------------------------------------------------------------------
// Quantise along the rows. Item i is quarter i % 4 of block i / 4, blocks
// counted row by row.
// ------------------------------------------------------------------------

template <int DT>
__global__ void __launch_bounds__(kBlock) mx_quantize_rows_kernel(const MxQuantArgs Q) {
  const int64_t kb = (Q.cols + kMxBlock - 1) / kMxBlock;
  const int64_t items = Q.rows * kb * kLanesPerBlock;
  constexpr int64_t T = static_cast<int64_t>(kBlock) * kMxGroups;
  for (int64_t t0 = blockIdx.x * T; t0 < items; t0 += gridDim.x * T) {
#pragma unroll
    for (int k = 0; k < kMxGroups; ++k) {
      const int64_t i = t0 + k * kBlock + threadIdx.x;
      const int64_t b = i / kLanesPerBlock;
      const int64_t row = Q.rows == 1 ? 0 : b / kb, bk = b - row * kb;
      const int64_t e = bk * kMxBlock + (i % kLanesPerBlock) * kLane;
      const int elem = DT == ZERO_DT_F32 ? 4 : 2;
      float v[8];
      load8<DT>(static_cast<const char*>(Q.src) + row * Q.src_ld * elem, e, i < items ? Q.cols - e : 0, v);
      const uint32_t byte = scale_byte(quad_max(max_bits8(v)));
      const uint32_t c = encode8(v, byte);
      if (i < items) {
        const int64_t at = row * Q.ld + bk;
        reinterpret_cast<uint32_t*>(Q.codes)[at * 4 + i % kLanesPerBlock] = c;
        if (i % kLanesPerBlock == 0) Q.scales[at] = static_cast<uint8_t>(byte);
      }
    }
  }
}

// ------------------------------------------------------------------------
// Quantise along the columns (the transpose's rows): item i is quarter i % 4
// of block i / 4, blocks counted column by column.
// ------------------------------------------------------------------------

template <int DT>
__global__ void __launch_bounds__(kBlock) mx_quantize_cols_kernel(const MxQuantArgs Q) {
  const int64_t rb = (Q.rows + kMxBlock - 1) / kMxBlock;
  const int64_t items = Q.cols * rb * kLanesPerBlock;
  for (int64_t t0 = blockIdx.x * static_cast<int64_t>(kBlock); t0 < items; t0 += static_cast<int64_t>(gridDim.x) * kBlock) {
    const int64_t i = t0 + threadIdx.x;
    const int64_t b = i / kLanesPerBlock;
    const int64_t col = b / rb, br = b - col * rb;
    const int64_t e = br * kMxBlock + (i % kLanesPerBlock) * kLane;
    float v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      float one[8] = {};
      if (i < items && e + q < Q.rows) {
        const int elem = DT == ZERO_DT_F32 ? 4 : 2;
        load8<DT>(static_cast<const char*>(Q.src) + (e + q) * Q.src_ld * elem, col, 1, one);
      }
      v[q] = one[0];
    }
    const uint32_t byte = scale_byte(quad_max(max_bits8(v)));
    const uint32_t c = encode8(v, byte);
    if (i < items) {
      const int64_t at = col * Q.ld_t + br;
      reinterpret_cast<uint32_t*>(Q.codes_t)[at * 4 + i % kLanesPerBlock] = c;
      if (i % kLanesPerBlock == 0) Q.scales_t[at] = static_cast<uint8_t>(byte);
    }
  }
}

// ------------------------------------------------------------------------
// Widen: 4-bit codes to fp32 / fp16 / bf16.
// ------------------------------------------------------------------------

// Eight codes as 16-bit values, rounded once from code * scale (exact in bf16;
// fp16 rounds to nearest even, overflows to infinity). NaN blocks give the
// canonical quiet NaN.
template <int DT>
__device__ __forceinline__ u4 widen8_16(uint32_t c, uint32_t byte) {
  const float s = scale_operand(byte);
  u4 w;
  if constexpr (DT == ZERO_DT_BF16) {
    w.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0));
    w.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1));
    w.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2));
    w.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3));
  } else {
    w.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 0));
    w.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 1));
    w.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 2));
    w.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 3));
  }
  if (byte == 255u) {
    const uint32_t q = DT == ZERO_DT_BF16 ? 0x7FC07FC0u : 0x7E007E00u;
    w = (u4){q, q, q, q};
  }
  return w;
}

template <int DT>
__global__ void __launch_bounds__(kBlock) mx_widen_kernel(const MxWidenArgs W) {
  const int64_t kb = (W.cols + kMxBlock - 1) / kMxBlock;
  const int64_t items = W.rows * kb * kLanesPerBlock;
  constexpr int64_t T = static_cast<int64_t>(kBlock) * kMxGroups;
  for (int64_t t0 = blockIdx.x * T; t0 < items; t0 += gridDim.x * T) {
#pragma unroll
    for (int k = 0; k < kMxGroups; ++k) {
      const int64_t i = t0 + k * kBlock + threadIdx.x;
      if (i >= items) continue;
      const int64_t b = i / kLanesPerBlock;
      const int64_t row = W.rows == 1 ? 0 : b / kb, bk = b - row * kb;
      const int64_t e = bk * kMxBlock + (i % kLanesPerBlock) * kLane;
      const int64_t at = row * W.ld + bk;
      const uint32_t c = reinterpret_cast<const uint32_t*>(W.codes)[at * 4 + i % kLanesPerBlock];
      const uint32_t byte = W.scales[at];
      const int64_t left = W.cols - e;
      if constexpr (DT == ZERO_DT_F32) {
        float v[8];
        decode8(c, scale_operand(byte), v);
        if (byte == 255u) {
#pragma unroll
          for (int q = 0; q < 8; ++q) v[q] = __uint_as_float(0x7FC00000u);
        }
        float* p = static_cast<float*>(W.out) + row * W.out_ld + e;
        if (left >= 8) {
          const f4 a = {v[0], v[1], v[2], v[3]}, d = {v[4], v[5], v[6], v[7]};
          __builtin_memcpy(p, &a, 16);
          __builtin_memcpy(p + 4, &d, 16);
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (q < left) p[q] = v[q];
        }
      } else {
        const u4 w = widen8_16<DT>(c, byte);
        uint16_t* p = static_cast<uint16_t*>(W.out) + row * W.out_ld + e;
        if (left >= 8) {
          __builtin_memcpy(p, &w, 16);
        } else {
          const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (q < left) p[q] = static_cast<uint16_t>(x[q / 2] >> (16 * (q & 1)));
        }
      }
    }
  }
}

// ------------------------------------------------------------------------
// Average of the N_d copies, and the norm / overflow partials of the unscaled
// gradient (as the 16-bit averaging pass).
// ------------------------------------------------------------------------

__global__ void __launch_bounds__(kBlock) mx_reduce_kernel(const MxReduceArgs R) {
  const float inv_scale = static_cast<float>(1.0 / static_cast<double>(R.state->loss_scale));
  double sumsq = 0.0;
  int bad = 0;
  const int64_t n = R.n;
  const int64_t items = (n + kLane - 1) / kLane;
  const MxCopies& S = R.src;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(kBlock) + threadIdx.x; i < items;
       i += static_cast<int64_t>(gridDim.x) * kBlock) {
    float acc[8] = {};
    for (int r = 0; r < S.n_d; ++r) {
      const uint8_t* codes = S.strided ? S.codes[0] + r * S.code_stride : S.codes[r];
      const uint8_t* scales = S.strided ? S.scales[0] + r * S.scale_stride : S.scales[r];
      float v[8];
      decode8(reinterpret_cast<const uint32_t*>(codes)[i], scale_operand(scales[i / kLanesPerBlock]), v);
#pragma unroll
      for (int q = 0; q < 8; ++q) acc[q] = acc[q] + v[q];
    }
    const int64_t e = i * kLane;
    const int64_t left = n - e;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if (q >= left) continue;
      const float a = S.n_d == 1 ? acc[q] : (S.inv_nd != 0.0f ? acc[q] * S.inv_nd : acc[q] / S.nd);
      account(a, a * inv_scale, sumsq, bad);
      R.avg_out[e + q] = a;
    }
  }
  write_block_partial(sumsq, bad, R.partials, R.fill);
}

int mx_grid(int64_t items, int64_t per_block) {
  int64_t b = (items + per_block - 1) / per_block;
  if (b < 1) b = 1;
  return limit_grid(static_cast<int>(b < kMaxGrid ? b : kMaxGrid));
}

template <int DT>
hipError_t quantize_launch(const MxQuantArgs& a, hipStream_t s) {
  if (a.codes) {
    MxQuantArgs q = a;
    if (q.cols % kMxBlock == 0 && q.src_ld == q.cols && q.ld == q.cols / kMxBlock) {
      q.cols *= q.rows;  // one long row
      q.rows = 1;
    }
    const int64_t items = q.rows * mx_blocks(q.cols) * kLanesPerBlock;
    hipLaunchKernelGGL((mx_quantize_rows_kernel<DT>), dim3(mx_grid(items, kBlock * kMxGroups)), dim3(kBlock), 0, s, q);
    if (hipError_t e = hipGetLastError()) return e;
  }
  if (a.codes_t) {
    const int64_t items = a.cols * mx_blocks(a.rows) * kLanesPerBlock;
    hipLaunchKernelGGL((mx_quantize_cols_kernel<DT>), dim3(mx_grid(items, kBlock)), dim3(kBlock), 0, s, a);
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_mx_quantize(const MxQuantArgs& a, int32_t src_dt, hipStream_t s) {
  if (src_dt == ZERO_DT_F32) return quantize_launch<ZERO_DT_F32>(a, s);
  if (src_dt == ZERO_DT_F16) return quantize_launch<ZERO_DT_F16>(a, s);
  if (src_dt == ZERO_DT_BF16) return quantize_launch<ZERO_DT_BF16>(a, s);
  return hipErrorInvalidValue;
}

hipError_t launch_mx_widen(const MxWidenArgs& args, int32_t dt, hipStream_t s) {
  MxWidenArgs a = args;
  if (a.cols % kMxBlock == 0 && a.out_ld == a.cols && a.ld == a.cols / kMxBlock) {
    a.cols *= a.rows;
    a.rows = 1;
  }
  const dim3 grid(mx_grid(a.rows * mx_blocks(a.cols) * kLanesPerBlock, kBlock * kMxGroups));
  if (dt == ZERO_DT_F32) hipLaunchKernelGGL(mx_widen_kernel<ZERO_DT_F32>, grid, dim3(kBlock), 0, s, a);
  else if (dt == ZERO_DT_F16) hipLaunchKernelGGL(mx_widen_kernel<ZERO_DT_F16>, grid, dim3(kBlock), 0, s, a);
  else if (dt == ZERO_DT_BF16) hipLaunchKernelGGL(mx_widen_kernel<ZERO_DT_BF16>, grid, dim3(kBlock), 0, s, a);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

hipError_t launch_mx_reduce(const MxReduceArgs& args, hipStream_t s, int* blocks) {
  const int grid = mx_grid((args.n + kLane - 1) / kLane, kBlock);
  const MxReduceArgs a = route_partials(args, grid, blocks);
  hipLaunchKernelGGL(mx_reduce_kernel, dim3(grid), dim3(kBlock), 0, s, a);
  return hipGetLastError();
}

}  // namespace zdp
