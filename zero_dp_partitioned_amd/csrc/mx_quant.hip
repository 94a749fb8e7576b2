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

// The eight values at p, at any alignment of the type, of which `left` exist; the missing ones are 0.
template <int DT>
__device__ __forceinline__ Raw8<DT> load8(const void* p, int64_t left) {
  Raw8<DT> x = {};
  if (left >= 8) {
    __builtin_memcpy(x.w, p, sizeof x.w);
  } else if constexpr (DT == ZERO_DT_F32) {
    const uint32_t* f = static_cast<const uint32_t*>(p);
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < left) x.w[q] = f[q];
  } else {
    const uint16_t* h = static_cast<const uint16_t*>(p);
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < left) x.w[q / 2] |= static_cast<uint32_t>(h[q]) << (16 * (q & 1));
  }
  return x;
}

// ------------------------------------------------------------------------
// Quantise along the rows. Item i is quarter i % 4 of block i / 4, blocks
// counted row by row. FLAT: one row (a shard, or a dense matrix of whole
// blocks); a full tile's loads are then all in flight before the first is used,
// which takes 117M fp32 values from FLAT_BEFORE to FLAT_AFTER us.
// ------------------------------------------------------------------------

template <int DT, bool FLAT>
__global__ void __launch_bounds__(kBlock) mx_quantize_rows_kernel(const MxQuantArgs Q) {
  constexpr int kElem = DT == ZERO_DT_F32 ? 4 : 2;
  const int64_t kb = (Q.cols + kMxBlock - 1) / kMxBlock;
  const int64_t items = (FLAT ? 1 : Q.rows) * kb * kLanesPerBlock;
  constexpr int64_t T = static_cast<int64_t>(kBlock) * kMxGroups;
  const int lane = threadIdx.x % kLanesPerBlock;
  const char* const src = static_cast<const char*>(Q.src);
  auto put = [&](const Raw8<DT>& x, int64_t at, bool there) {
    const uint32_t byte = scale_byte(quad_max(max_bits<DT>(x.w, Raw8<DT>::kWords)));
    const uint32_t c = encode8<DT>(x.w, byte);
    if (there) {
      st_stream(reinterpret_cast<uint32_t*>(Q.codes) + at * 4 + lane, c);
      if (lane == 0) Q.scales[at] = static_cast<uint8_t>(byte);
    }
  };
  for (int64_t t0 = blockIdx.x * T; t0 < items; t0 += gridDim.x * T) {
    if (FLAT && (t0 + T) * kLane <= Q.cols) {
      Raw8<DT> x[kMxGroups];
#pragma unroll
      for (int k = 0; k < kMxGroups; ++k) {
        const char* const p = src + (t0 + k * kBlock + threadIdx.x) * kLane * kElem;
        __builtin_memcpy(x[k].w, p, sizeof x[k].w);
      }
#pragma unroll
      for (int k = 0; k < kMxGroups; ++k) put(x[k], (t0 + k * kBlock + threadIdx.x) / kLanesPerBlock, true);
      continue;
    }
#pragma unroll
    for (int k = 0; k < kMxGroups; ++k) {
      const int64_t i = t0 + k * kBlock + threadIdx.x;
      const int64_t b = i / kLanesPerBlock;
      const int64_t row = FLAT ? 0 : b / kb, bk = b - row * kb;
      const int64_t e = bk * kMxBlock + lane * kLane;
      put(load8<DT>(src + (row * Q.src_ld + e) * kElem, i < items ? Q.cols - e : 0), row * Q.ld + bk, i < items);
    }
  }
}

// ------------------------------------------------------------------------
// Quantise along the columns (the transpose's rows) and, if wanted, along the
// rows from the same read. A block takes a tile of 128 x 128 values: it reads
// them row by row as the row kernel does (and quantises the rows), keeps them
// in LDS in their own type, and then takes every column's four blocks of 32
// from there. 128 values either way make a tile's codes 64 contiguous bytes of
// every row and of every column.
// LDS holds rows of dwords (two 16-bit values or one fp32 value each); dword c
// of row i stands at c ^ 16 * (i / 32). A wave's column reads take 16
// neighbouring dwords of four rows that are 32 rows apart, and the permutation
// puts those four runs into different banks.
// ------------------------------------------------------------------------

constexpr int kSide = 128;                     // values of a tile, either way
constexpr int kSideLanes = kSide / kLane;      // lanes that read a row
constexpr int kPasses = kSide / (kBlock / kSideLanes);
constexpr int kStrip = 4;                      // tiles next to each other that are worked on in turn

template <int DT>
__global__ void __launch_bounds__(kBlock) mx_quantize_tile_kernel(const MxQuantArgs Q) {
  constexpr int kElem = DT == ZERO_DT_F32 ? 4 : 2;
  constexpr int kDwords = kSide * kElem / 4;  // of a row
  constexpr int kPer = 4 / kElem;             // columns in a dword
  __shared__ __align__(16) uint32_t tile[kSide * kDwords];
  const int64_t tr = (Q.rows + kSide - 1) / kSide, tc = (Q.cols + kSide - 1) / kSide;
  const int64_t tiles = tr * tc;
  const int tid = threadIdx.x;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    // strips of kStrip tile columns, row by row: the halves of a line of codes
    // and the pieces of a line of scales are written soon after one another
    const int64_t strip = t / (tr * kStrip), at = t - strip * tr * kStrip;
    const int64_t wide = tc - strip * kStrip < kStrip ? tc - strip * kStrip : kStrip;
    const int64_t r0 = at / wide * kSide, c0 = (strip * kStrip + at % wide) * kSide;
    const int64_t e = c0 + (tid % kSideLanes) * kLane;
    const int i0 = tid / kSideLanes;
    const char* const src = static_cast<const char*>(Q.src) + ((r0 + i0) * Q.src_ld + e) * kElem;
    const int64_t down = Q.src_ld * kElem * (kBlock / kSideLanes);  // bytes from pass to pass
    Raw8<DT> v[kPasses];
    if (r0 + kSide <= Q.rows && c0 + kSide <= Q.cols) {
#pragma unroll
      for (int p = 0; p < kPasses; ++p) __builtin_memcpy(v[p].w, src + p * down, sizeof v[p].w);
    } else {
#pragma unroll
      for (int p = 0; p < kPasses; ++p)
        v[p] = load8<DT>(src + p * down, r0 + i0 + p * (kBlock / kSideLanes) < Q.rows ? Q.cols - e : 0);
    }
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int i = p * (kBlock / kSideLanes) + i0;
      uint32_t* const to = tile + i * kDwords;
      const int first = (tid % kSideLanes) * kLane / kPer;
#pragma unroll
      for (int h = 0; h < Raw8<DT>::kWords / 4; ++h)
        *reinterpret_cast<u4*>(to + ((first + 4 * h) ^ (i / 32 * 16))) =
            (u4){v[p].w[4 * h], v[p].w[4 * h + 1], v[p].w[4 * h + 2], v[p].w[4 * h + 3]};
      if (Q.codes) {
        const uint32_t byte = scale_byte(quad_max(max_bits<DT>(v[p].w, Raw8<DT>::kWords)));
        const uint32_t c = encode8<DT>(v[p].w, byte);
        if (r0 + i < Q.rows && e / kMxBlock * kMxBlock < Q.cols) {
          const int64_t b = (r0 + i) * Q.ld + e / kMxBlock;
          reinterpret_cast<uint32_t*>(Q.codes)[b * 4 + tid % 4] = c;
          if (tid % 4 == 0) Q.scales[b] = static_cast<uint8_t>(byte);
        }
      }
    }
    __syncthreads();
    const int rb = tid % 4;  // the column's block of 32
#pragma unroll
    for (int h = 0; h < 2 / kPer; ++h) {
      const int d = h * 64 + tid / 4;  // the dword: kPer columns
      uint32_t w[kMxBlock];
#pragma unroll
      for (int q = 0; q < kMxBlock; ++q) w[q] = tile[(rb * kMxBlock + q) * kDwords + (d ^ (rb * 16))];
#pragma unroll
      for (int y = 0; y < kPer; ++y) {
        uint32_t x[4 * Raw8<DT>::kWords];  // the column's 32 values
#pragma unroll
        for (int q = 0; q < 4 * Raw8<DT>::kWords; ++q) {
          if constexpr (DT == ZERO_DT_F32) x[q] = w[q];
          else x[q] = __builtin_amdgcn_perm(w[2 * q + 1], w[2 * q], y ? 0x07060302u : 0x05040100u);
        }
        constexpr int K = Raw8<DT>::kWords;
        const uint32_t byte = scale_byte(max_bits<DT>(x, 4 * K));
        const u4 c = {encode8<DT>(x, byte), encode8<DT>(x + K, byte), encode8<DT>(x + 2 * K, byte),
                      encode8<DT>(x + 3 * K, byte)};
        const int64_t col = c0 + d * kPer + y;
        if (col < Q.cols && r0 + rb * kMxBlock < Q.rows) {
          const int64_t b = col * Q.ld_t + r0 / kMxBlock + rb;
          *reinterpret_cast<u4*>(Q.codes_t + b * kMxCodeBytes) = c;
          Q.scales_t[b] = static_cast<uint8_t>(byte);
        }
      }
    }
    __syncthreads();
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

// Groups of 8 values a lane has in flight, and copies whose loads it issues at
// a time (the additions stay in the copies' order).
constexpr int kReduceGroups = 2;
constexpr int kReduceCopies = 8;

template <int N>
__device__ __forceinline__ void add_copies(const MxCopies& S, int r, const int64_t at[kReduceGroups],
                                           float acc[kReduceGroups][8]) {
  uint32_t c[N][kReduceGroups], e[N][kReduceGroups];
#pragma unroll
  for (int q = 0; q < N; ++q) {
    const uint8_t* codes = S.strided ? S.codes[0] + (r + q) * S.code_stride : S.codes[r + q];
    const uint8_t* scales = S.strided ? S.scales[0] + (r + q) * S.scale_stride : S.scales[r + q];
#pragma unroll
    for (int k = 0; k < kReduceGroups; ++k) {
      c[q][k] = ld_stream(reinterpret_cast<const uint32_t*>(codes) + at[k]);
      e[q][k] = scales[at[k] / kLanesPerBlock];
    }
  }
#pragma unroll
  for (int q = 0; q < N; ++q)
#pragma unroll
    for (int k = 0; k < kReduceGroups; ++k) {
      float v[8];
      decode8(c[q][k], scale_operand(e[q][k]), v);
#pragma unroll
      for (int x = 0; x < 8; ++x) acc[k][x] = acc[k][x] + v[x];
    }
}

__global__ void __launch_bounds__(kBlock) mx_reduce_kernel(const MxReduceArgs R) {
  const float inv_scale = static_cast<float>(1.0 / static_cast<double>(R.state->loss_scale));
  double sumsq = 0.0;
  int bad = 0;
  const int64_t n = R.n;
  const int64_t items = (n + kLane - 1) / kLane;
  const MxCopies& S = R.src;
  constexpr int64_t T = static_cast<int64_t>(kBlock) * kReduceGroups;
  for (int64_t t0 = blockIdx.x * T; t0 < items; t0 += gridDim.x * T) {
    float acc[kReduceGroups][8] = {};
    int64_t at[kReduceGroups];  // past the end: the last item again
#pragma unroll
    for (int k = 0; k < kReduceGroups; ++k) {
      const int64_t i = t0 + k * kBlock + threadIdx.x;
      at[k] = i < items ? i : items - 1;
    }
    int r = 0;
    for (; r + kReduceCopies <= S.n_d; r += kReduceCopies) add_copies<kReduceCopies>(S, r, at, acc);
    if (r + 4 <= S.n_d) { add_copies<4>(S, r, at, acc); r += 4; }
    if (r + 2 <= S.n_d) { add_copies<2>(S, r, at, acc); r += 2; }
    if (r < S.n_d) add_copies<1>(S, r, at, acc);
#pragma unroll
    for (int k = 0; k < kReduceGroups; ++k) {
      const int64_t e = (t0 + k * kBlock + threadIdx.x) * kLane;
      const int64_t left = n - e;
      float a[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        a[q] = S.n_d == 1 ? acc[k][q] : (S.inv_nd != 0.0f ? acc[k][q] * S.inv_nd : acc[k][q] / S.nd);
        if (q < left) account(a[q], a[q] * inv_scale, sumsq, bad);
      }
      float* const p = R.avg_out + e;
      if (left >= 8) {
        const f4 x = {a[0], a[1], a[2], a[3]}, y = {a[4], a[5], a[6], a[7]};
        __builtin_memcpy(p, &x, 16);
        __builtin_memcpy(p + 4, &y, 16);
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (q < left) p[q] = a[q];
      }
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
  if (a.codes_t) {
    const int64_t tiles = mx_tiles(a.rows, kSide) * mx_tiles(a.cols, kSide);
    hipLaunchKernelGGL((mx_quantize_tile_kernel<DT>), dim3(mx_grid(tiles, 1)), dim3(kBlock), 0, s, a);
    return hipGetLastError();
  }
  MxQuantArgs q = a;
  if (q.cols % kMxBlock == 0 && q.src_ld == q.cols && q.ld == q.cols / kMxBlock) {
    q.cols *= q.rows;  // one long row
    q.rows = 1;
  }
  const int64_t items = q.rows * mx_blocks(q.cols) * kLanesPerBlock;
  const dim3 grid(mx_grid(items, kBlock * kMxGroups));
  if (q.rows == 1) hipLaunchKernelGGL((mx_quantize_rows_kernel<DT, true>), grid, dim3(kBlock), 0, s, q);
  else hipLaunchKernelGGL((mx_quantize_rows_kernel<DT, false>), grid, dim3(kBlock), 0, s, q);
  return hipGetLastError();
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
  const int grid = mx_grid((args.n + kLane - 1) / kLane, kBlock * kReduceGroups);
  const MxReduceArgs a = route_partials(args, grid, blocks);
  hipLaunchKernelGGL(mx_reduce_kernel, dim3(grid), dim3(kBlock), 0, s, a);
  return hipGetLastError();
}

}  // namespace zdp
