// gfx950 kernels that write and read the microscaled 4-bit format: quantise,
// widen, and the average of a shard's N_d copies.
//
// All three are streaming passes. A lane moves 16 bytes of the wide side at a
// time (4 fp32 or 8 16-bit values), next to its neighbours' 16 bytes, with the
// non-temporal hint: the lines are then whole in one access and leave the
// caches to the narrow side. (With 8 fp32 values a lane, two accesses to every
// other 16 bytes, widening 117M values to fp32 took 136 us instead of 75;
// plain stores cost the 16-bit side 55 us instead of 43.) Eight or four lanes
// share a block; its maximum is two or three lane permutes.
#include "mx_device.h"

namespace zdp {
namespace {

constexpr int kMxGroups = 4;  // of 16 bytes a lane has in flight

// 16 bytes of values at p, at any alignment of the type.
template <int DT>
__device__ __forceinline__ Raw<DT> load16(const void* p) {
  Raw<DT> x;
  const u4_any y = __builtin_nontemporal_load(static_cast<const u4_any*>(p));
  __builtin_memcpy(x.w, &y, sizeof x.w);
  return x;
}

// The same, of which only `left` values exist; the missing ones are 0.
template <int DT>
__device__ __forceinline__ Raw<DT> load16(const void* p, int64_t left) {
  Raw<DT> x = {};
  if (left >= Raw<DT>::kVals) {
    x = load16<DT>(p);
  } else if constexpr (DT == ZERO_DT_F32) {
    const uint32_t* f = static_cast<const uint32_t*>(p);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (q < left) x.w[q] = f[q];
  } else {
    const uint16_t* h = static_cast<const uint16_t*>(p);
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < left) x.w[q / 2] |= static_cast<uint32_t>(h[q]) << (16 * (q & 1));
  }
  return x;
}

// 16 bytes of values to p, as far as they exist.
template <int DT>
__device__ __forceinline__ void store16(void* p, u4 x, int64_t left) {
  if (left >= Raw<DT>::kVals) {
    __builtin_nontemporal_store(static_cast<u4_any>(x), static_cast<u4_any*>(p));
  } else {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    if constexpr (DT == ZERO_DT_F32) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (q < left) static_cast<uint32_t*>(p)[q] = w[q];
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < left) static_cast<uint16_t*>(p)[q] = static_cast<uint16_t>(w[q / 2] >> (16 * (q & 1)));
    }
  }
}

// ------------------------------------------------------------------------
// Quantise along the rows. Item i is part i % kLanes of block i / kLanes, blocks
// counted row by row. FLAT: one row (a shard, or a dense matrix of whole
// blocks); a full tile's loads are then all in flight before the first is used.
// Bound by HBM: 117M fp32 values 87 us (6.1 TB/s), bf16 47 (6.3). Rows that are
// not one after another or not whole blocks wait for each load in turn and
// divide per item: 8192 x 14336 inside a wider array 103 us in fp32, 58 in bf16;
// 8192 x 14335 93 and 54.
// ------------------------------------------------------------------------

template <int DT, bool FLAT>
__global__ void __launch_bounds__(kBlock) mx_quantize_rows_kernel(const MxQuantArgs Q) {
  using R = Raw<DT>;
  const int64_t kb = (Q.cols + kMxBlock - 1) / kMxBlock;
  const int64_t items = (FLAT ? 1 : Q.rows) * kb * R::kLanes;
  constexpr int64_t T = static_cast<int64_t>(kBlock) * kMxGroups;
  const int lane = threadIdx.x % R::kLanes;
  const char* const src = static_cast<const char*>(Q.src);
  auto put = [&](const R& x, int64_t at, bool there) {
    const uint32_t byte = scale_byte(lanes_max<R::kLanes>(max_bits<DT>(x.w, 4)));
    const uint32_t c = encode<DT>(x.w, byte);
    if (there) {
      reinterpret_cast<typename R::Codes*>(Q.codes)[at * R::kLanes + lane] = static_cast<typename R::Codes>(c);
      if (lane == 0) Q.scales[at] = static_cast<uint8_t>(byte);
    }
  };
  for (int64_t t0 = blockIdx.x * T; t0 < items; t0 += gridDim.x * T) {
    if (FLAT && (t0 + T) * R::kVals <= Q.cols) {
      R x[kMxGroups];
#pragma unroll
      for (int k = 0; k < kMxGroups; ++k) x[k] = load16<DT>(src + (t0 + k * kBlock + threadIdx.x) * 16);
#pragma unroll
      for (int k = 0; k < kMxGroups; ++k) put(x[k], (t0 + k * kBlock + threadIdx.x) / R::kLanes, true);
      continue;
    }
#pragma unroll
    for (int k = 0; k < kMxGroups; ++k) {
      const int64_t i = t0 + k * kBlock + threadIdx.x;
      const int64_t b = i / R::kLanes;
      const int64_t row = FLAT ? 0 : b / kb, bk = b - row * kb;
      const int64_t e = bk * kMxBlock + lane * R::kVals;
      put(load16<DT>(src + (row * Q.src_ld + e) * R::kElem, i < items ? Q.cols - e : 0), row * Q.ld + bk, i < items);
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
// Bound by HBM traffic in the pieces of 64 bytes that this tile makes (half lines
// of codes both ways: 135 MB written instead of 125; more rows a tile would make
// whole lines of the columns' codes): 8192 x 14336 bf16 74-78 us (4.6-4.8 TB/s)
// between other passes, 87 several in a row, fp32 125; 8192 x 14335 104 and 139.
// LDS holds rows of dwords (two 16-bit values or one fp32 value each); dword c
// of row i stands at c ^ 16 * (i / 32). A wave's column reads take 16
// neighbouring dwords of four rows that are 32 rows apart, and the permutation
// puts those four runs into different banks.
// ------------------------------------------------------------------------

constexpr int kSide = 128;                     // values of a tile, either way
// Every XCD works along strips of kStrip tile rows, column by column: the halves
// of a line of codes are then written soon after one another by the same L2,
// and the tiles in flight cover all channels. (Neighbouring tiles on different
// XCDs, in strips of columns: an XCD's tiles lay in few channels, and 8192 x
// 14336 took 99 us instead of 87.)
constexpr int kStrip = 4;

template <int DT>
__global__ void __launch_bounds__(kBlock) mx_quantize_tile_kernel(const MxQuantArgs Q) {
  using R = Raw<DT>;
  constexpr int kDwords = kSide * R::kElem / 4;  // of a row
  constexpr int kPer = 4 / R::kElem;             // columns in a dword
  constexpr int kSideLanes = kSide / R::kVals;   // lanes that read a row
  constexpr int kStep = kBlock / kSideLanes;     // rows of a pass
  constexpr int kPasses = kSide / kStep;
  __shared__ __align__(16) uint32_t tile[kSide * kDwords];
  const int64_t tr = (Q.rows + kSide - 1) / kSide, tc = (Q.cols + kSide - 1) / kSide;
  const int64_t tiles = tr * tc;
  const int tid = threadIdx.x;
  // The rows' blocks of a lane's kPasses rows (i0, i0 + kStep, ...) of the tile at r0, value column e.
  auto rows_out = [&](const R* v, int64_t r0, int i0, int64_t e) {
    uint32_t c[kPasses], byte[kPasses];
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      byte[p] = scale_byte(lanes_max<R::kLanes>(max_bits<DT>(v[p].w, 4)));
      c[p] = encode<DT>(v[p].w, byte[p]);
    }
    const bool there = e / kMxBlock * kMxBlock < Q.cols;
    if constexpr (R::kLanes == 4) {
      // the four lanes of a block take one of four rows' blocks each: whole
      // blocks and a fourth of the stores
      const int l = tid % 4;
#pragma unroll
      for (int p = 0; p < kPasses; p += 4) {
        quad_transpose(c + p, l);
        const uint32_t mine = l & 2 ? (l & 1 ? byte[p + 3] : byte[p + 2]) : (l & 1 ? byte[p + 1] : byte[p]);
        const int64_t row = r0 + i0 + (p + l) * kStep;
        if (there && row < Q.rows) {
          const int64_t b = row * Q.ld + e / kMxBlock;
          *reinterpret_cast<u4*>(Q.codes + b * kMxCodeBytes) = (u4){c[p], c[p + 1], c[p + 2], c[p + 3]};
          Q.scales[b] = static_cast<uint8_t>(mine);
        }
      }
    } else {
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        const int64_t row = r0 + i0 + p * kStep;
        if (there && row < Q.rows) {
          const int64_t b = row * Q.ld + e / kMxBlock;
          reinterpret_cast<typename R::Codes*>(Q.codes)[b * R::kLanes + tid % R::kLanes] =
              static_cast<typename R::Codes>(c[p]);
          if (tid % R::kLanes == 0) Q.scales[b] = static_cast<uint8_t>(byte[p]);
        }
      }
    }
  };
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    // block t runs on XCD t % 8: a run of tiles for every XCD
    const int64_t each = tiles / 8, more = tiles % 8, x = t % 8;
    const int64_t i = x * each + (x < more ? x : more) + t / 8;
    const int64_t strip = i / (tc * kStrip), at = i - strip * tc * kStrip;
    const int64_t high = tr - strip * kStrip < kStrip ? tr - strip * kStrip : kStrip;
    const int64_t r0 = (strip * kStrip + at % high) * kSide, c0 = at / high * kSide;
    const int x0 = tid % kSideLanes * R::kVals, i0 = tid / kSideLanes;
    const int64_t e = c0 + x0;
    const char* const src = static_cast<const char*>(Q.src) + ((r0 + i0) * Q.src_ld + e) * R::kElem;
    const int64_t down = Q.src_ld * R::kElem * kStep;  // bytes from pass to pass
    R v[kPasses];
    if (r0 + kSide <= Q.rows && c0 + kSide <= Q.cols) {
#pragma unroll
      for (int p = 0; p < kPasses; ++p) v[p] = load16<DT>(src + p * down);
    } else {
#pragma unroll
      for (int p = 0; p < kPasses; ++p)
        v[p] = load16<DT>(src + p * down, r0 + i0 + p * kStep < Q.rows ? Q.cols - e : 0);
    }
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int i = p * kStep + i0;
      *reinterpret_cast<u4*>(tile + i * kDwords + (x0 / kPer ^ (i / 32 * 16))) =
          (u4){v[p].w[0], v[p].w[1], v[p].w[2], v[p].w[3]};
    }
    if (Q.codes) rows_out(v, r0, i0, e);
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
        constexpr int kWords = kMxBlock * R::kElem / 4;
        uint32_t x[kWords];  // the column's 32 values
#pragma unroll
        for (int q = 0; q < kWords; ++q) {
          if constexpr (DT == ZERO_DT_F32) x[q] = w[q];
          else x[q] = __builtin_amdgcn_perm(w[2 * q + 1], w[2 * q], y ? 0x07060302u : 0x05040100u);
        }
        const uint32_t byte = scale_byte(max_bits<DT>(x, kWords));
        uint32_t c[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if constexpr (DT == ZERO_DT_F32) c[q] = encode<DT>(x + 8 * q, byte) | encode<DT>(x + 8 * q + 4, byte) << 16;
          else c[q] = encode<DT>(x + 4 * q, byte);
        }
        const int64_t col = c0 + d * kPer + y;
        if (col < Q.cols && r0 + rb * kMxBlock < Q.rows) {
          const int64_t b = col * Q.ld_t + r0 / kMxBlock + rb;
          *reinterpret_cast<u4*>(Q.codes_t + b * kMxCodeBytes) = (u4){c[0], c[1], c[2], c[3]};
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

// Raw<DT>::kVals codes times the scale of `byte`, rounded once to DT (exact in
// bf16 and fp32; fp16 rounds to nearest even, overflows to infinity). NaN blocks
// give the canonical quiet NaN.
template <int DT>
__device__ __forceinline__ u4 widen(uint32_t c, uint32_t byte) {
  const float s = scale_operand(byte);
  u4 w;
  if constexpr (DT == ZERO_DT_F32) {
    w = __builtin_bit_cast(u4, decode4(c, s));
  } else if constexpr (DT == ZERO_DT_BF16) {
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
    const uint32_t q = DT == ZERO_DT_F32 ? 0x7FC00000u : (DT == ZERO_DT_BF16 ? 0x7FC07FC0u : 0x7E007E00u);
    w = (u4){q, q, q, q};
  }
  return w;
}

// Bound by HBM: 117M values to bf16 43 us (6.9 TB/s), to fp32 75 (7.1). Not FLAT:
// 8192 x 14336 into a wider array 51 and 92, 8192 x 14335 (rows off 16 bytes) 57
// and 111.
template <int DT, bool FLAT>
__global__ void __launch_bounds__(kBlock) mx_widen_kernel(const MxWidenArgs W) {
  using R = Raw<DT>;
  const int64_t kb = (W.cols + kMxBlock - 1) / kMxBlock;
  const int64_t items = (FLAT ? 1 : W.rows) * kb * R::kLanes;
  constexpr int64_t T = static_cast<int64_t>(kBlock) * kMxGroups;
  const int lane = threadIdx.x % R::kLanes;
  const typename R::Codes* const codes = reinterpret_cast<const typename R::Codes*>(W.codes);
  char* const out = static_cast<char*>(W.out);
  for (int64_t t0 = blockIdx.x * T; t0 < items; t0 += gridDim.x * T) {
    if (FLAT && (t0 + T) * R::kVals <= W.cols) {
      uint32_t c[kMxGroups], byte[kMxGroups];
#pragma unroll
      for (int k = 0; k < kMxGroups; ++k) {
        const int64_t i = t0 + k * kBlock + threadIdx.x;
        c[k] = codes[i];
        byte[k] = W.scales[i / R::kLanes];
      }
#pragma unroll
      for (int k = 0; k < kMxGroups; ++k)
        store16<DT>(out + (t0 + k * kBlock + threadIdx.x) * 16, widen<DT>(c[k], byte[k]), R::kVals);
      continue;
    }
#pragma unroll
    for (int k = 0; k < kMxGroups; ++k) {
      const int64_t i = t0 + k * kBlock + threadIdx.x;
      if (i >= items) continue;
      const int64_t b = i / R::kLanes;
      const int64_t row = FLAT ? 0 : b / kb, bk = b - row * kb;
      const int64_t e = bk * kMxBlock + lane * R::kVals;
      const int64_t at = row * W.ld + bk;
      store16<DT>(out + (row * W.out_ld + e) * R::kElem, widen<DT>(codes[at * R::kLanes + lane], W.scales[at]),
                  W.cols - e);
    }
  }
}

// ------------------------------------------------------------------------
// Average of the N_d copies, and the norm / overflow partials of the unscaled
// gradient (as the 16-bit averaging pass). A lane takes quads of values, the
// loads of up to eight copies of all its quads in flight at once; the additions
// stay in the copies' order. Bound by HBM: 8 copies of 117M values 161 us (6.0
// TB/s); with 2 quads a lane or 4 copies at a time 166-170, codes without the
// non-temporal hint 168. Other counts of the same shard: 2 copies 131, 9 220, 16
// 270 (5.4 TB/s), 64 1041, 65 (equally spaced) 1053 (4.3), 100 1701 (3.9).
// ------------------------------------------------------------------------

constexpr int kReduceQuads = 4;
constexpr int kReduceCopies = 8;
constexpr int kQuadLanes = kMxBlock / 4;

template <int N>
__device__ __forceinline__ void add_copies(const MxCopies& S, int r, const int64_t at[kReduceQuads], f4 acc[kReduceQuads]) {
  uint32_t c[N][kReduceQuads], e[N][kReduceQuads];
#pragma unroll
  for (int q = 0; q < N; ++q) {
    const uint8_t* codes = S.strided ? S.codes[0] + (r + q) * S.code_stride : S.codes[r + q];
    const uint8_t* scales = S.strided ? S.scales[0] + (r + q) * S.scale_stride : S.scales[r + q];
#pragma unroll
    for (int k = 0; k < kReduceQuads; ++k) {
      c[q][k] = ld_stream(reinterpret_cast<const uint16_t*>(codes) + at[k]);
      e[q][k] = scales[at[k] / kQuadLanes];
    }
  }
#pragma unroll
  for (int q = 0; q < N; ++q)
#pragma unroll
    for (int k = 0; k < kReduceQuads; ++k) acc[k] = acc[k] + decode4(c[q][k], scale_operand(e[q][k]));
}

__global__ void __launch_bounds__(kBlock) mx_reduce_kernel(const MxReduceArgs R) {
  const float inv_scale = static_cast<float>(1.0 / static_cast<double>(R.state->loss_scale));
  double sumsq = 0.0;
  int bad = 0;
  const int64_t n = R.n;
  const int64_t items = (n + 3) / 4;
  const MxCopies& S = R.src;
  constexpr int64_t T = static_cast<int64_t>(kBlock) * kReduceQuads;
  for (int64_t t0 = blockIdx.x * T; t0 < items; t0 += gridDim.x * T) {
    f4 acc[kReduceQuads] = {};
    int64_t at[kReduceQuads];  // past the end: the last item again
#pragma unroll
    for (int k = 0; k < kReduceQuads; ++k) {
      const int64_t i = t0 + k * kBlock + threadIdx.x;
      at[k] = i < items ? i : items - 1;
    }
    int r = 0;
    for (; r + kReduceCopies <= S.n_d; r += kReduceCopies) add_copies<kReduceCopies>(S, r, at, acc);
    if (r + 4 <= S.n_d) { add_copies<4>(S, r, at, acc); r += 4; }
    if (r + 2 <= S.n_d) { add_copies<2>(S, r, at, acc); r += 2; }
    if (r < S.n_d) add_copies<1>(S, r, at, acc);
#pragma unroll
    for (int k = 0; k < kReduceQuads; ++k) {
      const int64_t e = (t0 + k * kBlock + threadIdx.x) * 4;
      const int64_t left = n - e;
      f4 a = acc[k];
      if (S.n_d > 1) a = S.inv_nd != 0.0f ? a * S.inv_nd : a / S.nd;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (q < left) account(a[q], a[q] * inv_scale, sumsq, bad);
      store16<ZERO_DT_F32>(R.avg_out + e, __builtin_bit_cast(u4, a), left);
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
  const int64_t items = q.rows * mx_blocks(q.cols) * Raw<DT>::kLanes;
  const dim3 grid(mx_grid(items, kBlock * kMxGroups));
  if (q.rows == 1) hipLaunchKernelGGL((mx_quantize_rows_kernel<DT, true>), grid, dim3(kBlock), 0, s, q);
  else hipLaunchKernelGGL((mx_quantize_rows_kernel<DT, false>), grid, dim3(kBlock), 0, s, q);
  return hipGetLastError();
}

template <int DT>
hipError_t widen_launch(const MxWidenArgs& args, hipStream_t s) {
  MxWidenArgs a = args;
  if (a.cols % kMxBlock == 0 && a.out_ld == a.cols && a.ld == a.cols / kMxBlock) {
    a.cols *= a.rows;  // one long row
    a.rows = 1;
  }
  const dim3 grid(mx_grid(a.rows * mx_blocks(a.cols) * Raw<DT>::kLanes, kBlock * kMxGroups));
  if (a.rows == 1) hipLaunchKernelGGL((mx_widen_kernel<DT, true>), grid, dim3(kBlock), 0, s, a);
  else hipLaunchKernelGGL((mx_widen_kernel<DT, false>), grid, dim3(kBlock), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_quantize(const MxQuantArgs& a, int32_t src_dt, hipStream_t s) {
  if (src_dt == ZERO_DT_F32) return quantize_launch<ZERO_DT_F32>(a, s);
  if (src_dt == ZERO_DT_F16) return quantize_launch<ZERO_DT_F16>(a, s);
  if (src_dt == ZERO_DT_BF16) return quantize_launch<ZERO_DT_BF16>(a, s);
  return hipErrorInvalidValue;
}

hipError_t launch_mx_widen(const MxWidenArgs& a, int32_t dt, hipStream_t s) {
  if (dt == ZERO_DT_F32) return widen_launch<ZERO_DT_F32>(a, s);
  if (dt == ZERO_DT_F16) return widen_launch<ZERO_DT_F16>(a, s);
  if (dt == ZERO_DT_BF16) return widen_launch<ZERO_DT_BF16>(a, s);
  return hipErrorInvalidValue;
}

hipError_t launch_mx_reduce(const MxReduceArgs& args, hipStream_t s, int* blocks) {
  const int grid = mx_grid((args.n + 3) / 4, kBlock * kReduceQuads);
  const MxReduceArgs a = route_partials(args, grid, blocks);
  hipLaunchKernelGGL(mx_reduce_kernel, dim3(grid), dim3(kBlock), 0, s, a);
  return hipGetLastError();
}

}  // namespace zdp
