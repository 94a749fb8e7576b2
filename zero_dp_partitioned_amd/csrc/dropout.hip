// gfx950 kernel of dropout from a counter-based generator,
//   y = (keep ? x * 1 / (1 - p) : 0) + residual,
// whose mask is a function of (seed, offset, element) and is never stored:
// word i % 4 of Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", 2011) with the counter (i / 4, offset) and the
// key `seed` decides element i.
#include "layer_device.h"

namespace zdp {
namespace {

constexpr int kSlots = 2;  // 16-byte slots a lane handles, all loads first (four took 3 % more time at 16384 x 4096 bf16, one 1 %)
// Tensors from 64 MiB on are read with the non-temporal hint (16384 x 4096 bf16
// with a residual: 75 -> 71 us; 8192 x 1600 fp16, which the caches hold: 17.1 -> 18.2).
constexpr int64_t kOnceSlots = (64 << 20) / 16;

__device__ __forceinline__ u4 philox(uint64_t block, uint64_t offset, uint64_t seed) {
  uint32_t c0 = static_cast<uint32_t>(block), c1 = static_cast<uint32_t>(block >> 32);
  uint32_t c2 = static_cast<uint32_t>(offset), c3 = static_cast<uint32_t>(offset >> 32);
  uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = static_cast<uint64_t>(c0) * 0xD2511F53u, b = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
    c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
    c1 = static_cast<uint32_t>(b);
    c3 = static_cast<uint32_t>(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return (u4){c0, c1, c2, c3};
}

// A slot is 16 bytes of a row, and starts on a block of the generator: with an
// index off a multiple of four it is the memory accesses that are off 16 bytes
// (which costs them a line in nine), not the generator that runs twice. Bound by
// HBM with a residual (16384 x 4096 bf16: 67 us, 6.0 TB/s); without one the
// generator's 20 32-bit products for four values come into reach of it (55 us, 4.9
// TB/s).
template <int DT, bool RESIDUAL, bool ONCE>
__global__ void __launch_bounds__(256) dropout_kernel(const DropoutArgs D, int64_t row_slots, int64_t slots) {
  constexpr int kVals = Vec<DT>::kVals, kElem = Vec<DT>::kElem;
  uint64_t offset = D.offset;
  if (D.counter) offset += static_cast<uint64_t>(*D.counter);
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256 * kSlots;
  for (int64_t s0 = static_cast<int64_t>(blockIdx.x) * 256 * kSlots + threadIdx.x; s0 < slots; s0 += step) {
    int64_t row[kSlots], col[kSlots];
    u4 x[kSlots], r[kSlots];
#pragma unroll
    for (int q = 0; q < kSlots; ++q) {
      const int64_t s = s0 + q * 256;
      row[q] = 0;
      int64_t at = s;
      if (D.rows > 1) {
        row[q] = s / row_slots;
        at = s - row[q] * row_slots;
      }
      // the slot's first column; a row's first slot may begin before it
      const int lead = static_cast<int>((D.first + static_cast<uint64_t>(row[q]) * D.cols) & 3);
      col[q] = at * kVals - lead;
      x[q] = r[q] = (u4){0, 0, 0, 0};
      if (s >= slots) col[q] = D.cols;
      if (col[q] < 0 || col[q] >= D.cols) continue;
      x[q] = load_part<DT, ONCE>(static_cast<const char*>(D.x.p) + (row[q] * D.x.ld + col[q]) * kElem, D.cols - col[q]);
      if constexpr (RESIDUAL)
        r[q] = load_part<DT, ONCE>(static_cast<const char*>(D.residual.p) + (row[q] * D.residual.ld + col[q]) * kElem,
                             D.cols - col[q]);
    }
#pragma unroll
    for (int q = 0; q < kSlots; ++q) {
      if (col[q] >= D.cols) continue;
      const uint64_t index = D.first + static_cast<uint64_t>(row[q] * D.cols + col[q]);  // a multiple of four
      float v[kVals], b[kVals];
      if (col[q] < 0) {  // the part of a row's first slot that exists
#pragma unroll
        for (int e = 0; e < kVals; ++e) {
          const int64_t c = col[q] + e;
          v[e] = c >= 0 && c < D.cols ? load_one(D.x.p, row[q] * D.x.ld + c, DT) : 0.f;
          b[e] = RESIDUAL && c >= 0 && c < D.cols ? load_one(D.residual.p, row[q] * D.residual.ld + c, DT) : 0.f;
        }
      } else {
        widen<DT>(x[q], v);
        widen<DT>(r[q], b);
      }
      if (D.threshold) {
#pragma unroll
        for (int g = 0; g < kVals / 4; ++g) {
          const u4 w = philox((index >> 2) + g, offset, D.seed);
          const uint32_t word[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) v[4 * g + e] = word[e] >= D.threshold ? v[4 * g + e] * D.scale : 0.f;
        }
      }
      if constexpr (RESIDUAL) {
#pragma unroll
        for (int e = 0; e < kVals; ++e) v[e] += b[e];
      }
      if (col[q] < 0) {
#pragma unroll
        for (int e = 0; e < kVals; ++e)
          if (col[q] + e >= 0 && col[q] + e < D.cols) store_one(D.y.p, row[q] * D.y.ld + col[q] + e, DT, v[e]);
      } else {
        store_part<DT>(static_cast<char*>(D.y.p) + (row[q] * D.y.ld + col[q]) * kElem, D.cols - col[q], narrow<DT>(v));
      }
    }
  }
}

template <int DT>
hipError_t dropout_launch(DropoutArgs a, hipStream_t s) {
  if (a.rows > 1 && a.x.ld == a.cols && a.y.ld == a.cols && (!a.residual.p || a.residual.ld == a.cols)) {
    a.cols *= a.rows;  // one row
    a.rows = 1;
  }
  // slots of a row, the generator's blocks in front of it counted
  const int64_t lead = a.rows > 1 ? 3 : static_cast<int64_t>(a.first & 3);
  const int64_t row_slots = ceil_div(a.cols + lead, Vec<DT>::kVals), slots = row_slots * a.rows;
  const int64_t blocks = ceil_div(slots, 256 * kSlots);
  const int grid = limit_grid(static_cast<int>(blocks < kMaxGrid ? blocks : kMaxGrid));
  const auto kernel = slots >= kOnceSlots ? (a.residual.p ? dropout_kernel<DT, true, true> : dropout_kernel<DT, false, true>)
                                          : (a.residual.p ? dropout_kernel<DT, true, false> : dropout_kernel<DT, false, false>);
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(256), 0, s, a, row_slots, slots);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(const DropoutArgs& a, int32_t dt, hipStream_t s) {
  if (dt == ZERO_DT_F32) return dropout_launch<ZERO_DT_F32>(a, s);
  if (dt == ZERO_DT_F16) return dropout_launch<ZERO_DT_F16>(a, s);
  if (dt == ZERO_DT_BF16) return dropout_launch<ZERO_DT_BF16>(a, s);
  return hipErrorInvalidValue;
}

}  // namespace zdp
