// gfx950 kernels of layer norm over the rows of a matrix,
//   y = (x - mean) * rstd * w + b,   rstd = 1 / sqrt(var + eps),
// and of its backward pass, with xhat = (x - mean) * rstd and v = dy * w:
//   dx = rstd * (v - mean(v) - xhat * mean(v xhat)) + dresidual,
//   dw = sum over rows of dy xhat,   db = sum over rows of dy.
// Both are streaming passes bound by HBM: a row stays in registers between its
// sums and its results, so that every value is read and written once. Sums,
// statistics and the column sums are fp32; results are rounded once.
#include <type_traits>

#include "layer_device.h"

namespace zdp {
namespace {

// The sum over a wave's 64 lanes, in every lane.
__device__ __forceinline__ float wave_sum(float x) {
  auto add = [&](auto ctrl, auto rows) {
    x += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), decltype(ctrl)::value,
                                                               decltype(rows)::value, 0xF, false));
  };
  using std::integral_constant;
  add(integral_constant<int, 0xB1>{}, integral_constant<int, 0xF>{});   // lanes 1,0,3,2
  add(integral_constant<int, 0x4E>{}, integral_constant<int, 0xF>{});   // lanes 2,3,0,1
  add(integral_constant<int, 0x141>{}, integral_constant<int, 0xF>{});  // 8 lanes mirrored
  add(integral_constant<int, 0x140>{}, integral_constant<int, 0xF>{});  // 16 lanes mirrored
  add(integral_constant<int, 0x142>{}, integral_constant<int, 0xA>{});  // lanes 15 and 47 into the next 16
  add(integral_constant<int, 0x143>{}, integral_constant<int, 0xC>{});  // lane 31 into the upper 32
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 63));
}

// The sum over the W waves of a row, of which this is wave w; in wave order.
// `part` holds W floats and is free again after the next barrier but one.
template <int W>
__device__ __forceinline__ float row_sum(float x, float* part, int w, int lane) {
  x = wave_sum(x);
  if constexpr (W > 1) {
    if (lane == 0) part[w] = x;
    __syncthreads();
    x = 0.f;
#pragma unroll
    for (int q = 0; q < W; ++q) x += part[q];
  }
  return x;
}

// A row's sums may pass fp32's range though its values do not. Its mean is summed
// from values times a power of two below 1 / cols, which changes no bit of it (but for
// values under 2^-126 times cols, by less than 2^-148 times cols). Its squares are
// summed as they are and, if that sum is not finite, once more from distances times
// kFar; every wave of a row does that or none does. If they pass the range then too,
// the row is NaN.
constexpr float kFar = 0x1p-76f;  // 2^20 squares of values below 2^128

__device__ __forceinline__ float rstd_of_far(float sq, float inv, float eps) {
  return 1.0f / sqrtf(sq * inv + eps * kFar * kFar) * kFar + (sq - sq);  // NaN for infinity
}

// Vec<DT>::kVals values of the weight (or bias), of x's type or fp32, from column `col` on.
template <int DT>
__device__ __forceinline__ void load_weight(const void* p, int32_t w_dt, int col, float* v) {
  if (DT != ZERO_DT_F32 && w_dt == ZERO_DT_F32) {
    const float* const q = static_cast<const float*>(p) + col;
    widen<ZERO_DT_F32>(load_any(q), v);
    widen<ZERO_DT_F32>(load_any(q + 4), v + 4);
  } else {
    widen<DT>(load_any(static_cast<const char*>(p) + static_cast<int64_t>(col) * Vec<DT>::kElem), v);
  }
}

// The same as far as there are columns, the rest 0.
template <int DT>
__device__ __forceinline__ void load_weight_part(const void* p, int32_t w_dt, int col, int cols, float* v) {
  for (int e = 0; e < Vec<DT>::kVals; ++e) v[e] = col + e < cols ? load_one(p, col + e, w_dt) : 0.f;
}

// A lane's slot j of a row that a group of W waves holds: 16 bytes from column
// `at` on. The slot that would pass the row's end is moved back to end with it,
// so that all loads are whole and no branch stands around them; its first
// `skip` values are the slot's before (all of them where the row needs no slot).
template <int DT, int W>
struct Slot {
  int at, skip;
  __device__ __forceinline__ Slot(int j, int w, int lane, int cols) {
    const int col = ((j * W + w) * 64 + lane) * Vec<DT>::kVals;
    at = col < cols - Vec<DT>::kVals ? col : cols - Vec<DT>::kVals;
    skip = col - at;
  }
  __device__ __forceinline__ u4 load(const char* row) const { return load_any(row + at * Vec<DT>::kElem); }
  __device__ __forceinline__ u4 load_once(const char* row) const { return zdp::load_once(row + at * Vec<DT>::kElem); }
  __device__ __forceinline__ void store(char* row, u4 x) const {
    char* const p = row + at * Vec<DT>::kElem;
    if (skip == 0) store_once(p, x);
    else store_some<DT>(p, skip, Vec<DT>::kVals, x);
  }
};

// W waves a row, V 16-byte slots a lane; a block of one wave a row has four
// rows. At least Vec<DT>::kVals columns. Measured: 16384 x 4096 bf16 50 us (5.4
// TB/s), 8192 x 1600 fp16 12.5 (4.2), one row of 4096 3.0 in a graph. The output
// goes past the caches, the input does not: with the hint on both the first took 1 %
// more and the second, which the caches hold, 4 %.
template <int DT, int V, int W>
__global__ void __launch_bounds__(W == 1 ? 256 : 64 * W) norm_kernel(const NormArgs N) {
  constexpr int kVals = Vec<DT>::kVals, kElem = Vec<DT>::kElem, kRows = W == 1 ? 4 : 1;
  __shared__ float part[2 * W];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, w = W == 1 ? 0 : wave;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + (W == 1 ? wave : 0); row < N.rows;
       row += static_cast<int64_t>(gridDim.x) * kRows) {
    const char* const x = static_cast<const char*>(N.x.p) + row * N.x.ld * kElem;
    float v[V][kVals];
    u4 raw[V];
#pragma unroll
    for (int j = 0; j < V; ++j) raw[j] = Slot<DT, W>(j, w, lane, N.cols).load(x);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const Slot<DT, W> slot(j, w, lane, N.cols);
      widen<DT>(raw[j], v[j]);
#pragma unroll
      for (int e = 0; e < kVals; ++e) sum = __builtin_fmaf(e >= slot.skip ? v[j][e] : 0.f, N.scale, sum);
    }
    const float mean = row_sum<W>(sum, part, w, lane) * N.unscale;
    float sq = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const Slot<DT, W> slot(j, w, lane, N.cols);
#pragma unroll
      for (int e = 0; e < kVals; ++e) {
        v[j][e] -= mean;
        const float d = e >= slot.skip ? v[j][e] : 0.f;
        sq = __builtin_fmaf(d, d, sq);
      }
    }
    sq = row_sum<W>(sq, part + W, w, lane);
    float rstd = 1.0f / sqrtf(sq * N.inv + N.eps);
    if (__builtin_expect(!__builtin_isfinite(sq), 0)) {
      sq = 0.f;
      int again = lane;
      asm volatile("" : "+v"(again));  // the masks of `skip` are made anew, or they would be held up to here
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const Slot<DT, W> slot(j, w, again, N.cols);
#pragma unroll
        for (int e = 0; e < kVals; ++e) {
          const float d = e >= slot.skip ? v[j][e] * kFar : 0.f;
          sq = __builtin_fmaf(d, d, sq);
        }
      }
      if (W > 1) __syncthreads();  // the sums have been read
      rstd = rstd_of_far(row_sum<W>(sq, part + W, w, lane), N.inv, N.eps);
    }
    if (N.mean && lane == 0 && w == 0) {
      N.mean[row] = mean;
      N.rstd[row] = rstd;
    }
    char* const y = static_cast<char*>(N.y.p) + row * N.y.ld * kElem;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const Slot<DT, W> slot(j, w, lane, N.cols);
      if (slot.skip >= kVals) continue;
      float g[kVals], b[kVals] = {};
      load_weight<DT>(N.weight, N.w_dt, slot.at, g);
      if (N.bias) load_weight<DT>(N.bias, N.w_dt, slot.at, b);
#pragma unroll
      for (int e = 0; e < kVals; ++e) g[e] = __builtin_fmaf(v[j][e] * rstd, g[e], b[e]);
      slot.store(y, narrow<DT>(g));
    }
  }
}

// Rows too long for the registers of a block, or shorter than a slot: read three times.
// 8192 x 16384 bf16 in registers takes 111 us; a row that is read again costs as
// much more as the caches do not hold.
constexpr int kLongThreads = 1024;

template <int DT>
__global__ void __launch_bounds__(kLongThreads) norm_long_kernel(const NormArgs N) {
  constexpr int kVals = Vec<DT>::kVals, kElem = Vec<DT>::kElem, kWaves = kLongThreads / 64;
  __shared__ float part[2 * kWaves];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  for (int64_t row = blockIdx.x; row < N.rows; row += gridDim.x) {
    const char* const x = static_cast<const char*>(N.x.p) + row * N.x.ld * kElem;
    auto each = [&](auto&& f) {
      for (int col = threadIdx.x * kVals; col < N.cols; col += kLongThreads * kVals) {
        float v[kVals];
        widen<DT>(load_part<DT>(x + col * kElem, N.cols - col), v);
        f(col, v);
      }
    };
    float sum = 0.f;
    each([&](int, const float* v) {
      for (int e = 0; e < kVals; ++e) sum = __builtin_fmaf(v[e], N.scale, sum);
    });
    const float mean = row_sum<kWaves>(sum, part, w, lane) * N.unscale;
    auto squares = [&](float far) {
      float sq = 0.f;
      each([&](int col, const float* v) {
        for (int e = 0; e < kVals; ++e) {
          const float d = col + e < N.cols ? (v[e] - mean) * far : 0.f;
          sq = __builtin_fmaf(d, d, sq);
        }
      });
      return row_sum<kWaves>(sq, part + kWaves, w, lane);
    };
    const float sq = squares(1.f);
    float rstd = 1.0f / sqrtf(sq * N.inv + N.eps);
    if (__builtin_expect(!__builtin_isfinite(sq), 0)) {
      __syncthreads();  // the sums have been read
      rstd = rstd_of_far(squares(kFar), N.inv, N.eps);
    }
    if (N.mean && threadIdx.x == 0) {
      N.mean[row] = mean;
      N.rstd[row] = rstd;
    }
    char* const y = static_cast<char*>(N.y.p) + row * N.y.ld * kElem;
    each([&](int col, const float* v) {
      float g[kVals], b[kVals] = {};
      load_weight_part<DT>(N.weight, N.w_dt, col, N.cols, g);
      if (N.bias) load_weight_part<DT>(N.bias, N.w_dt, col, N.cols, b);
      for (int e = 0; e < kVals; ++e) g[e] = __builtin_fmaf((v[e] - mean) * rstd, g[e], b[e]);
      store_part<DT>(y + col * kElem, N.cols - col, narrow<DT>(g));
    });
  }
}

// ------------------------------------------------------------------------
// Backward
// ------------------------------------------------------------------------

// Floats of a row of column sums.
__host__ __device__ inline int64_t sums_pitch(int64_t cols) { return (cols + 3) / 4 * 4; }

// G groups of W waves a block; a group takes a row at a time, a lane V slots of
// it, always of the same columns, whose sums over the rows it keeps. At the
// end the block's groups add theirs in group order through LDS and the block
// leaves one row of sums. The next row's loads are in flight while a row is
// worked on. A block's groups take equally many turns, so that its barriers meet.
// Measured, 16384 x 4096 bf16 with dresidual: 91-92 us (5.8-5.9 TB/s) and 4.6 for
// the join; two blocks a CU instead of one are no faster there and 10 % slower
// at 8192 x 1600 fp16 (28 us with the join, 29 with dresidual). All of it goes past
// the caches (115 -> 107 us).
template <int DT, int V, int W, int G, bool RES>
__global__ void __launch_bounds__(64 * W * G, 2) norm_grad_kernel(const NormGradArgs N) {
  constexpr int kVals = Vec<DT>::kVals, kElem = Vec<DT>::kElem;
  __shared__ float part[2][2][G][W];
  __shared__ f4 sums[G > 1 ? (G - 1) * 64 * W * V * kVals / 4 * 2 : 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = wave / W, w = wave % W;
  const float inv = 1.0f / static_cast<float>(N.cols);
  auto slot = [&](int j) { return Slot<DT, W>(j, w, lane, N.cols); };
  u4 x[V], dy[V], res[V];
  float next_mean, next_rstd;
  auto fetch = [&](int64_t row) {  // the last row again past it
    row = row < N.rows ? row : N.rows - 1;
    next_mean = N.mean[row];
    next_rstd = N.rstd[row];
    const char* const px = static_cast<const char*>(N.x.p) + row * N.x.ld * kElem;
    const char* const pd = static_cast<const char*>(N.dy.p) + row * N.dy.ld * kElem;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      x[j] = slot(j).load_once(px);
      dy[j] = slot(j).load_once(pd);
    }
    if (RES) {
      const char* const pr = static_cast<const char*>(N.dresidual.p) + row * N.dresidual.ld * kElem;
#pragma unroll
      for (int j = 0; j < V; ++j) res[j] = slot(j).load_once(pr);
    }
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * G;
  int64_t row = static_cast<int64_t>(blockIdx.x) * G + g;
  fetch(row);
  float weight[V][kVals], dw[V][kVals] = {}, db[V][kVals] = {};
#pragma unroll
  for (int j = 0; j < V; ++j) load_weight<DT>(N.weight, N.w_dt, slot(j).at, weight[j]);
  int turn = 0;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * G; base < N.rows; base += step, row += step, turn ^= 1) {
    const bool mine = row < N.rows;
    const float mean = next_mean, rstd = next_rstd;
    u4 x0[V], dy0[V], res0[V];
    // xhat and v of slot j, formed again where they are used: keeping them in
    // fp32 would take the registers of half the waves
    auto values = [&](int j, float* d, float* xhat, float* v) {
      widen<DT>(x0[j], xhat);
      widen<DT>(dy0[j], d);
#pragma unroll
      for (int e = 0; e < kVals; ++e) {
        xhat[e] = (xhat[e] - mean) * rstd;
        v[e] = d[e] * weight[j][e];
      }
    };
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float d[kVals], xhat[kVals], v[kVals];
      x0[j] = x[j];
      dy0[j] = dy[j];
      if (RES) res0[j] = res[j];
      if (!mine) continue;
      values(j, d, xhat, v);
#pragma unroll
      for (int e = 0; e < kVals; ++e) {
        // values that another slot has too add nothing to the row's sums; of
        // the column sums theirs are not taken
        const bool own = e >= slot(j).skip;
        s1 += own ? v[e] : 0.f;
        s2 = __builtin_fmaf(own ? v[e] : 0.f, own ? xhat[e] : 0.f, s2);
        dw[j][e] = __builtin_fmaf(d[e], xhat[e], dw[j][e]);
        db[j][e] += d[e];
      }
    }
    fetch(row + step);
    s1 = wave_sum(s1);
    s2 = wave_sum(s2);
    if constexpr (W > 1) {
      if (lane == 0) {
        part[turn][0][g][w] = s1;
        part[turn][1][g][w] = s2;
      }
      __syncthreads();
      s1 = s2 = 0.f;
#pragma unroll
      for (int q = 0; q < W; ++q) {
        s1 += part[turn][0][g][q];
        s2 += part[turn][1][g][q];
      }
    }
    const float c1 = s1 * inv, c2 = s2 * inv;
    if (mine) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (slot(j).skip >= kVals) continue;
        float out[kVals] = {}, d[kVals], xhat[kVals], v[kVals];
        asm("" : "+v"(x0[j]), "+v"(dy0[j]));  // not the values of before
        values(j, d, xhat, v);
        if (RES) widen<DT>(res0[j], out);
#pragma unroll
        for (int e = 0; e < kVals; ++e) out[e] = __builtin_fmaf(rstd, __builtin_fmaf(-xhat[e], c2, v[e] - c1), out[e]);
        slot(j).store(static_cast<char*>(N.dx.p) + row * N.dx.ld * kElem, narrow<DT>(out));
      }
    }
  }
  if (!N.partials) return;
  constexpr int kQuads = V * kVals / 4;
  if constexpr (G > 1) {
    constexpr int kItem = 2 * kQuads, kGroup = 64 * W * kItem;
    f4* const at = sums + (w * 64 + lane) * kItem;
    if (g > 0) {
#pragma unroll
      for (int j = 0; j < kQuads; ++j) {
        const float *a = &dw[0][0] + 4 * j, *b = &db[0][0] + 4 * j;
        at[(g - 1) * kGroup + j] = (f4){a[0], a[1], a[2], a[3]};
        at[(g - 1) * kGroup + kQuads + j] = (f4){b[0], b[1], b[2], b[3]};
      }
    }
    __syncthreads();
    if (g == 0) {
#pragma unroll 1
      for (int q = 0; q < G - 1; ++q)
#pragma unroll
        for (int j = 0; j < kQuads; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            (&dw[0][0])[4 * j + e] += at[q * kGroup + j][e];
            (&db[0][0])[4 * j + e] += at[q * kGroup + kQuads + j][e];
          }
    }
  }
  if (g == 0) {
    const int64_t pitch = sums_pitch(N.cols);
    float* const to = N.partials + blockIdx.x * 2 * pitch;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float* const at = to + slot(j).at;
      if (slot(j).skip == 0) {
#pragma unroll
        for (int q = 0; q < kVals; q += 4) {
          *reinterpret_cast<f4*>(at + q) = (f4){dw[j][q], dw[j][q + 1], dw[j][q + 2], dw[j][q + 3]};
          *reinterpret_cast<f4*>(at + pitch + q) = (f4){db[j][q], db[j][q + 1], db[j][q + 2], db[j][q + 3]};
        }
      } else {
#pragma unroll
        for (int e = 0; e < kVals; ++e)
          if (e >= slot(j).skip) {
            at[e] = dw[j][e];
            at[pitch + e] = db[j][e];
          }
      }
    }
  }
}

// Rows too long for the registers, or shorter than a slot: dx by reading a row twice, and the column
// sums in a pass of their own, a column a lane, a run of rows a block row.
template <int DT>
__global__ void __launch_bounds__(kLongThreads) norm_grad_long_kernel(const NormGradArgs N) {
  constexpr int kVals = Vec<DT>::kVals, kElem = Vec<DT>::kElem, kWaves = kLongThreads / 64;
  __shared__ float part[2][2 * kWaves];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const float inv = 1.0f / static_cast<float>(N.cols);
  int turn = 0;
  for (int64_t row = blockIdx.x; row < N.rows; row += gridDim.x, turn ^= 1) {
    const float mean = N.mean[row], rstd = N.rstd[row];
    auto each = [&](auto&& f) {
      for (int col = threadIdx.x * kVals; col < N.cols; col += kLongThreads * kVals) {
        float x[kVals], d[kVals], g[kVals];
        widen<DT>(load_part<DT>(static_cast<const char*>(N.x.p) + (row * N.x.ld + col) * kElem, N.cols - col), x);
        widen<DT>(load_part<DT>(static_cast<const char*>(N.dy.p) + (row * N.dy.ld + col) * kElem, N.cols - col), d);
        load_weight_part<DT>(N.weight, N.w_dt, col, N.cols, g);
        for (int e = 0; e < kVals; ++e) {
          x[e] = col + e < N.cols ? (x[e] - mean) * rstd : 0.f;
          d[e] *= g[e];
        }
        f(col, x, d);
      }
    };
    float s1 = 0.f, s2 = 0.f;
    each([&](int, const float* xhat, const float* v) {
      for (int e = 0; e < kVals; ++e) {
        s1 += v[e];
        s2 = __builtin_fmaf(v[e], xhat[e], s2);
      }
    });
    const float c1 = row_sum<kWaves>(s1, part[turn], w, lane) * inv;
    const float c2 = row_sum<kWaves>(s2, part[turn] + kWaves, w, lane) * inv;
    each([&](int col, const float* xhat, const float* v) {
      float out[kVals], r[kVals] = {};
      if (N.dresidual.p)
        widen<DT>(load_part<DT>(static_cast<const char*>(N.dresidual.p) + (row * N.dresidual.ld + col) * kElem,
                                N.cols - col), r);
      for (int e = 0; e < kVals; ++e) out[e] = __builtin_fmaf(rstd, __builtin_fmaf(-xhat[e], c2, v[e] - c1), r[e]);
      store_part<DT>(static_cast<char*>(N.dx.p) + (row * N.dx.ld + col) * kElem, N.cols - col, narrow<DT>(out));
    });
  }
}

template <int DT>
__global__ void __launch_bounds__(256) norm_sums_long_kernel(const NormGradArgs N, int64_t rows_each) {
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (col >= N.cols) return;
  const int64_t first = blockIdx.y * rows_each, end = first + rows_each < N.rows ? first + rows_each : N.rows;
  float dw = 0.f, db = 0.f;
  for (int64_t row = first; row < end; ++row) {
    const float d = load_one(N.dy.p, row * N.dy.ld + col, DT);
    dw = __builtin_fmaf(d, (load_one(N.x.p, row * N.x.ld + col, DT) - N.mean[row]) * N.rstd[row], dw);
    db += d;
  }
  float* const to = N.partials + blockIdx.y * 2 * sums_pitch(N.cols);
  to[col] = dw;
  to[sums_pitch(N.cols) + col] = db;
}

// The blocks' column sums, added: 32 columns a block, 32 runs of partial rows,
// each in order, then the runs in order.
constexpr int kJoinCols = 32, kJoinRuns = 32;

__global__ void __launch_bounds__(256) norm_join_kernel(const NormGradArgs N, int count) {
  void* const out = blockIdx.y ? N.dbias : N.dweight;
  if (!out) return;
  __shared__ f4 run[kJoinRuns][kJoinCols / 4];
  const int q = threadIdx.x % (kJoinCols / 4), k = threadIdx.x / (kJoinCols / 4);
  const int64_t pitch = sums_pitch(N.cols), col = static_cast<int64_t>(blockIdx.x) * kJoinCols + 4 * q;
  const float* const from = N.partials + blockIdx.y * pitch + col;
  const int each = (count + kJoinRuns - 1) / kJoinRuns;
  f4 s = {0.f, 0.f, 0.f, 0.f};
  if (col < pitch) {
    const int end = (k + 1) * each < count ? (k + 1) * each : count;
#pragma unroll 4
    for (int i = k * each; i < end; ++i) s += *reinterpret_cast<const f4*>(from + i * 2 * pitch);
  }
  run[k][q] = s;
  __syncthreads();
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kJoinCols + threadIdx.x;
  if (threadIdx.x >= kJoinCols || c >= N.cols) return;
  float t = N.accumulate ? load_one(out, c, N.dw_dt) : 0.f;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kJoinRuns; ++i) sum += run[i][threadIdx.x / 4][threadIdx.x % 4];
  store_one(out, c, N.dw_dt, t + sum);
}

template <int DT, int V, int W>
hipError_t norm_start(const NormArgs& a, hipStream_t s) {
  constexpr int kRows = W == 1 ? 4 : 1;
  const int64_t blocks = ceil_div(a.rows, kRows);
  const int grid = limit_grid(static_cast<int>(blocks < kMaxGrid ? blocks : kMaxGrid));
  hipLaunchKernelGGL((norm_kernel<DT, V, W>), dim3(grid), dim3(W == 1 ? 256 : 64 * W), 0, s, a);
  return hipGetLastError();
}

// As many waves a row as leave a lane two to four slots (us at 16384 x 4096 bf16:
// four waves with two slots 49.7, two with four 54.4, eight with one 55.5).
template <int DT>
hipError_t norm_launch(const NormArgs& a, hipStream_t s) {
  const int64_t slots = ceil_div(a.cols, Vec<DT>::kVals);
  if (a.cols >= Vec<DT>::kVals) {
    if (slots <= 64) return norm_start<DT, 1, 1>(a, s);
    if (slots <= 128) return norm_start<DT, 2, 1>(a, s);
    if (slots <= 256) return norm_start<DT, 2, 2>(a, s);  // one wave with four slots: 7 % more at 8192 x 1600 fp16
    if (slots <= 512) return norm_start<DT, 2, 4>(a, s);
    if (slots <= 1024) return norm_start<DT, 4, 4>(a, s);
    if (slots <= 2048) return norm_start<DT, 4, 8>(a, s);
    if (slots <= 4096) return norm_start<DT, 4, 16>(a, s);
  }
  const int grid = limit_grid(static_cast<int>(a.rows < kMaxGrid ? a.rows : kMaxGrid));
  hipLaunchKernelGGL(norm_long_kernel<DT>, dim3(grid), dim3(kLongThreads), 0, s, a);
  return hipGetLastError();
}

constexpr int kGradBlocks = 256;  // one for each CU

template <int DT, int V, int W, int G>
hipError_t norm_grad_start(const NormGradArgs& a, int64_t limit, hipStream_t s, int* count) {
  int64_t blocks = ceil_div(a.rows, G);
  blocks = blocks < limit ? blocks : limit;
  *count = limit_grid(static_cast<int>(blocks < kGradBlocks ? blocks : kGradBlocks));
  if (a.dresidual.p) hipLaunchKernelGGL((norm_grad_kernel<DT, V, W, G, true>), dim3(*count), dim3(64 * W * G), 0, s, a);
  else hipLaunchKernelGGL((norm_grad_kernel<DT, V, W, G, false>), dim3(*count), dim3(64 * W * G), 0, s, a);
  return hipGetLastError();
}

template <int DT>
hipError_t norm_grad_launch(const NormGradArgs& a, hipStream_t s) {
  const int64_t slots = ceil_div(a.cols, Vec<DT>::kVals);
  if (a.rows == 0) {  // sums over no rows
    hipLaunchKernelGGL(norm_join_kernel, dim3(static_cast<uint32_t>(ceil_div(a.cols, kJoinCols)), 2), dim3(256), 0, s, a, 0);
    return hipGetLastError();
  }
  // the blocks whose sums the workspace holds
  const int64_t limit = static_cast<int64_t>(kScratchBytes / (2 * sizeof(float))) / sums_pitch(a.cols);
  int count = 0;
  hipError_t e;
  const bool whole = a.cols >= Vec<DT>::kVals;
  if (whole && slots <= 64) e = norm_grad_start<DT, 1, 1, 8>(a, limit, s, &count);
  else if (whole && slots <= 128) e = norm_grad_start<DT, 2, 1, 8>(a, limit, s, &count);
  else if (whole && slots <= 256) e = norm_grad_start<DT, 2, 2, 4>(a, limit, s, &count);
  else if (whole && slots <= 512) e = norm_grad_start<DT, 2, 4, 2>(a, limit, s, &count);
  else if (whole && slots <= 1024) e = norm_grad_start<DT, 2, 8, 1>(a, limit, s, &count);
  else if (whole && slots <= 2048) e = norm_grad_start<DT, 4, 8, 1>(a, limit, s, &count);
  else {
    const int grid = limit_grid(static_cast<int>(a.rows < kMaxGrid ? a.rows : kMaxGrid));
    hipLaunchKernelGGL(norm_grad_long_kernel<DT>, dim3(grid), dim3(kLongThreads), 0, s, a);
    if (hipError_t x = hipGetLastError()) return x;
    e = hipSuccess;
    if (a.partials) {
      int64_t runs = ceil_div(a.rows, 64);  // rows of a run, or more
      runs = runs < limit ? runs : limit;
      runs = runs < 64 ? runs : 64;
      const int64_t each = ceil_div(a.rows, runs);
      count = static_cast<int>(ceil_div(a.rows, each));
      hipLaunchKernelGGL(norm_sums_long_kernel<DT>, dim3(static_cast<uint32_t>(ceil_div(a.cols, 256)), count), dim3(256),
                         0, s, a, each);
      e = hipGetLastError();
    }
  }
  if (e != hipSuccess || !a.partials) return e;
  hipLaunchKernelGGL(norm_join_kernel, dim3(static_cast<uint32_t>(ceil_div(a.cols, kJoinCols)), 2), dim3(256), 0, s, a,
                     count);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, int32_t dt, hipStream_t s) {
  if (dt == ZERO_DT_F32) return norm_launch<ZERO_DT_F32>(a, s);
  if (dt == ZERO_DT_F16) return norm_launch<ZERO_DT_F16>(a, s);
  if (dt == ZERO_DT_BF16) return norm_launch<ZERO_DT_BF16>(a, s);
  return hipErrorInvalidValue;
}

hipError_t launch_norm_grad(const NormGradArgs& a, int32_t dt, hipStream_t s) {
  if (dt == ZERO_DT_F32) return norm_grad_launch<ZERO_DT_F32>(a, s);
  if (dt == ZERO_DT_F16) return norm_grad_launch<ZERO_DT_F16>(a, s);
  if (dt == ZERO_DT_BF16) return norm_grad_launch<ZERO_DT_BF16>(a, s);
  return hipErrorInvalidValue;
}

}  // namespace zdp
