// gfx950 kernels of the product of two microscaled 4-bit matrices,
//   out[i][j] = sum_k A[i][k] * B[j][k],
// on the scaled matrix instruction v_mfma_scale_f32_32x32x64 with both operands
// in E2M1: lane l of a wave gives row l & 31 of either operand and its 32-value
// block l >> 5 of the instruction's two, so a lane's operand is exactly one
// block (16 bytes of codes) and its scale byte. The instruction multiplies by
// both scales and sums in fp32. A's rows are the instruction's columns and B's
// rows its rows, so that a lane holds four consecutive columns of one output
// row. Both kernels walk the contraction in chunks of 8 blocks (256 values).
#include <atomic>
#include <type_traits>

#include "mx_device.h"

namespace zdp {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));

constexpr int kE2M1 = 4;     // the instruction's format code for both operands
constexpr int kChunk = 8;    // blocks of the contraction per chunk
constexpr int kSteps = 4;    // instructions per chunk and output tile of 32 x 32
constexpr int kFrag = 32;    // rows of an operand per instruction

// Step s of a chunk multiplies blocks 2s and 2s + 1. `sa` and `sb` hold the
// scales of a lane's blocks of the chunk, step s in byte 2 * (s & 1) of dword
// s >> 1 (chunk_scales).
template <int S>
__device__ __forceinline__ v16f mfma(v4i b, u2 sb, v4i a, u2 sa, v16f c) {
  const v8i A = {a.x, a.y, a.z, a.w, 0, 0, 0, 0}, B = {b.x, b.y, b.z, b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(B, A, c, kE2M1, kE2M1, 2 * (S & 1),
                                                         static_cast<int>(S < 2 ? sb.x : sb.y), 2 * (S & 1),
                                                         static_cast<int>(S < 2 ? sa.x : sa.y));
}

// A row's 8 scale bytes of a chunk, shifted so that the bytes of the lane's
// blocks (2s + g) stand at bytes 0, 2, 4, 6.
__device__ __forceinline__ u2 chunk_scales(u2 row, int g) {
  u2 s;
  s.x = __builtin_amdgcn_alignbyte(row.y, row.x, g);
  s.y = row.y >> (8 * g);
  return s;
}

// The 8 scale bytes at p, at any alignment; only the first `left` if fewer exist, then 0.
__device__ __forceinline__ u2 load_scales(const uint8_t* p, int64_t left) {
  u2 s = {0, 0};
  if (left >= kChunk) {
    __builtin_memcpy(&s, p, 8);
  } else {
#pragma unroll
    for (int q = 0; q < kChunk; ++q) {
      const uint32_t x = q < left ? p[q] : 0u;
      if (q < 4) s.x |= x << (8 * q);
      else s.y |= x << (8 * (q - 4));
    }
  }
  return s;
}

// Columns [col, col + 8) of an output row, as far as they exist.
template <int DT>
__device__ __forceinline__ void store8(void* out, int64_t at, int64_t left, const float v[8]) {
  if constexpr (DT == ZERO_DT_F32) {
    float* p = static_cast<float*>(out) + at;
    if (left >= 8) {
      const f4 a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
      __builtin_memcpy(p, &a, 16);
      __builtin_memcpy(p + 4, &b, 16);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < left) p[q] = v[q];
    }
  } else {
    uint16_t* p = static_cast<uint16_t*>(out) + at;
    uint32_t h[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) h[q] = encode16(v[q], DT);
    if (left >= 8) {
      const u4 w = {h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16)};
      __builtin_memcpy(p, &w, 16);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < left) p[q] = static_cast<uint16_t>(h[q]);
    }
  }
}

__device__ __forceinline__ uint32_t tiles_of(int64_t n, uint32_t size) { return (static_cast<uint32_t>(n) + size - 1) / size; }

// Tiles dealt to the eight XCDs (block b runs on XCD b % 8) in contiguous
// runs, and inside a run in columns of kGroup tile rows, so that the tiles that
// an XCD's 32 CUs work on at a time share their operands in its L2.
constexpr int kXcds = 8;
constexpr int kGroup = 8;

__device__ __forceinline__ void tile_of(uint32_t b, uint32_t tm, uint32_t tn, uint32_t* m, uint32_t* n) {
  const uint32_t total = tm * tn, q = total / kXcds, rem = total % kXcds;
  const uint32_t x = b % kXcds;
  const uint32_t i = x * q + (x < rem ? x : rem) + b / kXcds;
  const uint32_t width = kGroup * tn, first = i / width * kGroup;
  const uint32_t rows = tm - first < kGroup ? tm - first : kGroup;
  const uint32_t at = i % width;
  *m = __builtin_amdgcn_readfirstlane(first + at % rows);
  *n = __builtin_amdgcn_readfirstlane(at / rows);
}

// ------------------------------------------------------------------------
// Few output tiles: a block owns an output tile of 32 FM x 32 FN and its waves
// split the contraction, chunk by chunk in turn; operands go from global memory
// straight to registers, and the waves' sums are added through LDS in wave
// order.
// ------------------------------------------------------------------------

template <int FM, int FN, int NW, int DT>
__global__ void __launch_bounds__(64 * NW) mx_product_split_kernel(const MxProductArgs P) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int r = lane & 31, g = lane >> 5;
  uint32_t tm, tn;
  tile_of(blockIdx.x, tiles_of(P.m, kFrag * FM), tiles_of(P.n, kFrag * FN), &tm, &tn);
  const int64_t m0 = static_cast<int64_t>(tm) * kFrag * FM, n0 = static_cast<int64_t>(tn) * kFrag * FN;
  const v4i *ac[FM], *bc[FN];
  const uint8_t *as[FM], *bs[FN];
#pragma unroll
  for (int f = 0; f < FM; ++f) {
    const int64_t i = m0 + f * kFrag + r;
    const int64_t row = (i < P.m ? i : P.m - 1) * P.lda;
    ac[f] = reinterpret_cast<const v4i*>(P.a_codes) + row + g;
    as[f] = P.a_scales + row;
  }
#pragma unroll
  for (int f = 0; f < FN; ++f) {
    const int64_t j = n0 + f * kFrag + r;
    const int64_t row = (j < P.n ? j : P.n - 1) * P.ldb;
    bc[f] = reinterpret_cast<const v4i*>(P.b_codes) + row + g;
    bs[f] = P.b_scales + row;
  }
  v16f acc[FM][FN] = {};
  for (int64_t k = static_cast<int64_t>(w) * kChunk; k < P.kb; k += NW * kChunk) {
    v4i a[FM][kSteps], b[FN][kSteps];
    u2 sa[FM], sb[FN];
    const int64_t left = P.kb - k;
#pragma unroll
    for (int f = 0; f < FN; ++f) {
#pragma unroll
      for (int s = 0; s < kSteps; ++s) b[f][s] = 2 * s + g < left ? bc[f][k + 2 * s] : (v4i){};
      sb[f] = load_scales(bs[f] + k, left);
    }
#pragma unroll
    for (int f = 0; f < FM; ++f) {
#pragma unroll
      for (int s = 0; s < kSteps; ++s) a[f][s] = 2 * s + g < left ? ac[f][k + 2 * s] : (v4i){};
      sa[f] = load_scales(as[f] + k, left);
    }
#pragma unroll
    for (int f = 0; f < FN; ++f) sb[f] = chunk_scales(sb[f], g);
#pragma unroll
    for (int f = 0; f < FM; ++f) sa[f] = chunk_scales(sa[f], g);
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        acc[i][j] = mfma<0>(b[j][0], sb[j], a[i][0], sa[i], acc[i][j]);
        acc[i][j] = mfma<1>(b[j][1], sb[j], a[i][1], sa[i], acc[i][j]);
        acc[i][j] = mfma<2>(b[j][2], sb[j], a[i][2], sa[i], acc[i][j]);
        acc[i][j] = mfma<3>(b[j][3], sb[j], a[i][3], sa[i], acc[i][j]);
      }
  }
  // Sum over the waves, one 32 x 32 fragment at a time: wave w's in part[w],
  // row-major with a pad of 4 floats.
  __shared__ float part[NW][kFrag][kFrag + 4];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      if (i + j > 0) __syncthreads();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f4 x = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        *reinterpret_cast<f4*>(&part[w][r][8 * q + 4 * g]) = x;
      }
      __syncthreads();
      const int t = threadIdx.x;
      if (t < kFrag * kFrag / 8) {
        const int row = t >> 2, col = (t & 3) * 8;
        float v[8] = {};
#pragma unroll
        for (int u = 0; u < NW; ++u)
#pragma unroll
          for (int q = 0; q < 8; ++q) v[q] += part[u][row][col + q];
        const int64_t om = m0 + i * kFrag + row, on = n0 + j * kFrag + col;
        if (om < P.m && on < P.n) store8<DT>(P.out, om * P.ldo + on, P.n - on, v);
      }
    }
}

// ------------------------------------------------------------------------
// Many output tiles: WM x WN waves, each with FM x FN fragments, share an
// output tile through LDS, two stages of one chunk each. Codes go from global
// memory to LDS without passing registers, 16 bytes a lane: eight lanes fetch
// a row's 128 bytes of the chunk, lane l of eight its block l ^ (row & 7), and
// LDS holds row after row of eight 16-byte slots in the order the lanes fetch.
// The reading lane finds block b of a row in slot b ^ (row & 7), so the eight
// rows that a read touches at a time lie in different banks.
// A stage's loads are issued when the stage before the last has been read out,
// a whole stage's products ahead of their use.
// ------------------------------------------------------------------------

constexpr int kRowBytes = kChunk * kMxCodeBytes;  // of codes per row and stage

template <int FM, int FN, int WM, int WN>
struct Tile {
  static constexpr int kM = kFrag * FM * WM, kN = kFrag * FN * WN;
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr int kRows = kM + kN;                 // A's rows, then B's
  static constexpr int kLoads = kRows / 8 / kWaves;     // of 1 KiB, per wave and stage
  static constexpr int kScaleLoads = (kRows + kThreads - 1) / kThreads;
  static constexpr int kCodes = kRows * kRowBytes;
  static constexpr int kStage = kCodes + kRows * kChunk;
  static constexpr int kOutRow = kFrag * FN + 4;        // floats, padded
  static constexpr int kOut = kWaves * kFrag * kOutRow * 4;
  static constexpr int kLds = 2 * kStage > kOut ? 2 * kStage : kOut;
  static_assert(kLds <= 160 * 1024, "LDS of a CU");
  static_assert(kRows % (8 * kWaves) == 0 && kRows % kThreads == 0, "rows per wave and thread");
};

// Fetch 16 bytes a lane from base + off into LDS at `lds` + 16 * lane. No register is written; the caller waits on vmcnt.
__device__ __forceinline__ void fetch_to_lds(const uint8_t* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base) : "memory");
}

template <int FM, int FN, int WM, int WN, int DT>
__global__ void __launch_bounds__(64 * WM * WN, 1) mx_product_tile_kernel(const MxProductArgs P) {
  using T = Tile<FM, FN, WM, WN>;
  extern __shared__ __align__(16) uint8_t lds[];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 31, g = lane >> 5;
  uint32_t tm, tn;
  tile_of(blockIdx.x, tiles_of(P.m, T::kM), tiles_of(P.n, T::kN), &tm, &tn);
  const int64_t m0 = static_cast<int64_t>(tm) * T::kM, n0 = static_cast<int64_t>(tn) * T::kN;
  const int64_t mlast = P.m - 1 - m0, nlast = P.n - 1 - n0;  // rows past the end repeat the last one

  // where a lane's loads start: row of the tile, block of the chunk
  const uint8_t* const abase = P.a_codes + m0 * P.lda * kMxCodeBytes;
  const uint8_t* const bbase = P.b_codes + n0 * P.ldb * kMxCodeBytes;
  const int lb = (lane & 7) ^ (lane >> 3);
  uint32_t off[T::kLoads];
#pragma unroll
  for (int j = 0; j < T::kLoads; ++j) {
    int64_t row = (j * T::kWaves + w) * 8 + (lane >> 3);
    int64_t ld = P.lda;
    if (row >= T::kM) {
      row -= T::kM;
      row = row < nlast ? row : nlast;
      ld = P.ldb;
    } else {
      row = row < mlast ? row : mlast;
    }
    off[j] = static_cast<uint32_t>((row * ld + lb) * kMxCodeBytes);
  }
  const uint8_t* srow[T::kScaleLoads];
#pragma unroll
  for (int j = 0; j < T::kScaleLoads; ++j) {
    int64_t row = j * T::kThreads + threadIdx.x;
    if (row >= T::kM) {
      row -= T::kM;
      srow[j] = P.b_scales + (n0 + (row < nlast ? row : nlast)) * P.ldb;
    } else {
      srow[j] = P.a_scales + (m0 + (row < mlast ? row : mlast)) * P.lda;
    }
  }

  // A partial last chunk is stage 0, so that every later stage is whole.
  const int64_t part = P.kb % kChunk, stages = (P.kb + kChunk - 1) / kChunk;
  auto chunk_of = [&](int64_t i) { return part ? (i == 0 ? stages - 1 : i - 1) : i; };
  u2 scales[T::kScaleLoads];
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)lds));
  auto fetch_scales = [&](int64_t k, int64_t left) {
#pragma unroll
    for (int j = 0; j < T::kScaleLoads; ++j) scales[j] = load_scales(srow[j] + k * kChunk, left);
  };
  auto fetch = [&](int64_t i, int64_t k, int j) {  // load j of stage i, chunk k
    const uint8_t* const from = ((j * T::kWaves) * 8 >= T::kM ? bbase : abase) + k * kRowBytes;
    fetch_to_lds(from, off[j], lds0 + static_cast<uint32_t>(i & 1) * T::kStage + (j * T::kWaves + w) * 1024);
  };
  auto publish = [&](int64_t i) {  // the fetched stage, to every wave
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    uint8_t* const at = lds + (i & 1) * T::kStage + T::kCodes;
#pragma unroll
    for (int j = 0; j < T::kScaleLoads; ++j)
      *reinterpret_cast<u2*>(at + (j * T::kThreads + threadIdx.x) * kChunk) = scales[j];
    __syncthreads();
  };

  const int wm = w / WN, wn = w % WN;
  const int arow = wm * FM * kFrag + r, brow = T::kM + wn * FN * kFrag + r;
  v4i a[2][FM], b[2][FN];
  u2 sa[FM], sb[FN];
  auto read_scales = [&](int64_t i) {
    const uint8_t* const at = lds + (i & 1) * T::kStage + T::kCodes;
#pragma unroll
    for (int f = 0; f < FM; ++f) sa[f] = chunk_scales(*reinterpret_cast<const u2*>(at + (arow + f * kFrag) * kChunk), g);
#pragma unroll
    for (int f = 0; f < FN; ++f) sb[f] = chunk_scales(*reinterpret_cast<const u2*>(at + (brow + f * kFrag) * kChunk), g);
  };
  // Fragment f of step s of stage i: B's first two, A's first, then the rest,
  // in the order in which the products need them.
  auto read = [&](int64_t i, int s, int f) {
    const uint8_t* const at = lds + (i & 1) * T::kStage + ((2 * s + g) ^ (r & 7)) * kMxCodeBytes;
    constexpr int kFirst = 2;
    if (f < kFirst) b[s & 1][f] = *reinterpret_cast<const v4i*>(at + (brow + f * kFrag) * kRowBytes);
    else if (f == kFirst) a[s & 1][0] = *reinterpret_cast<const v4i*>(at + arow * kRowBytes);
    else if (f <= FN) b[s & 1][f - 1] = *reinterpret_cast<const v4i*>(at + (brow + (f - 1) * kFrag) * kRowBytes);
    else a[s & 1][f - FN] = *reinterpret_cast<const v4i*>(at + (arow + (f - FN) * kFrag) * kRowBytes);
  };

  v16f acc[FM][FN] = {};
  constexpr int kGroups = FM * FN / 2;  // pairs of products per step
  constexpr int kReads = (FM + FN + kGroups - 1) / kGroups, kFetches = (T::kLoads + 2 * kGroups - 1) / (2 * kGroups);
  // One step: per group, a load or two of the next stage (steps 0 and 1), two
  // products, and a read or two of the next step's fragments. The order is
  // fixed, so that loads, reads and products leave in turn.
  auto step = [&](auto sc, auto morec, int64_t i) {
    constexpr int S = decltype(sc)::value;
    constexpr bool more = decltype(morec)::value;  // there is a next stage
    const int64_t k = more && S < 2 ? chunk_of(i + 1) : 0;
    u2 ta[FM], tb[FN];
#pragma unroll
    for (int f = 0; f < FM; ++f) ta[f] = sa[f];
#pragma unroll
    for (int f = 0; f < FN; ++f) tb[f] = sb[f];
    if constexpr (more && S == 0) fetch_scales(k, kChunk);
#pragma unroll
    for (int t = 0; t < kGroups; ++t) {
      if constexpr (more && S < 2) {
#pragma unroll
        for (int q = 0; q < kFetches; ++q) {
          const int j = (S * kGroups + t) * kFetches + q;
          if (j < T::kLoads) fetch(i + 1, k, j);
        }
      }
      if constexpr (more && S == 3) {
        if (t == 1) {
          publish(i + 1);
          read_scales(i + 1);
        }
      }
      const int x = 2 * t / FN, y = 2 * t % FN;
      acc[x][y] = mfma<S>(b[S & 1][y], tb[y], a[S & 1][x], ta[x], acc[x][y]);
      acc[x][y + 1] = mfma<S>(b[S & 1][y + 1], tb[y + 1], a[S & 1][x], ta[x], acc[x][y + 1]);
      if constexpr (S < 3) {
#pragma unroll
        for (int q = 0; q < kReads; ++q)
          if (t * kReads + q < FM + FN) read(i, S + 1, t * kReads + q);
      } else if constexpr (more) {
        // the reads of the next stage follow its publication
        constexpr int kLate = (FM + FN + kGroups - 2) / (kGroups - 1);
        if (t > 0) {
#pragma unroll
          for (int q = 0; q < kLate; ++q)
            if ((t - 1) * kLate + q < FM + FN) read(i + 1, 0, (t - 1) * kLate + q);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto stage = [&](auto morec, int64_t i) {
    step(std::integral_constant<int, 0>{}, morec, i);
    step(std::integral_constant<int, 1>{}, morec, i);
    step(std::integral_constant<int, 2>{}, morec, i);
    step(std::integral_constant<int, 3>{}, morec, i);
  };

  if (stages > 0) {
    if (part) {
      // blocks past the end are zero
      const int64_t k = stages - 1;
#pragma unroll
      for (int j = 0; j < T::kLoads; ++j) {
        v4i x = {};
        if (lb < part)
          x = *reinterpret_cast<const v4i*>(((j * T::kWaves) * 8 >= T::kM ? bbase : abase) + k * kRowBytes + off[j]);
        *reinterpret_cast<v4i*>(lds + (j * T::kWaves + w) * 1024 + lane * 16) = x;
      }
      fetch_scales(k, part);
    } else {
#pragma unroll
      for (int j = 0; j < T::kLoads; ++j) fetch(0, 0, j);
      fetch_scales(0, kChunk);
    }
    publish(0);
    read_scales(0);
#pragma unroll
    for (int f = 0; f < FM + FN; ++f) read(0, 0, f);
    for (int64_t i = 0; i + 1 < stages; ++i) stage(std::true_type{}, i);
    stage(std::false_type{}, stages - 1);
    __syncthreads();
  }

  // 32 rows of the wave's part of the tile at a time, through LDS, so that a
  // row leaves in runs of 8 columns a lane.
  float* const mine = reinterpret_cast<float*>(lds) + w * kFrag * T::kOutRow;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f4 x = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        *reinterpret_cast<f4*>(mine + r * T::kOutRow + j * kFrag + 8 * q + 4 * g) = x;
      }
    __builtin_amdgcn_wave_barrier();
    constexpr int kRuns = kFrag * FN / 8;  // of a row
#pragma unroll
    for (int t = 0; t < kFrag * kRuns / 64; ++t) {
      const int row = (t * 64 + lane) / kRuns, col = (t * 64 + lane) % kRuns * 8;
      const f4 x = *reinterpret_cast<const f4*>(mine + row * T::kOutRow + col);
      const f4 y = *reinterpret_cast<const f4*>(mine + row * T::kOutRow + col + 4);
      const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
      const int64_t om = m0 + (wm * FM + i) * kFrag + row, on = n0 + wn * FN * kFrag + col;
      if (om < P.m && on < P.n) store8<DT>(P.out, om * P.ldo + on, P.n - on, v);
    }
    __builtin_amdgcn_wave_barrier();
  }
}

template <int FM, int FN, int NW, int DT>
hipError_t split_launch(const MxProductArgs& a, hipStream_t s) {
  const int64_t tiles = mx_tiles(a.m, kFrag * FM) * mx_tiles(a.n, kFrag * FN);
  hipLaunchKernelGGL((mx_product_split_kernel<FM, FN, NW, DT>), dim3(static_cast<uint32_t>(tiles)), dim3(64 * NW), 0, s,
                     a);
  return hipGetLastError();
}

template <int FM, int FN, int WM, int WN, int DT>
hipError_t tile_launch(const MxProductArgs& a, hipStream_t s) {
  using T = Tile<FM, FN, WM, WN>;
  const auto kernel = mx_product_tile_kernel<FM, FN, WM, WN, DT>;
  // more than the default limit of 64 KiB of dynamic LDS, granted once per device
  static std::atomic<uint64_t> granted{0};
  int dev = 0;
  if (hipError_t e = hipGetDevice(&dev)) return e;
  const uint64_t bit = uint64_t{1} << (dev & 63);
  if (dev > 63 || !(granted.load(std::memory_order_acquire) & bit)) {
    if (hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, T::kLds))
      return e;
    granted.fetch_or(bit, std::memory_order_release);
  }
  const int64_t tiles = mx_tiles(a.m, T::kM) * mx_tiles(a.n, T::kN);
  hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(tiles)), dim3(T::kThreads), T::kLds, s, a);
  return hipGetLastError();
}

enum Variant { kSplit32, kSplit64x32, kSplit64, kTile256 };

Variant pick(const MxProductArgs& a) {
  if (mx_tiles(a.m, 256) * mx_tiles(a.n, 256) >= 128) return kTile256;
  if (a.m > 64 && a.n > 64) return kSplit64;
  return a.m > 32 ? kSplit64x32 : kSplit32;
}

template <int DT>
hipError_t product_launch(const MxProductArgs& a, hipStream_t s) {
  switch (pick(a)) {
    case kSplit32: return split_launch<1, 1, 8, DT>(a, s);
    case kSplit64x32: return split_launch<2, 1, 8, DT>(a, s);
    case kSplit64: return split_launch<2, 2, 4, DT>(a, s);
    case kTile256: return tile_launch<4, 2, 2, 4, DT>(a, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_mx_product(const MxProductArgs& a, int32_t dt, hipStream_t s) {
  if (dt == ZERO_DT_F32) return product_launch<ZERO_DT_F32>(a, s);
  if (dt == ZERO_DT_F16) return product_launch<ZERO_DT_F16>(a, s);
  if (dt == ZERO_DT_BF16) return product_launch<ZERO_DT_BF16>(a, s);
  return hipErrorInvalidValue;
}

}  // namespace zdp
