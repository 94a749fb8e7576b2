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
constexpr int kFrag = 32;    // rows of an operand per instruction

// Step s of a chunk multiplies blocks 2s and 2s + 1. `sa` and `sb` hold the
// scales of a lane's blocks of the chunk, step s in byte 2 * (s & 1) of dword
// s >> 1 (chunk_scales).
template <int S>
__device__ __forceinline__ v16f mfma(v4i b, uint32_t sb, v4i a, uint32_t sa, v16f c) {
  const v8i A = {a.x, a.y, a.z, a.w, 0, 0, 0, 0}, B = {b.x, b.y, b.z, b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(B, A, c, kE2M1, kE2M1, 2 * (S & 1), static_cast<int>(sb),
                                                         2 * (S & 1), static_cast<int>(sa));
}

template <int S>
__device__ __forceinline__ uint32_t step_scales(u2 s) {
  return S < 2 ? s.x : s.y;
}

// A row's 8 scale bytes of a chunk, shifted so that the bytes of the lane's
// blocks 2s + g stand at bytes 0, 2, 4, 6.
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

// A run of kRun = 16 bytes' worth of columns of an output row from column `at` on,
// as far as they exist. WHOLE: every row starts at a multiple of 16 bytes, so
// that lanes side by side write whole lines; those go past the caches (8192 x
// 14336 x 4096 in bf16: 280 -> 258 us; with rows off alignment, where lines are
// shared between two accesses, the hint cost 98 us instead of 80 at 1001 x
// 50257 x 1600).
template <int DT>
struct Run {
  static constexpr int kElem = DT == ZERO_DT_F32 ? 4 : 2;
  static constexpr int kCols = 16 / kElem;
};

__device__ __forceinline__ bool whole_lines(const void* out, int64_t ldo, int elem) {
  return ((reinterpret_cast<uintptr_t>(out) | static_cast<uintptr_t>(ldo * elem)) & 15) == 0;
}

template <int DT, bool WHOLE>
__device__ __forceinline__ void store_run(void* out, int64_t at, int64_t left, const float* v) {
  u4 x;
  if constexpr (DT == ZERO_DT_F32) {
    x = (u4){__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
  } else {
    uint32_t h[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) h[q] = encode16(v[q], DT);
    x = (u4){h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16)};
  }
  char* const p = static_cast<char*>(out) + at * Run<DT>::kElem;
  if (left >= Run<DT>::kCols) {
    if constexpr (WHOLE) st_stream(reinterpret_cast<u4*>(p), x);
    else __builtin_memcpy(p, &x, 16);
  } else {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    if constexpr (DT == ZERO_DT_F32) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (q < left) reinterpret_cast<uint32_t*>(p)[q] = w[q];
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < left) reinterpret_cast<uint16_t*>(p)[q] = static_cast<uint16_t>(w[q / 2] >> (16 * (q & 1)));
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

// Operands reach LDS in pieces of 1 KiB: eight lanes fetch the 128 bytes of a
// row's chunk, and LDS holds rows of eight 16-byte slots in the order the lanes
// fetch. Block b of row i stands in slot b ^ (i / 2) % 8, so that the same
// block of 16 neighbouring rows lies in 16 different groups of four of the 64
// banks. (Straight to registers a wave would touch 32 rows, 32 bytes each, per
// load: every line is then asked for four times, and the product of one token
// with 14336 x 4096 took 13.4 us instead of 8.4.)
constexpr int kRowBytes = kChunk * kMxCodeBytes;  // of a row's codes in a chunk
constexpr int kPieceRows = 8;
constexpr int kPiece = kPieceRows * kRowBytes;

__device__ __forceinline__ int fetch_block(int piece, int lane) { return (lane & 7) ^ (4 * (piece & 1) + (lane >> 4)); }

// Where block `block` of row `row` (from the start of a piece) stands.
__device__ __forceinline__ int slot_of(int row, int block) {
  return row * kRowBytes + (block ^ (row >> 1 & 7)) * kMxCodeBytes;
}

__device__ __forceinline__ uint32_t lds_address(const uint8_t* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const uint8_t*)p));
}

// m0 is named as overwritten, so that the compiler keeps no value of its own
// there across a fetch. It warns about every such list because it reserves m0
// and cannot save it; nothing needs it saved.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"

// Fetch 16 bytes a lane from base + off into LDS at `lds` + 16 * lane. No vector
// register is written; the caller waits on vmcnt. The hardware wants one wait
// state between the write of m0 and the load that takes its LDS base from it;
// inside an asm the compiler puts none in.
__device__ __forceinline__ void fetch_to_lds(const uint8_t* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base)
               : "memory", "m0");
}

// The same if i < n (uniform). The branch is the asm's own: one that the
// compiler sees splits the loop around it, and its accumulators are then kept
// twice. The compare and the branch are the wait states.
__device__ __forceinline__ void fetch_to_lds_if(uint32_t i, uint32_t n, const uint8_t* base, uint32_t off, uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %0\n\ts_cmp_ge_u32 %3, %4\n\ts_cbranch_scc1 .Lzdp_skip%=\n\t"
      "global_load_lds_dwordx4 %1, %2\n.Lzdp_skip%=:" ::"s"(lds), "v"(off), "s"(base), "s"(i), "s"(n)
      : "memory", "scc", "m0");
}

#pragma clang diagnostic pop

// ------------------------------------------------------------------------
// Few output tiles: a block owns an output tile of 32 FM x 32 FN and its waves
// take the contraction's chunks in turn, each through an LDS space of its own,
// so that no wave waits for another; the waves' sums are added through LDS in
// wave order.
// ------------------------------------------------------------------------

template <int FM, int FN, int NW>
struct Split {
  static constexpr int kSpace = (FM + FN) * kFrag * kRowBytes;  // of a wave
  static constexpr int kPartRow = kFrag + 4;                    // floats, padded
  static constexpr int kParts = NW * kFrag * kPartRow * 4;
  static constexpr int kLds = NW * kSpace > kParts ? NW * kSpace : kParts;
  static_assert(kLds <= 160 * 1024, "LDS of a CU");
};

template <int FM, int FN, int NW, int DT>
__global__ void __launch_bounds__(64 * NW) mx_product_split_kernel(const MxProductArgs P) {
  using T = Split<FM, FN, NW>;
  extern __shared__ __align__(16) uint8_t lds[];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 31, g = lane >> 5;
  uint32_t tm, tn;
  tile_of(blockIdx.x, tiles_of(P.m, kFrag * FM), tiles_of(P.n, kFrag * FN), &tm, &tn);
  const int64_t m0 = static_cast<int64_t>(tm) * kFrag * FM, n0 = static_cast<int64_t>(tn) * kFrag * FN;
  const int64_t mlast = P.m - 1 - m0, nlast = P.n - 1 - n0;  // rows past the end repeat the last one
  const uint8_t* const abase = P.a_codes + m0 * P.lda * kMxCodeBytes;
  const uint8_t* const bbase = P.b_codes + n0 * P.ldb * kMxCodeBytes;
  constexpr int kPieces = (FM + FN) * kFrag / kPieceRows, kPiecesA = FM * kFrag / kPieceRows;
  uint32_t off[kPieces];
#pragma unroll
  for (int j = 0; j < kPieces; ++j) {
    const bool is_a = j < kPiecesA;
    int64_t row = (is_a ? j : j - kPiecesA) * kPieceRows + (lane >> 3);
    const int64_t last = is_a ? mlast : nlast;
    row = row < last ? row : last;
    off[j] = static_cast<uint32_t>((row * (is_a ? P.lda : P.ldb) + fetch_block(j, lane)) * kMxCodeBytes);
  }
  const uint8_t *as[FM], *bs[FN];
#pragma unroll
  for (int f = 0; f < FM; ++f) {
    const int64_t i = f * kFrag + r;
    as[f] = P.a_scales + (m0 + (i < mlast ? i : mlast)) * P.lda;
  }
#pragma unroll
  for (int f = 0; f < FN; ++f) {
    const int64_t j = f * kFrag + r;
    bs[f] = P.b_scales + (n0 + (j < nlast ? j : nlast)) * P.ldb;
  }
  uint8_t* const mine = lds + w * T::kSpace;
  const uint32_t to = lds_address(mine);
  v16f acc[FM][FN] = {};
  const int64_t full = P.kb / kChunk, chunks = (P.kb + kChunk - 1) / kChunk;
  for (int64_t c = w; c < chunks; c += NW) {
    const uint8_t* const ab = abase + c * kRowBytes;
    const uint8_t* const bb = bbase + c * kRowBytes;
    const int64_t left = P.kb - c * kChunk;
    u2 sa[FM], sb[FN];
    if (c < full) {
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        // A's pieces past its last row hold rows that no output needs
        if (j >= kPiecesA || j * kPieceRows <= mlast) fetch_to_lds(j < kPiecesA ? ab : bb, off[j], to + j * kPiece);
      }
    } else {
      // the last, partial chunk: blocks past the end are zero
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        v4i x = {};
        if (fetch_block(j, lane) < left) x = *reinterpret_cast<const v4i*>((j < kPiecesA ? ab : bb) + off[j]);
        *reinterpret_cast<v4i*>(mine + j * kPiece + lane * 16) = x;
      }
    }
#pragma unroll
    for (int f = 0; f < FN; ++f) sb[f] = load_scales(bs[f] + c * kChunk, left);
#pragma unroll
    for (int f = 0; f < FM; ++f) sa[f] = load_scales(as[f] + c * kChunk, left);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
    for (int f = 0; f < FN; ++f) sb[f] = chunk_scales(sb[f], g);
#pragma unroll
    for (int f = 0; f < FM; ++f) sa[f] = chunk_scales(sa[f], g);
    auto step = [&](auto sc) {
      constexpr int S = decltype(sc)::value;
      v4i a[FM], b[FN];
#pragma unroll
      for (int f = 0; f < FM; ++f) a[f] = *reinterpret_cast<const v4i*>(mine + slot_of(f * kFrag + r, 2 * S + g));
#pragma unroll
      for (int f = 0; f < FN; ++f) b[f] = *reinterpret_cast<const v4i*>(mine + slot_of((FM + f) * kFrag + r, 2 * S + g));
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = mfma<S>(b[j], step_scales<S>(sb[j]), a[i], step_scales<S>(sa[i]), acc[i][j]);
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 3>{});
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read out before the next chunk lands there
  }
  __syncthreads();
  // Sum over the waves, one 32 x 32 fragment at a time.
  float* const part = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      if (i + j > 0) __syncthreads();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f4 x = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        *reinterpret_cast<f4*>(part + (w * kFrag + r) * T::kPartRow + 8 * q + 4 * g) = x;
      }
      __syncthreads();
      constexpr int kCols = Run<DT>::kCols, kRuns = kFrag / kCols;  // of a row
      static_assert(kFrag * kRuns <= 64 * NW, "a run per thread");
      const int row = threadIdx.x / kRuns, col = threadIdx.x % kRuns * kCols;
      const int64_t om = m0 + i * kFrag + row, on = n0 + j * kFrag + col;
      if (row < kFrag && om < P.m && on < P.n) {
        f4 x[kCols / 4] = {};
#pragma unroll
        for (int u = 0; u < NW; ++u)
#pragma unroll
          for (int q = 0; q < kCols / 4; ++q)
            x[q] += *reinterpret_cast<const f4*>(part + (u * kFrag + row) * T::kPartRow + col + 4 * q);
        float v[kCols];
#pragma unroll
        for (int q = 0; q < kCols; ++q) v[q] = x[q / 4][q % 4];
        if (whole_lines(P.out, P.ldo, Run<DT>::kElem)) store_run<DT, true>(P.out, om * P.ldo + on, P.n - on, v);
        else store_run<DT, false>(P.out, om * P.ldo + on, P.n - on, v);
      }
    }
}

// ------------------------------------------------------------------------
// Many output tiles: WM x WN waves, each with FM x FN fragments, share an
// output tile through LDS, two stages of one chunk each. A stage's codes are
// fetched while the stage before is multiplied, the loads between the products.
//
// Scales pass through registers, four chunks (a group) of a row at a time, a
// chunk per lane, a quarter of the rows per stage. A row's 8 bytes per stage
// alone would ask the L2 for a sector of every row in every stage (with that
// and a stage's codes fetched in its first two steps: 297 us at 8192 x 14336 x
// 4096 instead of 274). The loop holds no branch that the compiler sees
// (fetch_to_lds_if).
//
// Measured at 8192 x 14336 x 4096 with bf16 output: 243-256 us, 3.8-4.0
// PFLOP/s; the instruction alone reaches 6.4 on random codes and 5.6 with its
// operands read from LDS (power holds the clock at 1.85 GHz there). With 4096 x
// 4096 x 14336 (110.5 us where this took 247.5) that splits into 1.9 us a
// stage, 4.6 PFLOP/s, and 5 us a tile that no product covers (prologue and
// output; one block fills a CU's LDS): 37 of the 247 us. Between 3.9 and 5.6
// the matrix pipes wait; power does not explain it. 8 waves of 128 x 64 beat 4
// of 128 x 128 (274), whose one wave per SIMD shows every wait.
// ------------------------------------------------------------------------

constexpr int kGroupChunks = 4;

// One of four values by a uniform index, by value: selects over an array become
// an array in scratch memory, whose loads hold up the wave in every stage.
__device__ __forceinline__ uint32_t turn_of(uint32_t turn, uint32_t v0, uint32_t v1, uint32_t v2, uint32_t v3) {
  const uint32_t lo = turn & 1 ? v1 : v0, hi = turn & 1 ? v3 : v2;
  return turn & 2 ? hi : lo;
}

template <int FM, int FN, int WM, int WN>
struct Tile {
  static constexpr int kM = kFrag * FM * WM, kN = kFrag * FN * WN;
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr int kRows = kM + kN;                 // A's rows, then B's
  static constexpr int kLoads = kRows / kPieceRows / kWaves;  // pieces, per wave and stage
  static constexpr int kTurns = kGroupChunks;           // stages that fetch a group's scales
  static constexpr int kTurnRows = kRows / kTurns;      // whose scales a stage fetches
  static constexpr int kPend = kTurnRows * kGroupChunks / kThreads;  // in so many loads a lane
  static constexpr int kStage = kRows * kRowBytes;      // codes of a stage
  static constexpr int kPlane = kRows * kChunk;         // scales of a stage
  static constexpr int kOutRow = kFrag * FN + 4;        // floats, padded
  static constexpr int kOut = kWaves * kFrag * kOutRow * 4;
  static constexpr int kIn = 2 * kStage + 2 * kGroupChunks * kPlane;
  static constexpr int kLds = kIn > kOut ? kIn : kOut;
  static_assert(kLds <= 160 * 1024, "LDS of a CU");
  static_assert(kM % (kPieceRows * kWaves) == 0 && kN % (kPieceRows * kWaves) == 0, "a load's rows belong to one operand");
  static_assert(kM % kTurnRows == 0 && kN % kTurnRows == 0, "a turn's rows belong to one operand");
  static_assert(kWaves % 2 == 0, "the pieces of a wave have one parity, so one block per lane");
};

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
  const int lb = fetch_block(w, lane);
  uint32_t off[T::kLoads];
#pragma unroll
  for (int j = 0; j < T::kLoads; ++j) {
    int64_t row = (j * T::kWaves + w) * kPieceRows + (lane >> 3);
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
  const uint8_t* const sabase = P.a_scales + m0 * P.lda;
  const uint8_t* const sbbase = P.b_scales + n0 * P.ldb;
  uint32_t soff[T::kTurns][T::kPend];
#pragma unroll
  for (int j = 0; j < T::kTurns; ++j)
#pragma unroll
    for (int p = 0; p < T::kPend; ++p) {
      int64_t row = j * T::kTurnRows + p * (T::kTurnRows / T::kPend) + threadIdx.x / kGroupChunks;
      if (row >= T::kM) {
        row -= T::kM;
        soff[j][p] = static_cast<uint32_t>((row < nlast ? row : nlast) * P.ldb);
      } else {
        soff[j][p] = static_cast<uint32_t>((row < mlast ? row : mlast) * P.lda);
      }
    }

  // A partial last chunk is stage 0, so that every later stage is whole; there
  // is at least one whole chunk.
  const uint32_t part = P.kb % kChunk, whole = P.kb / kChunk, stages = whole + (part != 0);
  const uint32_t first = part ? 1 : 0;  // the stage of chunk 0
  const uint32_t lds0 = lds_address(lds);
  uint8_t* const planes = lds + 2 * T::kStage;
  // Chunk c's scales stand in plane c % 8, the partial chunk's in plane 4 until
  // the chunk that needs it.
  constexpr int kPartPlane = kGroupChunks;
  auto plane = [&](uint32_t c) -> uint8_t* { return planes + c % (2 * kGroupChunks) * T::kPlane; };
  // Turn `turn` of group q: lane l of four fetches chunk 4 q + l (the last whole
  // one again where there are fewer; nothing uses that copy).
  u2 pend[T::kPend];
  auto fetch_scales = [&](uint32_t q, uint32_t turn, u2* to) {
    const uint32_t want = q * kGroupChunks + threadIdx.x % kGroupChunks;
    const uint32_t at = (want < whole ? want : whole - 1) * kChunk;
    const uint8_t* base = sabase;
#pragma unroll
    for (int j = 1; j < T::kTurns; ++j) base = turn == j ? (j * T::kTurnRows < T::kM ? sabase : sbbase) : base;
#pragma unroll
    for (int p = 0; p < T::kPend; ++p) {
      const uint32_t row = turn_of(turn, soff[0][p], soff[1][p], soff[2][p], soff[3][p]);
      __builtin_memcpy(&to[p], base + (row + at), kChunk);
    }
  };
  auto store_scales = [&](uint32_t q, uint32_t turn, const u2* from) {
    uint8_t* const to = plane(q * kGroupChunks) + threadIdx.x % kGroupChunks * T::kPlane +
                        (turn * T::kTurnRows + threadIdx.x / kGroupChunks) * kChunk;
#pragma unroll
    for (int p = 0; p < T::kPend; ++p) *reinterpret_cast<u2*>(to + p * (T::kTurnRows / T::kPend) * kChunk) = from[p];
  };
  auto fetch = [&](uint32_t i, int j) {  // load j of stage i (a whole chunk), if there is that stage
    const uint32_t c = i - first;
    const uint8_t* const from = (j * T::kWaves * kPieceRows >= T::kM ? bbase : abase) + static_cast<uint64_t>(c) * kRowBytes;
    fetch_to_lds_if(i, stages, from, off[j], lds0 + (i & 1) * T::kStage + (j * T::kWaves + w) * kPiece);
  };
  // The fetched stage i (a whole chunk c), to every wave, with the scales that
  // the stage before asked for: turn (c - 1) % kTurns of the group after chunk
  // c - 1's. Then the next turn is asked for.
  auto publish = [&](uint32_t i) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    const uint32_t c = i - first, before = c + kGroupChunks - 1;
    store_scales(before / kGroupChunks, before % T::kTurns, pend);
    __syncthreads();
    fetch_scales(c / kGroupChunks + 1, c % T::kTurns, pend);
  };

  const int wm = w / WN, wn = w % WN;
  const int arow = wm * FM * kFrag + r, brow = T::kM + wn * FN * kFrag + r;
  v4i a[2][FM], b[2][FN];
  u2 ra[FM], rb[FN];  // a stage's scales as they stand in LDS
  u2 sa[FM], sb[FN];
  auto read_scales = [&](const uint8_t* at) {
#pragma unroll
    for (int f = 0; f < FM; ++f) ra[f] = *reinterpret_cast<const u2*>(at + (arow + f * kFrag) * kChunk);
#pragma unroll
    for (int f = 0; f < FN; ++f) rb[f] = *reinterpret_cast<const u2*>(at + (brow + f * kFrag) * kChunk);
  };
  auto own_scales = [&]() {
#pragma unroll
    for (int f = 0; f < FM; ++f) sa[f] = chunk_scales(ra[f], g);
#pragma unroll
    for (int f = 0; f < FN; ++f) sb[f] = chunk_scales(rb[f], g);
  };
  // Fragment f of step s of stage i: B's first two, A's first, then the rest,
  // in the order in which the products need them.
  auto read = [&](uint32_t i, int s, int f) {
    // (a fragment's first row is a multiple of 32, so r alone gives the slot)
    const uint8_t* const at = lds + (i & 1) * T::kStage + ((2 * s + g) ^ (r >> 1 & 7)) * kMxCodeBytes;
    constexpr int kFirst = 2;
    if (f < kFirst) b[s & 1][f] = *reinterpret_cast<const v4i*>(at + (brow + f * kFrag) * kRowBytes);
    else if (f == kFirst) a[s & 1][0] = *reinterpret_cast<const v4i*>(at + arow * kRowBytes);
    else if (f <= FN) b[s & 1][f - 1] = *reinterpret_cast<const v4i*>(at + (brow + (f - 1) * kFrag) * kRowBytes);
    else a[s & 1][f - FN] = *reinterpret_cast<const v4i*>(at + (arow + (f - FN) * kFrag) * kRowBytes);
  };

  v16f acc[FM][FN] = {};
  constexpr int kGroups = FM * FN / 2;  // pairs of products per step
  constexpr int kReads = (FM + FN + kGroups - 1) / kGroups;            // per group
  constexpr int kLateReads = (FM + FN + kGroups - 2) / (kGroups - 1);  // per group of step 3 but its first
  constexpr int kFetches = (T::kLoads + 2 * kGroups) / (2 * kGroups + 1);
  // One step: per group two products and a few reads of the next step's
  // fragments, the order fixed so that reads and products leave in turn. Step 3
  // publishes the next stage behind its first group (every wave has read this
  // stage out by then) and starts fetching the one after it into this stage's
  // place; the next stage's first steps fetch the rest. Behind the last stage
  // the same happens without fetches, to no effect.
  auto step = [&](auto sc, uint32_t i) {
    constexpr int S = decltype(sc)::value;
    // the scales of this step, kept while the next stage's are read
    uint32_t ta[FM], tb[FN];
#pragma unroll
    for (int f = 0; f < FM; ++f) ta[f] = step_scales<S>(sa[f]);
#pragma unroll
    for (int f = 0; f < FN; ++f) tb[f] = step_scales<S>(sb[f]);
#pragma unroll
    for (int t = 0; t < kGroups; ++t) {
      if constexpr (S == 3) {
        if (t == 1) {
          publish(i + 1);
          read_scales(plane(i + 1 - first));
        }
      }
      const int slot = S == 3 ? t - 1 : kGroups - 1 + S * kGroups + t;
#pragma unroll
      for (int q = 0; q < kFetches; ++q)
        if (slot >= 0 && slot * kFetches + q < T::kLoads) fetch(i + (S == 3 ? 2 : 1), slot * kFetches + q);
      const int x = 2 * t / FN, y = 2 * t % FN;
      acc[x][y] = mfma<S>(b[S & 1][y], tb[y], a[S & 1][x], ta[x], acc[x][y]);
      acc[x][y + 1] = mfma<S>(b[S & 1][y + 1], tb[y + 1], a[S & 1][x], ta[x], acc[x][y + 1]);
      if constexpr (S < 3) {
#pragma unroll
        for (int q = 0; q < kReads; ++q)
          if (t * kReads + q < FM + FN) read(i, S + 1, t * kReads + q);
      } else {
        if (t > 0) {
#pragma unroll
          for (int q = 0; q < kLateReads; ++q)
            if ((t - 1) * kLateReads + q < FM + FN) read(i + 1, 0, (t - 1) * kLateReads + q);
        }
        if (t == kGroups - 1) own_scales();
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // The first stage's codes (the partial chunk's through registers, blocks past
  // the end zero) and group 0's scales, all in flight at once; the last turn's
  // are left for the first whole stage. Of the second stage what step 3 of the
  // stage before would have fetched.
  constexpr int kEarly = (kGroups - 1) * kFetches < T::kLoads ? (kGroups - 1) * kFetches : T::kLoads;
  constexpr int kOwnRows = (T::kRows + T::kThreads - 1) / T::kThreads;
  v4i part_codes[T::kLoads];
  u2 part_scales[kOwnRows], group[T::kTurns][T::kPend];
  if (part) {
#pragma unroll
    for (int j = 0; j < T::kLoads; ++j) {
      part_codes[j] = (v4i){};
      if (lb < static_cast<int>(part))
        part_codes[j] = *reinterpret_cast<const v4i*>((j * T::kWaves * kPieceRows >= T::kM ? bbase : abase) +
                                                      static_cast<uint64_t>(whole) * kRowBytes + off[j]);
    }
#pragma unroll
    for (int j = 0; j < kOwnRows; ++j) {
      const int row = j * T::kThreads + threadIdx.x < T::kRows ? j * T::kThreads + threadIdx.x : T::kRows - 1;
      const bool of_b = row >= T::kM;
      const int64_t i = of_b ? row - T::kM : row, last = of_b ? nlast : mlast;
      const uint8_t* const from = (of_b ? sbbase : sabase) + (i < last ? i : last) * (of_b ? P.ldb : P.lda);
      part_scales[j] = load_scales(from + static_cast<uint64_t>(whole) * kChunk, part);
    }
#pragma unroll
    for (int j = 0; j < kEarly; ++j) fetch(1, j);
  } else {
#pragma unroll
    for (int j = 0; j < T::kLoads; ++j) fetch(0, j);
  }
#pragma unroll
  for (int j = 0; j < T::kTurns; ++j) fetch_scales(0, j, group[j]);
#pragma unroll
  for (int j = 0; j < T::kTurns - 1; ++j) store_scales(0, j, group[j]);
#pragma unroll
  for (int p = 0; p < T::kPend; ++p) pend[p] = group[T::kTurns - 1][p];
  if (part) {
#pragma unroll
    for (int j = 0; j < T::kLoads; ++j)
      *reinterpret_cast<v4i*>(lds + (j * T::kWaves + w) * kPiece + lane * 16) = part_codes[j];
#pragma unroll
    for (int j = 0; j < kOwnRows; ++j) {
      const int row = j * T::kThreads + threadIdx.x;
      if (row < T::kRows) *reinterpret_cast<u2*>(plane(kPartPlane) + row * kChunk) = part_scales[j];
    }
    __syncthreads();
  } else {
    publish(0);
  }
  read_scales(part ? plane(kPartPlane) : plane(0));
  own_scales();
#pragma unroll
  for (int f = 0; f < FM + FN; ++f) read(0, 0, f);
  if (!part) {
#pragma unroll
    for (int j = 0; j < kEarly; ++j) fetch(1, j);
  }
  uint32_t i = 0;
  do {
    step(std::integral_constant<int, 0>{}, i);
    step(std::integral_constant<int, 1>{}, i);
    step(std::integral_constant<int, 2>{}, i);
    step(std::integral_constant<int, 3>{}, i);
  } while (++i < stages);
  __syncthreads();

  // 32 rows of the wave's part of the tile at a time, through LDS, so that a
  // row leaves in runs of 16 bytes a lane.
  float* const mine = reinterpret_cast<float*>(lds) + w * kFrag * T::kOutRow;
  auto write = [&](auto whole) {
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
      constexpr int kCols = Run<DT>::kCols, kRuns = kFrag * FN / kCols;  // of a row
#pragma unroll
      for (int t = 0; t < kFrag * kRuns / 64; ++t) {
        const int row = (t * 64 + lane) / kRuns, col = (t * 64 + lane) % kRuns * kCols;
        float v[kCols];
#pragma unroll
        for (int q = 0; q < kCols / 4; ++q) {
          const f4 x = *reinterpret_cast<const f4*>(mine + row * T::kOutRow + col + 4 * q);
          v[4 * q] = x.x;
          v[4 * q + 1] = x.y;
          v[4 * q + 2] = x.z;
          v[4 * q + 3] = x.w;
        }
        const int64_t om = m0 + (wm * FM + i) * kFrag + row, on = n0 + wn * FN * kFrag + col;
        if (om < P.m && on < P.n) store_run<DT, decltype(whole)::value>(P.out, om * P.ldo + on, P.n - on, v);
      }
      __builtin_amdgcn_wave_barrier();
    }
  };
  if (whole_lines(P.out, P.ldo, Run<DT>::kElem)) write(std::true_type{});
  else write(std::false_type{});
}

// Launch with more than the default limit of 64 KiB of dynamic LDS, granted once per kernel and device.
template <typename Kernel>
hipError_t launch_with_lds(Kernel kernel, int64_t tiles, int threads, int lds, std::atomic<uint64_t>& granted,
                           const MxProductArgs& a, hipStream_t s) {
  if (tiles > UINT32_MAX / threads) return hipErrorInvalidConfiguration;  // a launch counts its threads in 32 bits
  int dev = 0;
  if (hipError_t e = hipGetDevice(&dev)) return e;
  const uint64_t bit = uint64_t{1} << (dev & 63);
  if (dev > 63 || !(granted.load(std::memory_order_acquire) & bit)) {
    if (hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, lds))
      return e;
    granted.fetch_or(bit, std::memory_order_release);
  }
  hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(tiles)), dim3(threads), lds, s, a);
  return hipGetLastError();
}

template <int FM, int FN, int NW, int DT>
hipError_t split_launch(const MxProductArgs& a, hipStream_t s) {
  static std::atomic<uint64_t> granted{0};
  return launch_with_lds(mx_product_split_kernel<FM, FN, NW, DT>, mx_tiles(a.m, kFrag * FM) * mx_tiles(a.n, kFrag * FN),
                         64 * NW, Split<FM, FN, NW>::kLds, granted, a, s);
}

template <int FM, int FN, int WM, int WN, int DT>
hipError_t tile_launch(const MxProductArgs& a, hipStream_t s) {
  using T = Tile<FM, FN, WM, WN>;
  static std::atomic<uint64_t> granted{0};
  return launch_with_lds(mx_product_tile_kernel<FM, FN, WM, WN, DT>, mx_tiles(a.m, T::kM) * mx_tiles(a.n, T::kN),
                         T::kThreads, T::kLds, granted, a, s);
}

// The largest tile of which there are enough to keep the 256 CUs busy, and for
// a few tiles the waves of a block split the contraction. Measured (us, K =
// 4096, the variant taken and its neighbour): 4096 x 3100, 208 tiles of 256^2:
// 40 against 50 (128^2); 4096 x 2048, 128 tiles: 30 (128^2) against 34; 1000 x
// 4096, 256 tiles of 128^2: 20 against 26 (64^2); 700 x 2500, 120 tiles: 15
// (64^2) against 18; 300 x 2000, 160 tiles of 64^2: 9.7 against 10.1 (32^2);
// 100 x 4096, 128 tiles: 7.3 (32^2) against 9.8. The tiles' loop needs a whole
// chunk. Eight waves a block leave room for two blocks on a CU, four for four:
// 1 x 14336, 448 tiles of 32^2: 7.8 with four waves against 8.4 with eight;
// 1 x 4096 at K = 14336, 128 tiles: 8.8 with eight against 13.1 with four.
constexpr int64_t kEnoughTiles = 160;
constexpr int64_t kCus = 256;

template <int DT>
hipError_t product_launch(const MxProductArgs& a, hipStream_t s) {
  auto tiles = [&](int64_t side) { return mx_tiles(a.m, side) * mx_tiles(a.n, side); };
  const int64_t side = a.m < a.n ? a.m : a.n;  // a tile has more than half its rows and columns to do
  if (a.kb >= kChunk && side > 128 && tiles(256) >= kEnoughTiles) return tile_launch<4, 2, 2, 4, DT>(a, s);
  if (a.kb >= kChunk && side > 64 && tiles(128) >= kEnoughTiles) return tile_launch<2, 2, 2, 2, DT>(a, s);
  if (side > 32 && tiles(64) >= kEnoughTiles) return split_launch<2, 2, 4, DT>(a, s);
  return tiles(32) > kCus ? split_launch<1, 1, 4, DT>(a, s) : split_launch<1, 1, 8, DT>(a, s);
}

}  // namespace

hipError_t launch_mx_product(const MxProductArgs& a, int32_t dt, hipStream_t s) {
  if (dt == ZERO_DT_F32) return product_launch<ZERO_DT_F32>(a, s);
  if (dt == ZERO_DT_F16) return product_launch<ZERO_DT_F16>(a, s);
  if (dt == ZERO_DT_BF16) return product_launch<ZERO_DT_BF16>(a, s);
  return hipErrorInvalidValue;
}

}  // namespace zdp
