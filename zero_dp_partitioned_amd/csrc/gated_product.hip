// gfx950 kernels of a gated feed-forward block's first half and its gradients,
//   g = x wg^T,  u = x wu^T,  h = act(g) * u,
//   dg = dh act'(g) u,  du = dh act(g),
//   dx = dg wg + du wu,  dwg = dg^T x,  dwu = du^T x,
// in fp16 or bf16 on v_mfma_f32_16x16x32 (fp32 sums). The products are three
// uses of one tile kernel, which differ in how their operands lie in memory:
//   forward  A = x, B = wg and wu side by side: contraction along the rows of both;
//   dx       A = dg then du, along its rows; B = wg then wu, along its columns;
//   dw       A = dg or du, B = x, along the columns of both.
// Operands reach LDS as they lie. An operand along the rows is read back 16
// bytes a lane; one along the columns through ds_read_b64_tr_b16, which
// transposes 4 x 16 values on the way, so no transposed copy is ever made.
#include <atomic>
#include <type_traits>

#include "gated_route.h"
#include "layer_device.h"

namespace zdp {
namespace {

typedef short s4 __attribute__((ext_vector_type(4)));
typedef short s8 __attribute__((ext_vector_type(8)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));

// How operands reach LDS: kDirect by fetches that write it themselves (every
// 16-byte slot of the operands aligned and whole), kStaged through registers
// (aligned to elements), kMasked value by value (a dimension smaller than the tile).
enum Fetch { kDirect, kStaged, kMasked };

constexpr int kFrag = 16;      // rows of an operand per instruction
constexpr int kSteps = 2;      // of 32, per chunk
constexpr int kPiece = 1024;   // bytes that a wave moves at a time
constexpr int kPieceRows = 8;  // rows, or as much of the contraction as a piece's columns leave, of a piece

struct ProductArgs {
  const char* a[2];
  const char* b[2];
  int64_t a_ld, b_ld;  // bytes from row to row
  int64_t m, n, k;     // rows and columns of an output; contraction (of one of dx's two parts)
  void* out[3];
  int64_t out_ld[3];
  int32_t act, accumulate;
  bool dry;        // launch nothing, say whether a launch holds the tiles
  int32_t splits;  // blocks that share a tile's contraction, each leaving fp32 sums at `partial`
  float* partial;  // [splits][outputs][m][n]
};

// ------------------------------------------------------------------------
// The activation and its derivative. exp and 1 / x are the hardware's: within
// (|x| + 4) 2^-24 of themselves, far inside the 16-bit results' rounding, as far
// as fp32's normal values go. The hardware's exp flushes what is smaller, and
// exp(-x) overflows where exp(x) is; bf16 results (silu(-90) is -7e-38) need values
// there. So far exponents are cut by kFar first and the result multiplied by
// exp(-kFar), which rounds at a subnormal's last bit.
// ------------------------------------------------------------------------

constexpr float kFar = 64.f, kExpFar = 1.6038108905486378e-28f;  // exp(-64)

// exp(-x) for x >= 0.
__device__ __forceinline__ float exp_minus(float x) {
  const bool far = x > kFar;
  const float e = __expf(far ? kFar - x : -x);
  return far ? e * kExpFar : e;
}

__device__ __forceinline__ float sigmoid(float x) {
  const bool far = x < -kFar;
  const float e = __expf(far ? x + kFar : -x);
  return far ? e * kExpFar : __builtin_amdgcn_rcpf(1.f + e);
}

constexpr float kTanhA = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kTanhB = 0.044715f;

__device__ __forceinline__ float activation(float g, int32_t act) {
  switch (act) {
    case ZERO_ACT_SILU: return g * sigmoid(g);
    case ZERO_ACT_GELU: return 0.5f * g * erfcf(-0.70710678118654752f * g);
    case ZERO_ACT_GELU_TANH: return g * sigmoid(kTanhA * g * __builtin_fmaf(kTanhB * g, g, 1.f));
    case ZERO_ACT_RELU: return g <= 0.f ? 0.f : g;  // NaN stays
    default: return sigmoid(g);
  }
}

__device__ __forceinline__ void activation_grad(float g, int32_t act, float* a, float* da) {
  switch (act) {
    case ZERO_ACT_SILU: {
      const float s = sigmoid(g), r = sigmoid(-g);
      *a = g * s;
      *da = __builtin_fmaf(*a, r, s);
      return;
    }
    case ZERO_ACT_GELU: {
      const float c = 0.5f * erfcf(-0.70710678118654752f * g);
      *a = g * c;
      *da = __builtin_fmaf(0.3989422804014327f * g, exp_minus(0.5f * g * g), c);
      return;
    }
    case ZERO_ACT_GELU_TANH: {
      const float z = kTanhA * g * __builtin_fmaf(kTanhB * g, g, 1.f), s = sigmoid(z), r = sigmoid(-z);
      // past 64 one of s and r is 0, and so is the term with the slope of z, which
      // g's own square would make 0 times infinity from 5e19 on
      const float c = __builtin_fminf(__builtin_fmaxf(g, -64.f), 64.f);
      *a = g * s;
      *da = __builtin_fmaf(*a * r, kTanhA * __builtin_fmaf(3.f * kTanhB * c, c, 1.f), s);
      return;
    }
    case ZERO_ACT_RELU:
      *a = g <= 0.f ? 0.f : g;
      *da = g <= 0.f ? 0.f : 1.f;
      return;
    default: {
      const float s = sigmoid(g);
      *a = s;
      *da = s * sigmoid(-g);
    }
  }
}

// ------------------------------------------------------------------------
// Pieces of the tile kernel
// ------------------------------------------------------------------------

template <int DT>
__device__ __forceinline__ f4 mfma(s8 b, s8 a, f4 c) {
  if constexpr (DT == ZERO_DT_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, b), __builtin_bit_cast(b8, a), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, b), __builtin_bit_cast(h8, a), c, 0, 0, 0);
}

__device__ __forceinline__ s8 read16(uint32_t lds) {
  return *reinterpret_cast<const __attribute__((address_space(3))) s8*>(lds);
}

__device__ __forceinline__ s4 read_tr(uint32_t lds) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<__attribute__((address_space(3))) s4*>(lds));
}

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void*)p));
}

// m0 is named as overwritten, so that the compiler keeps no value of its own
// there across a fetch. It warns about every such list because it reserves m0
// and cannot save it; nothing needs it saved.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"

// If i < n (uniform): fetch 16 bytes a lane from base + off into LDS at `lds` +
// 16 * lane. No vector register is written; the caller waits on vmcnt. The
// branch is the asm's own, as one that the compiler sees would split the loop
// around it; compare and branch are the wait state that the hardware wants
// between the write of m0 and the load that takes its LDS base from it.
__device__ __forceinline__ void fetch_to_lds_if(uint32_t i, uint32_t n, const char* base, uint32_t off, uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %0\n\ts_cmp_ge_u32 %3, %4\n\ts_cbranch_scc1 .Lzdp_skip%=\n\t"
      "global_load_lds_dwordx4 %1, %2\n.Lzdp_skip%=:" ::"s"(lds), "v"(off), "s"(base), "s"(i), "s"(n)
      : "memory", "scc", "m0");
}

#pragma clang diagnostic pop

// Tiles dealt to the eight XCDs (block b runs on XCD b % 8) in contiguous
// runs, and inside a run in columns of kGroup tile rows, so that the tiles that
// an XCD's 32 CUs work on at a time share their operands in its L2.
template <uint32_t kGroup>
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

// An operand of SIZE rows (or columns) in LDS, kChunk of the contraction.
//
// Along the rows: rows of 128 bytes, eight slots of 16; slot b of row i stands
// at b ^ (i / 2) % 8, so that one slot of 16 neighbouring rows lies in 16
// different groups of four of the 64 banks.
//
// Along the columns: SIZE columns side by side, kChunk lines of them. A
// transposing read takes 8 bytes a lane, four lines of 32 bytes for 16 lanes;
// slot b of line k stands at b ^ mix(k), so that the lines which are read
// together lie in different banks.
template <int SIZE, bool COLS>
struct Operand {
  static constexpr int kBytes = SIZE * kChunk * 2;
  static constexpr int kSlots = COLS ? SIZE / 8 : 8;  // of a line
  static constexpr int kLine = kSlots * 16;
  static constexpr int kPieceLines = kPiece / kLine;

  static __device__ __forceinline__ int mix(int line) {
    if constexpr (!COLS) return line >> 1 & 7;
    else if constexpr (kSlots >= 16) return (line & 3) << 2 | (line >> 3 & 1) << 1;
    else return (line >> 1 & 1) << 2 | (line >> 3 & 1) << 1;
  }
  // The line and slot (of 8 values) that lane `lane` of piece p moves.
  static __device__ __forceinline__ int line(int p, int lane) { return p * kPieceLines + lane / kSlots; }
  static __device__ __forceinline__ int slot(int p, int lane) { return (lane % kSlots) ^ mix(line(p, lane)); }

  // Where a lane reads fragment rows (columns) first .. first + 15 of step 0;
  // `first` is a multiple of 16.
  static __device__ __forceinline__ uint32_t fragment(int first, int lane) {
    if constexpr (!COLS) {
      return (first + (lane & 15)) * kLine + ((lane >> 4) ^ mix(lane & 15)) * 16;
    } else {
      const int k = 8 * (lane >> 4) + (lane >> 2 & 3);
      return k * kLine + ((first / 8 + (lane >> 1 & 1)) ^ mix(k)) * 16 + (lane & 1) * 8;
    }
  }
  static __device__ __forceinline__ s8 read(uint32_t at, int step) {
    if constexpr (!COLS) {
      return read16(at ^ (step * 64));  // slots 4 * step + ...: the mix is an exclusive or
    } else {
      const s4 lo = read_tr(at + step * 32 * kLine), hi = read_tr(at + (step * 32 + 4) * kLine);
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
};

// ------------------------------------------------------------------------
// The tile kernel: WM x WN waves, each with FM x FN fragments, share an output
// tile through LDS in stages of one chunk, NB of them: one is multiplied while the
// others are fetched, the loads between the products. KG groups of such waves may
// share the contraction, each with stages of its own. The rows of B of
// a forward tile are, wave column by wave column, FN / 2 fragments of wg and the
// same of wu, so that a lane holds g and u of the same outputs.
// ------------------------------------------------------------------------

template <Use USE, int FM, int FN, int WM, int WN, int kBuffers = 2, int kGroups = 1>
struct Tile {
  static constexpr int kM = kFrag * FM * WM, kN = kFrag * FN * WN;
  static constexpr int kOutN = USE == kForward ? kN / 2 : kN;  // columns of an output
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves * kGroups;  // waves of a group, threads of a block
  using A = Operand<kM, USE == kDw>;
  using B = Operand<kN, USE != kForward>;
  static constexpr int kPiecesA = A::kBytes / kPiece, kPiecesB = B::kBytes / kPiece;
  static constexpr int kLoadsA = kPiecesA / kWaves, kLoads = (kPiecesA + kPiecesB) / kWaves;
  static constexpr int kStage = A::kBytes + B::kBytes;
  static constexpr int kRunN = kOutN / WN;  // columns of a wave's output
  static constexpr int kOutRow = kRunN + 4;  // floats, padded
  static constexpr int kOut = kWaves * 2 * kFrag * kOutRow * 4;
  static constexpr int kShared = kWaves * FM * FN * 1024;  // a group's sums
  static constexpr int kIn = kGroups * kBuffers * kStage, kEnd = (kGroups - 1) * kShared > kOut ? (kGroups - 1) * kShared : kOut;
  static constexpr int kLds = kIn > kEnd ? kIn : kEnd;
  static_assert(kLds <= 160 * 1024, "LDS of a CU");
  static_assert(kPiecesA % kWaves == 0 && kPiecesB % kWaves == 0, "a load's pieces belong to one operand");
};

__device__ __forceinline__ uint32_t tiles_of(int64_t n, uint32_t size) { return static_cast<uint32_t>((n + size - 1) / size); }

// Registers: two waves a SIMD (256 each) for the largest tile, of which one
// block fills a CU; more blocks of the smaller ones.
//
// What bounds the large tile (256 x 256, eight waves of 128 x 64 or 64 x 128) is
// power: 8192 x 4096 x 14336 in bf16 takes 1375-1470 us (1.31-1.40 PFLOP/s), dx
// 1340-1410, dw 1380-1430 on several cards, at 1.5-1.9 GHz; with the wait for
// fetches left out it took 1-2 % less. The instruction alone reaches 2.08 PFLOP/s on
// such values (32 x 32 x 16: 1.83, and the kernel was 2-3 % slower with it). Four
// waves of 128 x 128, which read a third less from LDS, were 5 % slower for dw: one
// wave a SIMD shows every wait. Higher priority for one wave of each SIMD, or around
// the products, changed 1 % either way.
template <Use USE, Fetch FETCH, int FM, int FN, int WM, int WN, int NB, int KG, int DT, int ODT>
__device__ __forceinline__ void gated_tile(const ProductArgs& P, uint32_t block, uint8_t* lds) {
  using T = Tile<USE, FM, FN, WM, WN, NB, KG>;
  using A = typename T::A;
  using B = typename T::B;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = KG > 1 ? wave / T::kWaves : 0, w = KG > 1 ? wave % T::kWaves : wave;
  const uint32_t tiles_m = tiles_of(P.m, T::kM), tiles_n = tiles_of(P.n, T::kOutN);
  const uint32_t rows = USE == kDw ? 2 * tiles_m : tiles_m;  // dwu's tiles behind dwg's
  const uint32_t split = P.splits > 1 ? block / (rows * tiles_n) : 0;
  uint32_t tm, tn;
  // (4 or 8 tile rows a group, us at 8192 x 4096 x 14336: forward 1457 or 1414, dx 1416 or 1365, dw 1379 or 1439)
  tile_of<USE == kDw ? 4 : 8>(P.splits > 1 ? block % (rows * tiles_n) : block, rows, tiles_n, &tm, &tn);
  const int z = USE == kDw && tm >= tiles_m;  // which output
  if (z) tm -= tiles_m;
  // The tile's first row and column, and the first of the operands': along the
  // columns the last tile is moved back to end with the operand, so that every
  // load is whole; what the tile before has is not written again.
  const int64_t m0 = static_cast<int64_t>(tm) * T::kM, n0 = static_cast<int64_t>(tn) * T::kOutN;
  int64_t am0 = m0, bn0 = n0;
  if (FETCH != kMasked) {
    if (USE == kDw && am0 > P.m - T::kM) am0 = P.m - T::kM;
    if (USE != kForward && bn0 > P.n - T::kN) bn0 = P.n - T::kN;
  }

  // The contraction: `parts` runs of `whole` chunks, of which this block takes
  // [c0, c0 + stages); what is left of a run behind its last whole chunk goes
  // first, to split 0.
  constexpr int kParts = USE == kDx ? 2 : 1;
  const uint32_t rest = FETCH == kMasked ? 0 : static_cast<uint32_t>(P.k % kChunk);
  const uint32_t whole = static_cast<uint32_t>(FETCH == kMasked ? (P.k + kChunk - 1) / kChunk : P.k / kChunk);
  const uint32_t all = kParts * whole;
  const uint32_t c0 = P.splits > 1 ? static_cast<uint32_t>(static_cast<uint64_t>(all) * split / P.splits) : 0;
  const uint32_t c1 = P.splits > 1 ? static_cast<uint32_t>(static_cast<uint64_t>(all) * (split + 1) / P.splits) : all;
  // Each of the block's groups takes as many chunks; those that do not divide
  // stand first and go to group 0, one by one.
  const uint32_t loose = (c1 - c0) % KG, stages = (c1 - c0) / KG, first = c0 + loose + group * stages;

  // Load j of a wave: a piece of A (j < kLoadsA) or B. Where its lanes start,
  // from the operand's first row (column) of the tile.
  uint32_t off[T::kLoads];
  // (scalars: selects over an array become an array in scratch memory)
  const int64_t atile = USE == kDw ? am0 * 2 : m0 * P.a_ld, btile = USE == kForward ? n0 * P.b_ld : bn0 * 2;
  const char* const a0 = (z ? P.a[1] : P.a[0]) + atile;
  const char* const a1 = USE == kDx ? P.a[1] + atile : a0;
  const char* const b0 = P.b[0] + btile;
  const char* const b1 = USE == kDw ? b0 : P.b[1] + btile;
  const int64_t astep = USE == kDw ? kChunk * P.a_ld : kChunk * 2, bstep = USE == kForward ? kChunk * 2 : kChunk * P.b_ld;
  auto piece = [&](int j) { return j < T::kLoadsA ? j * T::kWaves + w : (j - T::kLoadsA) * T::kWaves + w; };
  // Row of B's operand in wg or wu that LDS row `row` holds, and which of them.
  constexpr int kHalf = kFrag * FN / 2;
  auto weight_row = [&](int row) { return row / (2 * kHalf) * kHalf + row % kHalf; };
  auto weight_of = [&](int row) { return row / kHalf & 1; };
#pragma unroll
  for (int j = 0; j < T::kLoads; ++j) {
    const bool is_a = j < T::kLoadsA;
    const int line = is_a ? A::line(piece(j), lane) : B::line(piece(j), lane);
    const int slot = is_a ? A::slot(piece(j), lane) : B::slot(piece(j), lane);
    int64_t row = line;  // rows past the end repeat the last one
    if (is_a && USE != kDw) row = row < P.m - 1 - m0 ? row : P.m - 1 - m0;
    if (!is_a && USE == kForward) {
      row = weight_row(line);
      row = row < P.n - 1 - n0 ? row : P.n - 1 - n0;
    }
    off[j] = static_cast<uint32_t>(row * (is_a ? P.a_ld : P.b_ld) + slot * 16);
  }
  // One of two uniform pointers, by arithmetic: a select may end in vector
  // registers, and a fetch takes its base from scalar ones.
  auto pick = [](uint32_t second, const char* p0, const char* p1) {
    return p0 + (-static_cast<int64_t>(second) & (p1 - p0));
  };
  // Where load j of chunk c starts.
  auto from = [&](uint32_t c, int j) -> const char* {
    const uint32_t part = kParts == 2 && c >= whole;
    const uint64_t at = part ? c - whole : c;
    if (j < T::kLoadsA) return pick(part, a0, a1) + at * astep;
    return pick(USE == kForward ? weight_of(piece(j) * kPieceRows) : part, b0, b1) + at * bstep;
  };
  // The lane's 16 bytes of load j of a chunk that is not whole, or of an operand
  // smaller than the tile: what does not exist is zero.
  auto masked = [&](uint32_t part, uint32_t at, int j) -> u4 {
    const bool is_a = j < T::kLoadsA, cols = is_a ? USE == kDw : USE != kForward;
    const int line = is_a ? A::line(piece(j), lane) : B::line(piece(j), lane);
    const int slot = is_a ? A::slot(piece(j), lane) : B::slot(piece(j), lane);
    const char* base = is_a ? pick(part, a0, a1) : pick(USE == kForward ? weight_of(piece(j) * kPieceRows) : part, b0, b1);
    base += static_cast<uint64_t>(at) * (is_a ? astep : bstep) + off[j];
    const int64_t k0 = static_cast<int64_t>(at) * kChunk;
    int64_t left;
    if (cols) left = k0 + line < P.k ? (is_a ? P.m - am0 : P.n - bn0) - slot * 8 : 0;
    else left = P.k - k0 - slot * 8;
    u4 x = {0, 0, 0, 0};
    if (left > 0) x = load_part<DT>(base, left);
    return x;
  };
  uint8_t* const space = lds + group * (FETCH == kDirect ? NB : 2) * T::kStage;  // the group's
  auto put = [&](int buffer, int j, u4 x) {
    *reinterpret_cast<u4*>(space + buffer * T::kStage + (j < T::kLoadsA ? 0 : A::kBytes) + piece(j) * kPiece + lane * 16) = x;
  };

  const int wm = w / WN, wn = w % WN;
  const uint32_t lds0 = lds_address(space);
  uint32_t aat[FM], bat[FN];
#pragma unroll
  for (int f = 0; f < FM; ++f) aat[f] = lds0 + A::fragment((wm * FM + f) * kFrag, lane);
#pragma unroll
  for (int f = 0; f < FN; ++f) bat[f] = lds0 + A::kBytes + B::fragment((wn * FN + f) * kFrag, lane);
  // Of the operand with more fragments (`ring`) a few are held ahead of their
  // products, of the other one (`kept`) this step's and the next step's.
  constexpr bool kRingA = FM > FN;
  constexpr int kRing = kRingA ? FM : FN, kKept = kRingA ? FN : FM;
  constexpr int kHeld = 4;                     // fragments of the ring in registers
  constexpr int kAhead = kRing >= 8 ? 3 : 2;   // groups of products from a read to its use
  static_assert(kRing % kHeld == 0 && kAhead < kHeld, "");
  s8 ring[kHeld], kept[2][kKept];
  auto read_ring = [&](uint32_t buffer, int s, int f) {
    const uint32_t at = buffer * T::kStage;
    ring[f % kHeld] = kRingA ? A::read(aat[f % FM] + at, s) : B::read(bat[f % FN] + at, s);
  };
  auto read_kept = [&](uint32_t buffer, int s, int f) {
    const uint32_t at = buffer * T::kStage;
    kept[s & 1][f] = kRingA ? B::read(bat[f % FN] + at, s) : A::read(aat[f % FM] + at, s);
  };
  f4 acc[FM][FN] = {};
  auto product = [&](int s, int r, int k) {
    const int x = kRingA ? r : k, y = kRingA ? k : r;
    const s8 av = kRingA ? ring[r % kHeld] : kept[s & 1][k], bv = kRingA ? kept[s & 1][k] : ring[r % kHeld];
    acc[x][y] = mfma<DT>(bv, av, acc[x][y]);
  };

  // What is left behind the whole chunks, one run after the other, and the loose chunks.
  const int rests = FETCH != kMasked && rest && split == 0 ? kParts : 0;
  if (KG > 1 ? rests + static_cast<int>(loose) > 0 : rests > 0) {
#pragma unroll 1
    for (int q = 0; q < rests + (KG > 1 ? static_cast<int>(loose) : 0); ++q) {
      if (q) __syncthreads();  // read out
      if (group == 0) {
        const bool is_rest = KG == 1 || q < rests;
        const uint32_t c = c0 + q - rests;
        const uint32_t part = is_rest ? q : kParts == 2 && c >= whole;
        const uint32_t at = is_rest ? whole : (part ? c - whole : c);
        u4 x[T::kLoads];
#pragma unroll
        for (int j = 0; j < T::kLoads; ++j) x[j] = masked(part, at, j);
#pragma unroll
        for (int j = 0; j < T::kLoads; ++j) put(1, j, x[j]);
      }
      __syncthreads();
      if (group == 0) {
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
#pragma unroll
          for (int k = 0; k < kKept; ++k) read_kept(1, s, k);
#pragma unroll
          for (int r = 0; r < kRing; ++r) {
            read_ring(1, s, r);
#pragma unroll
            for (int k = 0; k < kKept; ++k) product(s, r, k);
          }
        }
      }
    }
    __syncthreads();
  }

  if (stages) {
    u4 pend[FETCH == kDirect ? 1 : T::kLoads];
    // Load j of stage i: into LDS if there is that stage, or (the last stage
    // again past the end) into registers.
    constexpr uint32_t kBuffers = FETCH == kDirect ? NB : 2;
    uint32_t buffer = 0;  // of the stage that is worked on
    auto buffer_of = [&](uint32_t ahead) {  // of the stage `ahead` of it
      const uint32_t b = buffer + ahead;
      return b < kBuffers ? b : b - kBuffers;
    };
    auto fetch = [&](uint32_t i, int j, uint32_t to) {
      if constexpr (FETCH == kDirect) {
        const uint32_t c = first + i;
        fetch_to_lds_if(i, stages, from(c, j), off[j],
                        lds0 + to * T::kStage + (j < T::kLoadsA ? 0 : A::kBytes) + piece(j) * kPiece);
      } else {
        const uint32_t c = first + (i < stages ? i : stages - 1);
        if constexpr (FETCH == kStaged) pend[j] = load_any(from(c, j) + off[j]);
        else pend[j] = masked(kParts == 2 && c >= whole, kParts == 2 && c >= whole ? c - whole : c, j);
      }
    };
    // Stage i, fetched into buffer `to`, to every wave. All of them have read out
    // the stage that was there before. Up to kBuffers - 2 younger stages stay in flight.
    auto publish = [&](uint32_t i, uint32_t to) {
      if constexpr (FETCH == kDirect) {
        constexpr int kYounger = (kBuffers - 2) * T::kLoads;
        if constexpr (kYounger > 0)
          asm volatile(
              "s_waitcnt vmcnt(%2)\n\ts_cmp_lt_u32 %0, %1\n\ts_cbranch_scc1 .Lzdp_some%=\n\ts_waitcnt vmcnt(0)\n.Lzdp_some%=:" ::"s"(
                  i + kBuffers - 2),
              "s"(stages), "i"(kYounger)
              : "memory", "scc");
        else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      } else {
#pragma unroll
        for (int j = 0; j < T::kLoads; ++j) put(to, j, pend[j]);
      }
      __syncthreads();
    };
    // A step is a group of products for each fragment of the ring, and with each
    // group the ring's fragment that is kAhead groups away is read, and some of
    // the next step's kept ones; the order is fixed. Once the last step's own
    // fragments have been asked for (group kTurn), the next stage is published,
    // and what follows is read from there; the fetches of the stage after it
    // start into this stage's place, one a group, and run on into the next
    // stage's first step; those that pass through registers, which publishing has
    // just emptied, at the same time.
    constexpr int kTurn = kRing - kAhead;
    auto step = [&](auto sc, uint32_t i) {
      constexpr int S = decltype(sc)::value;
      constexpr bool kLast = S == kSteps - 1;
#pragma unroll
      for (int t = 0; t < kRing; ++t) {
        if (kLast && t == kTurn) publish(i + 1, buffer_of(1));
        constexpr int kEach = (T::kLoads + kRing - 1) / kRing;
        const int slot = kLast ? t - kTurn : kAhead + S * kRing + t;
#pragma unroll
        for (int q = 0; q < kEach; ++q)
          if (slot >= 0 && slot * kEach + q < T::kLoads)
            fetch(i + kBuffers - (kLast ? 0 : 1), slot * kEach + q, kLast ? buffer : buffer_of(kBuffers - 1));
#pragma unroll
        for (int k = 0; k < kKept; ++k) product(S, t, k);
        const bool next = kLast && t >= kTurn;  // the next stage's
        read_ring(next ? buffer_of(1) : buffer, t < kTurn ? S : (S + 1) % kSteps, (t + kAhead) % kRing);
        constexpr int kFirst = kLast ? kTurn : 0, kSpan = kLast ? kAhead - 1 : kRing - 1;  // groups with reads of kept ones
#pragma unroll
        for (int k = 0; k < kKept; ++k)
          if (k * kSpan / kKept == t - kFirst) read_kept(next ? buffer_of(1) : buffer, (S + 1) % kSteps, k);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
#pragma unroll
    for (uint32_t q = 0; q < kBuffers - 1; ++q)
#pragma unroll
      for (int j = 0; j < T::kLoads; ++j) fetch(q, j, q);
    publish(0, 0);
#pragma unroll
    for (int k = 0; k < kKept; ++k) read_kept(0, 0, k);
#pragma unroll
    for (int r = 0; r < kAhead; ++r) read_ring(0, 0, r);
    constexpr int kEarly = kAhead * ((T::kLoads + kRing - 1) / kRing);
#pragma unroll
    for (int j = 0; j < (kEarly < T::kLoads ? kEarly : T::kLoads); ++j) fetch(kBuffers - 1, j, kBuffers - 1);
    uint32_t i = 0;
    do {
      step(std::integral_constant<int, 0>{}, i);
      step(std::integral_constant<int, 1>{}, i);
      buffer = buffer_of(1);
    } while (++i < stages);
    __syncthreads();
  }

  // The other groups' sums, added in their order.
  if constexpr (KG > 1) {
    f4* const shared = reinterpret_cast<f4*>(lds) + w * FM * FN * 64 + lane;
    constexpr int kEach = T::kShared / 16;
    if (group > 0) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) shared[(group - 1) * kEach + (i * FN + j) * 64] = acc[i][j];
    }
    __syncthreads();
    if (group == 0) {
#pragma unroll 1
      for (int q = 0; q < KG - 1; ++q)
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j) acc[i][j] += shared[q * kEach + (i * FN + j) * 64];
    }
    __syncthreads();  // the rows below go through the same LDS
    if (group > 0) return;
  }

  // 32 rows of the wave's part of the tile at a time, through LDS, so that a row
  // leaves in runs of 16 bytes a lane. A lane holds columns 4 (lane / 16) + 0..3
  // of row lane % 16 of a fragment.
  constexpr int kBatch = 2;  // fragments
  float* const mine = reinterpret_cast<float*>(lds) + w * kBatch * kFrag * T::kOutRow;
  auto rows_out = [&](auto type, int i, void* out, int64_t ld, bool add, auto&& value) {
    constexpr int O = decltype(type)::value, kVals = Vec<O>::kVals, kElem = Vec<O>::kElem;
#pragma unroll
    for (int f = 0; f < kBatch; ++f)
#pragma unroll
      for (int j = 0; j < T::kRunN / kFrag; ++j) {
        f4 x;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = value(i + f, j, e);
        *reinterpret_cast<f4*>(mine + (f * kFrag + (lane & 15)) * T::kOutRow + j * kFrag + 4 * (lane >> 4)) = x;
      }
    __builtin_amdgcn_wave_barrier();
    constexpr int kRuns = T::kRunN / kVals;  // of a row
    // Runs of whole lines go past the caches (8192 x 4096 x 4096 with h, g and u
    // written: 435 -> 405 us; the products' operands keep their place there).
    const bool whole_lines = ((reinterpret_cast<uintptr_t>(out) | static_cast<uintptr_t>(ld * kElem) | static_cast<uintptr_t>(bn0 * kElem)) & 15) == 0;
#pragma unroll
    for (int t = 0; t < kBatch * kFrag * kRuns / 64; ++t) {
      const int row = (t * 64 + lane) / kRuns, col = (t * 64 + lane) % kRuns * kVals;
      float v[kVals];
#pragma unroll
      for (int q = 0; q < kVals / 4; ++q) {
        const f4 x = *reinterpret_cast<const f4*>(mine + row * T::kOutRow + col + 4 * q);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * q + e] = x[e];
      }
      const int64_t om = am0 + (wm * FM + i) * kFrag + row, on = bn0 + wn * T::kRunN + col;
      if (om < m0 || om >= P.m || on >= P.n || on + kVals <= n0) continue;
      char* const to = static_cast<char*>(out) + (om * ld + on) * kElem;
      const int first = on < n0 ? static_cast<int>(n0 - on) : 0;
      const int end = P.n - on < kVals ? static_cast<int>(P.n - on) : kVals;
      if (first == 0 && end == kVals) {
        if (add) {
          float old[kVals];
          widen<O>(load_any(to), old);
#pragma unroll
          for (int e = 0; e < kVals; ++e) v[e] += old[e];
        }
        const u4 x = narrow<O>(v);
        if (whole_lines) __builtin_nontemporal_store(x, reinterpret_cast<u4*>(to));
        else __builtin_memcpy(to, &x, 16);
      } else {
        if (add) {
#pragma unroll
          for (int e = 0; e < kVals; ++e)
            if (e >= first && e < end) v[e] += load_one(to, e, O);
        }
        store_some<O>(to, first, end, narrow<O>(v));
      }
    }
    __builtin_amdgcn_wave_barrier();
  };
  using Type = std::integral_constant<int, ODT>;
#pragma unroll
  for (int i = 0; i < FM; i += kBatch) {
    if constexpr (USE == kForward) {
      constexpr int H = FN / 2;
      f4 h[kBatch][H];
      // (one switch a batch: with one for each value 8192 x 64 x 14336 took 142 us with silu, 127 with relu, now 110 and 79)
      auto form = [&](auto act) {
#pragma unroll
        for (int f = 0; f < kBatch; ++f)
#pragma unroll
          for (int j = 0; j < H; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              h[f][j][e] = activation(acc[i + f][j][e], decltype(act)::value) * acc[i + f][j + H][e];
      };
      using std::integral_constant;
      switch (P.act) {
        case ZERO_ACT_SILU: form(integral_constant<int, ZERO_ACT_SILU>{}); break;
        case ZERO_ACT_GELU: form(integral_constant<int, ZERO_ACT_GELU>{}); break;
        case ZERO_ACT_GELU_TANH: form(integral_constant<int, ZERO_ACT_GELU_TANH>{}); break;
        case ZERO_ACT_RELU: form(integral_constant<int, ZERO_ACT_RELU>{}); break;
        default: form(integral_constant<int, ZERO_ACT_SIGMOID>{});
      }
      rows_out(Type{}, i, P.out[0], P.out_ld[0], false, [&](int at, int j, int e) { return h[at - i][j][e]; });
      if (P.out[1]) {
        rows_out(Type{}, i, P.out[1], P.out_ld[1], false, [&](int i, int j, int e) { return acc[i][j][e]; });
        rows_out(Type{}, i, P.out[2], P.out_ld[2], false, [&](int i, int j, int e) { return acc[i][j + H][e]; });
      }
    } else if (P.splits > 1) {
      float* const to = P.partial + (static_cast<int64_t>(split) * (USE == kDw ? 2 : 1) + z) * P.m * P.n;
      rows_out(std::integral_constant<int, ZERO_DT_F32>{}, i, to, P.n, false, [&](int i, int j, int e) { return acc[i][j][e]; });
    } else {
      rows_out(Type{}, i, P.out[z], P.out_ld[z], P.accumulate, [&](int i, int j, int e) { return acc[i][j][e]; });
    }
  }
}

template <Use USE, Fetch FETCH, int FM, int FN, int WM, int WN, int NB, int KG, int DT, int ODT>
__global__ void __launch_bounds__(64 * WM * WN * KG, 2) gated_tile_kernel(const ProductArgs P) {
  extern __shared__ __align__(1024) uint8_t lds[];
  gated_tile<USE, FETCH, FM, FN, WM, WN, NB, KG, DT, ODT>(P, blockIdx.x, lds);
}

// dx and dw in one launch, for sizes whose blocks fill neither's last round over
// the CUs: `first` blocks of dx's middle tiles (those behind `of_dx` have nothing to
// do, so that dw's blocks stand on the XCDs that their mapping expects), then dw's
// large ones. Either takes a CU's LDS.
template <int DT, int ODT>
__global__ void __launch_bounds__(512, 2) gated_pair_kernel(const ProductArgs X, const ProductArgs W, uint32_t of_dx,
                                                            uint32_t first) {
  extern __shared__ __align__(1024) uint8_t lds[];
  if (blockIdx.x >= first) gated_tile<kDw, kDirect, 8, 4, 2, 4, 2, 1, DT, ODT>(W, blockIdx.x - first, lds);
  else if (blockIdx.x < of_dx) gated_tile<kDx, kDirect, 2, 4, 4, 2, 4, 1, DT, DT>(X, blockIdx.x, lds);
}

// ------------------------------------------------------------------------
// Forward for very few rows, kTokens of them at most, which is one pass over the
// weights: a block takes 16 rows of wg and the same of wu. A wave takes runs of
// 512 of the contraction, 8 a lane, and goes through the block's rows, so that a
// load is one contiguous KiB of a row whatever its alignment, and x stays in
// registers; the next rows' loads are in flight while a few are worked on. The
// lanes' sums are added once, at the end. Measured with 14336 x 4096 weights in
// bf16: one row 41 us (5.7 TB/s; 4.3 times as much code in the sums over lanes
// took 57), four 44, of the tiles 47 at any number up to 16. Fragments loaded
// straight to the matrix instruction, 64 bytes of each of 16 rows a load, took 44
// and 50 us for one and 16 rows.
// ------------------------------------------------------------------------

// N values a lane added over the 64 lanes, by halves: in each step every lane
// hands half of its values over and keeps the sums of the other half. Lane l ends
// with N / 64 values from l * N / 64 on, or 64 / N lanes with value l * N / 64.
template <int N, int LANES>
__device__ __forceinline__ void lanes_sums(float* v, int lane) {
  if constexpr (LANES > 0) {
    constexpr int kHalf = N / 2;
    if constexpr (kHalf > 0) {
#pragma unroll
      for (int i = 0; i < kHalf; ++i) {
        const float keep = lane & LANES ? v[i + kHalf] : v[i], give = lane & LANES ? v[i] : v[i + kHalf];
        v[i] = keep + __shfl_xor(give, LANES, 64);
      }
      lanes_sums<kHalf, LANES / 2>(v, lane);
    } else {
      v[0] += __shfl_xor(v[0], LANES, 64);
      lanes_sums<1, LANES / 2>(v, lane);
    }
  }
}

constexpr int64_t kTokens = 4;
constexpr int kTokenRun = 512;
constexpr int kTokenWaves = 4;  // of a block: with eight, four rows took 60 us instead of 44

template <int T, int DT>
__global__ void __launch_bounds__(64 * kTokenWaves) gated_token_kernel(const ProductArgs P) {
  constexpr int NW = kTokenWaves, kValues = 2 * kFrag * T;
  constexpr int kTogether = 4;  // rows of wg and of wu that are loaded at once (2 or 8: 47 and 60 us)
  __shared__ float sums[NW][kValues];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kFrag;
  const int last = P.n - 1 - n0 < kFrag - 1 ? static_cast<int>(P.n - 1 - n0) : kFrag - 1;
  const char* const wg = P.b[0] + n0 * P.b_ld;
  const char* const wu = P.b[1] + n0 * P.b_ld;
  float acc[kValues] = {};  // of product z, row r, token t at (z * 16 + r) * T + t
  // A run; the contraction's last one may end inside it. A lane that would pass the
  // end takes the last 8 values there, and what another lane has is zero on both
  // sides (an infinite weight times a zero of x alone would be NaN).
  auto work = [&](auto ends, int64_t run) {
    constexpr bool kEnds = decltype(ends)::value;
    const int64_t k = run + lane * 8, at = !kEnds || k < P.k - 8 ? k : P.k - 8;
    const int skip = kEnds ? static_cast<int>(k - at) : 0;
    const int32_t off = static_cast<int32_t>((at - run) * 2);
    auto values = [&](u4 raw, float* v) {
      widen<DT>(raw, v);
      if constexpr (kEnds) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e >= skip ? v[e] : 0.f;
      }
    };
    float x[T][8];
#pragma unroll
    for (int t = 0; t < T; ++t) values(load_any(P.a[0] + (t < P.m ? t : P.m - 1) * P.a_ld + at * 2), x[t]);
    u4 v[2][2][kTogether];
    auto fetch = [&](int r0, u4 (&to)[2][kTogether]) {
#pragma unroll
      for (int r = 0; r < kTogether; ++r) {
        const int64_t row = r0 + r < last ? r0 + r : last;
        to[0][r] = load_any(wg + row * P.b_ld + run * 2 + off);
        to[1][r] = load_any(wu + row * P.b_ld + run * 2 + off);
      }
    };
    fetch(0, v[0]);
#pragma unroll
    for (int r0 = 0; r0 < kFrag; r0 += kTogether) {
      const int now = r0 / kTogether & 1;
      if (r0 + kTogether < kFrag) fetch(r0 + kTogether, v[now ^ 1]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int z = 0; z < 2; ++z)
#pragma unroll
        for (int r = 0; r < kTogether; ++r) {
          float y[8];
          values(v[now][z][r], y);
#pragma unroll
          for (int t = 0; t < T; ++t)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float& s = acc[(z * kFrag + r0 + r) * T + t];
              s = __builtin_fmaf(y[e], x[t][e], s);
            }
        }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  int64_t run = static_cast<int64_t>(w) * kTokenRun;
  for (; run + kTokenRun <= P.k; run += NW * kTokenRun) work(std::false_type{}, run);
  if (run < P.k) work(std::true_type{}, run);
  lanes_sums<kValues, 32>(acc, lane);
  constexpr int kEach = kValues >= 64 ? kValues / 64 : 1, kLanes = kValues >= 64 ? 1 : 64 / kValues;  // values a lane, lanes a value
#pragma unroll
  for (int i = 0; i < kEach; ++i) sums[w][lane / kLanes * kEach + i] = acc[i];
  __syncthreads();
  for (int i = threadIdx.x; i < kFrag * T; i += 64 * NW) {
    const int r = i / T, t = i % T;
    if (t >= P.m || r > last) continue;
    float g = 0.f, u = 0.f;
#pragma unroll
    for (int q = 0; q < NW; ++q) {
      g += sums[q][i];
      u += sums[q][kFrag * T + i];
    }
    const int64_t n = n0 + r;
    store_one(P.out[0], t * P.out_ld[0] + n, DT, activation(g, P.act) * u);
    if (P.out[1]) {
      store_one(P.out[1], t * P.out_ld[1] + n, DT, g);
      store_one(P.out[2], t * P.out_ld[2] + n, DT, u);
    }
  }
}

// The splits' sums, added in order; the grid's y is the output of a pair. A value a
// lane: 7 us for two splits of 1001 x 1600, which the caches hold.
template <int ODT>
__global__ void __launch_bounds__(256) gated_join_kernel(const ProductArgs P, int outputs) {
  const int64_t each = P.m * P.n;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < each; i += static_cast<int64_t>(gridDim.x) * 256) {
    const int z = blockIdx.y;
    float s = 0.f;
    for (int q = 0; q < P.splits; ++q) s += P.partial[(static_cast<int64_t>(q) * outputs + z) * each + i];
    const int64_t row = i / P.n, at = row * P.out_ld[z] + (i - row * P.n);
    if (P.accumulate) s += load_one(P.out[z], at, ODT);
    store_one(P.out[z], at, ODT, s);
  }
}

// ------------------------------------------------------------------------
// dg = dh act'(g) u, du = dh act(g): a streaming pass, 8192 x 14336 in bf16 196 us
// (6.0 TB/s). dg and du may lie where g and u do. They are rounded to the operands'
// type because the products that follow take no other on the matrix pipes: as
// two 16-bit terms each they would double the products' time. dx and dw are then 1.4 times as far from the
// formula as their own rounding makes them (2.3e-3 in bf16, 2.9e-4 in fp16, in the
// 2-norm), and what passes fp16's range is infinite, as any fp16 gradient is.
// ------------------------------------------------------------------------

struct GateGradArgs {
  Rows dh, pre[2];
  RowsOut dpre[2];
  int64_t rows, cols;
  int32_t act;
};

template <int DT>
__global__ void __launch_bounds__(256) gate_grad_kernel(const GateGradArgs G, int64_t row_slots, int64_t slots) {
  constexpr int kVals = Vec<DT>::kVals;
  for (int64_t s = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; s < slots; s += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t row = G.rows > 1 ? s / row_slots : 0, col = (s - row * row_slots) * kVals, left = G.cols - col;
    float dh[kVals], g[kVals], u[kVals];
    widen<DT>(load_part<DT, true>(static_cast<const char*>(G.dh.p) + (row * G.dh.ld + col) * 2, left), dh);
    widen<DT>(load_part<DT, true>(static_cast<const char*>(G.pre[0].p) + (row * G.pre[0].ld + col) * 2, left), g);
    widen<DT>(load_part<DT, true>(static_cast<const char*>(G.pre[1].p) + (row * G.pre[1].ld + col) * 2, left), u);
#pragma unroll
    for (int e = 0; e < kVals; ++e) {
      float a, da;
      activation_grad(g[e], G.act, &a, &da);
      g[e] = dh[e] * da * u[e];
      u[e] = dh[e] * a;
    }
    store_part<DT>(static_cast<char*>(G.dpre[0].p) + (row * G.dpre[0].ld + col) * 2, left, narrow<DT>(g));
    store_part<DT>(static_cast<char*>(G.dpre[1].p) + (row * G.dpre[1].ld + col) * 2, left, narrow<DT>(u));
  }
}

// ------------------------------------------------------------------------
// Launches
// ------------------------------------------------------------------------

// More than the default limit of 64 KiB of dynamic LDS, granted once per kernel and device.
template <typename Kernel>
hipError_t grant_lds(Kernel kernel, int lds, std::atomic<uint64_t>& granted) {
  int dev = 0;
  if (hipError_t e = hipGetDevice(&dev)) return e;
  const uint64_t bit = uint64_t{1} << (dev & 63);
  if (dev > 63 || !(granted.load(std::memory_order_acquire) & bit)) {
    if (hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, lds))
      return e;
    granted.fetch_or(bit, std::memory_order_release);
  }
  return hipSuccess;
}

template <Use USE, Fetch FETCH, int FM, int FN, int WM, int WN, int NB, int KG, int DT, int ODT>
hipError_t tile_launch(const ProductArgs& a, hipStream_t s) {
  using T = Tile<USE, FM, FN, WM, WN, NB, KG>;
  const auto kernel = gated_tile_kernel<USE, FETCH, FM, FN, WM, WN, NB, KG, DT, ODT>;
  const int64_t tiles = ceil_div(a.m, T::kM) * ceil_div(a.n, T::kOutN) * (USE == kDw ? 2 : 1);
  if (tiles > INT32_MAX / T::kThreads / (a.splits > 1 ? a.splits : 1)) return hipErrorInvalidConfiguration;
  if (a.dry) return hipSuccess;
  static std::atomic<uint64_t> granted{0};
  if (hipError_t e = grant_lds(kernel, T::kLds, granted)) return e;
  const int64_t blocks = tiles * (a.splits > 1 ? a.splits : 1);
  hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(blocks)), dim3(T::kThreads), T::kLds, s, a);
  return hipGetLastError();
}

bool aligned16(const void* p, int64_t ld_bytes) { return ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld_bytes)) & 15) == 0; }

constexpr int64_t kScratchFloats = kScratchBytes / sizeof(float);
constexpr int64_t kFewSmall = 448;
constexpr int64_t kVeryFew = 128;

// Whether every slot of the operands is aligned and whole. (A moved tile starts at
// n - kN: on 16 bytes if n is.)
template <Use USE>
bool direct_fetch(const ProductArgs& a) {
  return aligned16(a.a[0], a.a_ld) && aligned16(a.b[0], a.b_ld) && (!a.a[1] || aligned16(a.a[1], a.a_ld)) &&
         (!a.b[1] || aligned16(a.b[1], a.b_ld)) && (USE != kDw || a.m % 8 == 0) && (USE == kForward || a.n % 8 == 0);
}

// One tile shape with the fetch that the operands allow; fetches that write LDS
// themselves keep NB - 1 stages in flight.
template <Use USE, int FM, int FN, int WM, int WN, int NB, int KG, int DT, int ODT>
hipError_t fetch_launch(const ProductArgs& a, hipStream_t s) {
  using T = Tile<USE, FM, FN, WM, WN>;
  if constexpr (T::kM == 64 && USE != kForward) {
    if ((USE == kDw && a.m < T::kM) || a.n < T::kN) return tile_launch<USE, kMasked, FM, FN, WM, WN, 2, KG, DT, ODT>(a, s);
  }
  if (direct_fetch<USE>(a)) return tile_launch<USE, kDirect, FM, FN, WM, WN, NB, KG, DT, ODT>(a, s);
  return tile_launch<USE, kStaged, FM, FN, WM, WN, 2, KG, DT, ODT>(a, s);
}

template <int ODT>
hipError_t join_launch(const ProductArgs& a, int outputs, hipStream_t s) {
  const int64_t blocks = ceil_div(a.m * a.n, 256);
  hipLaunchKernelGGL((gated_join_kernel<ODT>), dim3(static_cast<uint32_t>(blocks < 4096 ? blocks : 4096), outputs), dim3(256),
                     0, s, a, outputs);
  return hipGetLastError();
}

template <Use USE, int DT, int ODT>
hipError_t product_launch(ProductArgs a, float* scratch, hipStream_t s) {
  constexpr int kOutputs = USE == kDw ? 2 : 1;
  if constexpr (USE == kForward) {
    if (a.m <= kTokens && a.k >= 8 && ceil_div(a.n, kFrag) <= INT32_MAX / (64 * kTokenWaves)) {
      const dim3 blocks(static_cast<uint32_t>(ceil_div(a.n, kFrag))), threads(64 * kTokenWaves);
      if (a.m == 1) hipLaunchKernelGGL((gated_token_kernel<1, DT>), blocks, threads, 0, s, a);
      else if (a.m == 2) hipLaunchKernelGGL((gated_token_kernel<2, DT>), blocks, threads, 0, s, a);
      else hipLaunchKernelGGL((gated_token_kernel<4, DT>), blocks, threads, 0, s, a);
      return hipGetLastError();
    }
  }
  auto tiles = [&](int64_t tm, int64_t tn) { return ceil_div(a.m, tm) * ceil_div(a.n, tn) * kOutputs; };
  constexpr int kHalf = USE == kForward ? 2 : 1;
  const Route route = route_of(USE, a.m, a.n, a.k, kScratchFloats);
  const bool middle = route.tile == Route::kMiddle;
  a.splits = static_cast<int32_t>(route.splits);
  a.partial = a.splits > 1 ? scratch : nullptr;
  if (route.tile == Route::kLarge) {
    if constexpr (USE == kForward) return fetch_launch<USE, 4, 8, 4, 2, 2, 1, DT, ODT>(a, s);
    else return fetch_launch<USE, 8, 4, 2, 4, 2, 1, DT, ODT>(a, s);
  }
  hipError_t e;
  // A middle tile with a CU to itself takes eight waves and keeps three stages in
  // flight; where there are two a CU, four waves and one stage each are as good (dx
  // of 2000 x 2048 x 8000, 256 tiles: 215 us with four waves, 203 with eight, 138
  // with three stages in flight too; forward of 128 x 4096 x 14336, 224: 74, 70, 58).
  // Small tiles of a forward pass, which has no scratch to split over, are halved where
  // that still leaves a CU no more than one (kVeryFew), and two groups of waves share the
  // contraction (16 x 8192 x 2048: 47 -> 26.5 us; 64 x 4096 x 4096: 26 -> 17; 64 x 4096 x
  // 14336, 224 tiles: 14 % more; twelve random sizes each: up to 128 tiles took 37 %
  // less to 5 % more time, 129 to 300 31 to 75 % more, one 14 % less). The small tile has
  // two stages in flight where its blocks do not fill the CUs (kFewSmall; forward of
  // 17 x 4096 x 14336, 224 blocks: 61 -> 47.5 us; dx of 1001 x 1600 x 6400, 416: 74 -> 65;
  // twelve random sizes each: 34 % less to 12 % more forward, 3 and 12 % less to 1 and
  // 5 % more in dx and dw) and one where they do, two blocks a CU (dx of 16 x 4096 x
  // 14336, 512: 46.5 against 50; of 24 random sizes within 2 % but one).
  const int64_t blocks = (middle ? tiles(128, 128 / kHalf) : tiles(64, 128 / kHalf)) * a.splits;
  if constexpr (USE == kForward) {
    if (!middle && blocks <= kVeryFew) return fetch_launch<USE, 4, 2, 1, 2, 4, 2, DT, ODT>(a, s);
  }
  if (middle && blocks <= kCus) e = fetch_launch<USE, 2, 4, 4, 2, 4, 1, DT, ODT>(a, s);
  else if (middle) e = fetch_launch<USE, 4, 4, 2, 2, 2, 1, DT, ODT>(a, s);
  else if (blocks <= kFewSmall) e = fetch_launch<USE, 2, 4, 2, 2, 3, 1, DT, ODT>(a, s);
  else e = fetch_launch<USE, 2, 4, 2, 2, 2, 1, DT, ODT>(a, s);
  if (e != hipSuccess || a.splits <= 1 || a.dry) return e;
  return join_launch<ODT>(a, kOutputs, s);
}

// dx and dw together, if that pays: *done says whether they were launched.
template <int DT, int ODT>
hipError_t pair_launch(ProductArgs x, ProductArgs w, float* scratch, hipStream_t s, bool* done) {
  using X = Tile<kDx, 2, 4, 4, 2, 4>;
  using W = Tile<kDw, 8, 4, 2, 4, 2>;
  *done = false;
  const PairRoute route = pair_route(x.m, x.n, x.k, kScratchFloats);
  if (!route.together || !direct_fetch<kDx>(x) || !direct_fetch<kDw>(w)) return hipSuccess;
  *done = true;
  x.splits = static_cast<int32_t>(route.splits);
  x.partial = scratch;
  w.splits = 1;
  w.partial = nullptr;
  static_assert(X::kM == 128 && X::kN == 128 && W::kM == 256 && W::kN == 256, "as pair_route counts them");
  const auto kernel = gated_pair_kernel<DT, ODT>;
  constexpr int kLds = X::kLds > W::kLds ? X::kLds : W::kLds;
  static_assert(X::kThreads == 512 && W::kThreads == 512, "");
  static std::atomic<uint64_t> granted{0};
  if (hipError_t e = grant_lds(kernel, kLds, granted)) return e;
  const uint32_t of_dx = static_cast<uint32_t>(route.dx_blocks), first = (of_dx + kXcds - 1) / kXcds * kXcds;
  hipLaunchKernelGGL(kernel, dim3(first + static_cast<uint32_t>(route.tiles)), dim3(512), kLds, s, x, w, of_dx, first);
  if (hipError_t e = hipGetLastError()) return e;
  return x.splits > 1 ? join_launch<DT>(x, 1, s) : hipSuccess;
}

template <int DT>
hipError_t forward_launch(const GatedArgs& g, hipStream_t s) {
  ProductArgs a = {};
  a.a[0] = static_cast<const char*>(g.x.p);
  a.a_ld = g.x.ld * 2;
  for (int i = 0; i < 2; ++i) a.b[i] = static_cast<const char*>(g.w[i].p);
  a.b_ld = g.w[0].ld * 2;
  a.m = g.m;
  a.n = g.f;
  a.k = g.d;
  for (int i = 0; i < 3; ++i) {
    a.out[i] = g.out[i].p;
    a.out_ld[i] = g.out[i].ld;
  }
  a.act = g.act;
  return product_launch<kForward, DT, DT>(a, nullptr, s);
}

template <int DT, int ODT>
hipError_t products_of_grad(const GatedGradArgs& g, bool dry, hipStream_t s) {
  ProductArgs x = {}, w = {};
  x.dry = w.dry = dry;
  for (int i = 0; i < 2; ++i) {
    x.a[i] = w.a[i] = static_cast<const char*>(g.dpre[i].p);
    x.b[i] = static_cast<const char*>(g.w[i].p);
    w.out[i] = g.dw[i].p;
    w.out_ld[i] = g.dw[i].ld;
  }
  x.a_ld = w.a_ld = g.dpre[0].ld * 2;
  x.b_ld = g.w[0].ld * 2;
  x.m = g.m;
  x.n = g.d;
  x.k = g.f;
  x.out[0] = g.dx.p;
  x.out_ld[0] = g.dx.ld;
  w.b[0] = static_cast<const char*>(g.x.p);
  w.b_ld = g.x.ld * 2;
  w.m = g.f;
  w.n = g.d;
  w.k = g.m;
  w.accumulate = g.accumulate;
  const bool of_x = g.dx.p && g.m > 0 && g.d > 0, of_w = g.dw[0].p && g.f > 0 && g.d > 0;
  if (of_x && of_w && !dry) {
    bool done = false;
    const hipError_t e = pair_launch<DT, ODT>(x, w, g.scratch, s, &done);
    if (done || e != hipSuccess) return e;
  }
  if (of_x)
    if (hipError_t e = product_launch<kDx, DT, DT>(x, g.scratch, s)) return e;
  return of_w ? product_launch<kDw, DT, ODT>(w, g.scratch, s) : hipSuccess;
}

template <int DT>
hipError_t grad_launch(const GatedGradArgs& g, hipStream_t s) {
  // a call that cannot launch all of it launches nothing
  const bool wide = g.dw_dt == ZERO_DT_F32;
  if (hipError_t e = wide ? products_of_grad<DT, ZERO_DT_F32>(g, true, s) : products_of_grad<DT, DT>(g, true, s)) return e;
  if (g.m > 0 && g.f > 0) {
    GateGradArgs e = {g.dh, {g.pre[0], g.pre[1]}, {g.dpre[0], g.dpre[1]}, g.m, g.f, g.act};
    if (g.dh.ld == g.f && g.pre[0].ld == g.f && g.dpre[0].ld == g.f) {  // one row
      e.cols *= e.rows;
      e.rows = 1;
    }
    const int64_t row_slots = ceil_div(e.cols, Vec<DT>::kVals), slots = row_slots * e.rows, blocks = ceil_div(slots, 256);
    const int grid = limit_grid(static_cast<int>(blocks < kMaxGrid ? blocks : kMaxGrid));
    hipLaunchKernelGGL((gate_grad_kernel<DT>), dim3(grid), dim3(256), 0, s, e, row_slots, slots);
    if (hipError_t x = hipGetLastError()) return x;
  }
  return wide ? products_of_grad<DT, ZERO_DT_F32>(g, false, s) : products_of_grad<DT, DT>(g, false, s);
}

}  // namespace

hipError_t launch_gated(const GatedArgs& a, int32_t dt, hipStream_t s) {
  if (dt == ZERO_DT_F16) return forward_launch<ZERO_DT_F16>(a, s);
  if (dt == ZERO_DT_BF16) return forward_launch<ZERO_DT_BF16>(a, s);
  return hipErrorInvalidValue;
}

hipError_t launch_gated_grad(const GatedGradArgs& a, int32_t dt, hipStream_t s) {
  if (dt == ZERO_DT_F16) return grad_launch<ZERO_DT_F16>(a, s);
  if (dt == ZERO_DT_BF16) return grad_launch<ZERO_DT_BF16>(a, s);
  return hipErrorInvalidValue;
}

}  // namespace zdp
