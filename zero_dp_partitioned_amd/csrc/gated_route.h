// Which tiles and launches the gated product's products take (host only): rules on
// sizes, with what was measured on both sides of each.
#pragma once

#include <stdint.h>

namespace zdp {

enum Use { kForward, kDx, kDw };

constexpr int kChunk = 64;  // contraction per stage of a tile: 128 bytes of a row
constexpr int kXcds = 8;
constexpr int64_t kCus = 256;

// Middle tiles that leave no more than three of eight CUs idle. Twelve random sizes
// each: 160 to 255 middle tiles took up to 40 % less time than small ones forward, up
// to 16 % less in dw and 10 % less in dx (one 58 % more); 96 to 159 took up to 24 %
// more, 11 % more and 9 % more, tall ones up to 31, 17 and 14 % less.
constexpr int64_t kEnoughTiles = 160;
// Blocks of shared middle tiles that leave fewer than a fifth of the CUs idle: 209 to
// 250 took up to 15 % less time than small tiles (most 1 to 8 % less, a few up to 9 %
// more), 151 to 208 from 13 % less to 6 % more.
constexpr int64_t kMostCus = 208;

inline int64_t tiles_over(int64_t n, int64_t size) { return n / size + (n % size != 0); }

// The tiles of one product, and the blocks that share a tile's contraction.
struct Route {
  enum Tile { kLarge, kMiddle, kSmall } tile;  // 256 x 256, 128 x 128, 64 x 128
  int64_t splits;
};

// m x n outputs over a contraction of k (of one of dx's two parts); `room` floats for partial sums.
inline Route route_of(Use use, int64_t m, int64_t n, int64_t k, int64_t room) {
  const int64_t outputs = use == kDw ? 2 : 1, half = use == kForward ? 2 : 1;
  auto tiles = [&](int64_t tm, int64_t tn) { return tiles_over(m, tm) * tiles_over(n, tn) * outputs; };
  // a tile has more than half its rows and columns to do; along the columns it must fit its operand
  auto fits = [&](int64_t side) {
    return m > (use == kDw ? side - 1 : side / 2) && n > (use != kForward ? side - 1 : side / half / 2);
  };
  // By rounds over the CUs: a round of one 256 x 256 tile a CU takes as long as 1.5
  // rounds of two 128 x 128 tiles a CU, and a round of one of those half of that.
  // (us, large and middle tiles: forward of 1001 x 1600 x 6400, 200 and 800 tiles: 40,
  // 50; of 2048 x 4096 x 14336, 896 and 3584: 413, 494; dx of 2048 x 4096 x 14336, 128
  // and 512: 640, 479.)
  const int64_t mid = tiles(128, 128 / half);
  const int64_t large = tiles_over(tiles(256, 256 / half), kCus) * 6, pairs = tiles_over(mid, 2 * kCus) * 4;
  if (fits(256) && large <= (mid <= kCus ? 2 : pairs)) return {Route::kLarge, 1};
  bool middle = fits(128) && mid >= kEnoughTiles;
  if (use == kForward) return {middle ? Route::kMiddle : Route::kSmall, 1};
  // Few tiles over a long contraction are shared among blocks, as far as the
  // scratch holds their sums: middle tiles where that gives nearly every CU one (dx
  // of 256 x 4096 x 14336, 64 tiles in 4 splits: 123 us with small tiles, 87; of 300
  // rows, 96 in 2: 140 and 159), else small ones, two blocks a CU.
  const int64_t chunks = tiles_over(k, kChunk) * (use == kDx ? 2 : 1);
  room /= m * n * outputs;
  const int64_t most = room < chunks / 4 ? room : chunks / 4;
  auto shared = [&](int64_t have, int64_t want) { return want / have < most ? want / have : most; };
  const int64_t one = fits(128) ? shared(mid, kCus) : 0;
  middle = middle || mid * one > kMostCus;
  const int64_t splits = middle ? (mid >= kEnoughTiles ? shared(mid, 2 * kCus) : one) : shared(tiles(64, 128), 2 * kCus);
  return {middle ? Route::kMiddle : Route::kSmall, splits > 1 ? splits : 1};
}

// dx (m x d over two parts of f) in middle tiles and dw (two of f x d over m) in large
// ones, in one launch.
struct PairRoute {
  bool together;
  int64_t splits;            // of dx
  int64_t dx_blocks, tiles;  // dx's blocks, dw's tiles
};

inline PairRoute pair_route(int64_t m, int64_t d, int64_t f, int64_t room) {
  PairRoute r = {false, 1, 0, 0};
  if (m <= 64 || d < 256 || f < 256) return r;
  const int64_t tiles_x = tiles_over(m, 128) * tiles_over(d, 128);
  r.tiles = 2 * tiles_over(f, 256) * tiles_over(d, 256);
  if (tiles_x > kCus || r.tiles > 4 * kCus) return r;
  const int64_t chunks = 2 * tiles_over(f, kChunk);
  r.splits = kCus / tiles_x;
  r.splits = r.splits < room / (m * d) ? r.splits : room / (m * d);
  r.splits = r.splits < chunks / 4 ? r.splits : chunks / 4;
  r.splits = r.splits > 1 ? r.splits : 1;
  r.dx_blocks = tiles_x * r.splits;
  // Where dw alone takes large tiles too, one launch fills what either leaves of its
  // last round: of 77 sizes, most of them random, none took more than 1 % more time
  // and the best 38 % less (the whole backward pass, us apart and together: 1500 x
  // 1600 x 6400 219, 176; 2048 rows 245, 232; 500 rows 96, 85; 1001 rows 145, 141; 529 x
  // 3752 x 2440 114, 71; 291 x 3384 x 2080 54, 49; 1024 x 4096 x 4096 156, 155).
  const Route w = route_of(kDw, f, d, m, room);
  if (w.tile == Route::kLarge) {
    r.together = true;
    return r;
  }
  // Else by when the last block ends: a stage of a middle tile takes 0.55 us, one of a
  // large tile 1.45 and its ends 6. An XCD's 32 CUs take its share of dx's blocks
  // first, then of dw's; a large tile does all of its contraction.
  const double tx = 0.55 * chunks / r.splits, tw = 1.45 * tiles_over(m, kChunk) + 6;
  const int64_t cus = kCus / kXcds, busy = tiles_over(r.dx_blocks, kXcds);
  double idle_from = 0, dx_from = tx, end = tx;
  for (int64_t left = tiles_over(r.tiles, kXcds); left > 0;) {
    const bool idle = busy < cus && idle_from <= dx_from;
    double& from = idle ? idle_from : dx_from;
    left -= idle ? cus - busy : busy;
    from += tw;
    end = end > from ? end : from;
  }
  // Apart, dw takes as long as its large tiles and a launch, 2. Of sizes with a round of
  // them at most, 59 that end within three quarters of that time took from 4 % more to
  // 36 % less together (2079 x 1000 x 3776 133, 91; 1500 x 1608 x 1000 52, 46; 2118 x 1088 x
  // 1032 55, 57), 74 others from 6 % less to 34 % more (1500 x 1600 x 640 38, 43; 2048 x
  // 768 x 3000 87, 99; 3953 x 672 x 2624, where an XCD gets one block too many, 111,
  // 149). With more than a round 13 up to 0.84 took as long to 26 % less (2960 x 344 x
  // 19952 391, 351), three above it 6 % more.
  // A dw that shares its contraction among blocks takes every CU, and 22 for its
  // launches, its ends and the join: of 23 sizes within nine tenths of that time 21
  // took 2 to 35 % less together (451 x 776 x 976 41, 32; 712 x 2704 x 280 35, 28), two 4
  // and 5 % more; of 61 others 58 took up to 3.6 times as long (4096 x 1024 x 1024 66,
  // 115; 8192 x 512 x 512 49, 176), three up to 11 % less.
  const bool shares = w.splits > 1;
  const double alone = shares ? 4.0 / 3 * r.tiles * (tw - 6) / kCus + 22 : tw * tiles_over(r.tiles, kCus) + 2;
  r.together = end <= (shares ? 0.9 : r.tiles > kCus ? 0.85 : 0.75) * (tx + alone);
  return r;
}

}  // namespace zdp
