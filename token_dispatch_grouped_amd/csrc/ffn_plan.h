// Which kernel runs a product of the dense block (ffn.hip) or of the dense
// product with bias, activation and residual (linear.hip), and over which rows.
#pragma once

#include "ffn_kernel.h"

namespace moe {

// The kernel of a product of M rows whose B operand has NB rows (gate/up: 2F).
//   few     M <= kFfnFewTokens, forward: reads the weights once (ffn_few.h)
//   small   64 x 64 tiles, 4 k groups a workgroup
//   narrow  64 x 128 tiles, 2 k groups
//   pair    128 x 128 tiles, 2 k groups
//   half    64 x 128 tiles, two workgroups a CU
//   square  128 x 128 tiles, two workgroups a CU
//   large   256 x 256 tiles
// While a tile shape does not fill the card, a smaller one ends sooner (its
// workgroups are bound by the latency of a stage, which the k groups hide).
// Forward at d = 2048, F = 1408, us: 256 tokens small 20.6, narrow 26.7, square
// 39; 512: narrow 28.0, half 29.8, square 40; 1400: pair 40.3, half 43.1; 1472:
// half 43.0, square 49.3; 1536: square 49, half 55; the input gradient at 1400
// tokens pair 48.5, square 52.4, at 2000 58.0, 62.7. In the 8-bit form (d =
// 4096, F = 2816) gate/up 192 tokens narrow 20.3, small 26.7, down small 12.7,
// narrow 16.3; 700 tokens in all pair 55.5, square 57.7.
// Few against the next (us, whole forward, no h kept): at 96 tokens 12.4
// against 18.5 (2048 x 1408), 27.8 against 46.1 (4096 x 2816), 29.9 against
// 48.7 (7168 x 2048), 8-bit 22.5 against 28.1 (4096 x 2816); at 144 tokens
// 16.5 against 19.2, 41.5 against 38.8, 49.1 against 44.0, 8-bit 32.8 against
// 29.0, and 9.2 against 12.2 for 512 x 320: from there on the tiles win more.
// One border for all sizes costs the larger ones 7-13% just below it.
// Large against square: a round of large tiles (one a CU) takes 1.45 times a
// round of square ones (two a CU) and does twice the work (56-59 against 38 us
// in bf16 at K = 2048, 57 against 40 us in the 8-bit form).
enum Tile { kFew, kSmall, kNarrow, kPair, kHalf, kSquare, kLarge };

inline Tile choose(int M, int NB, bool mx8, bool swiglu, bool kmajor) {
  if (!kmajor && M <= kFfnFewTokens) return kFew;
  const int64_t cus = persistent_grid();
  const auto tiles = [&](int bm, int bn) { return ceil_div(M, bm) * ceil_div(NB, bn); };
  if (!kmajor && !(mx8 && swiglu) && tiles(64, 64) <= cus) return kSmall;
  if (tiles(64, 128) <= cus) return kNarrow;
  if (tiles(128, 128) <= cus) return kPair;
  if (!kmajor && !mx8 && tiles(64, 128) <= 2 * cus) return kHalf;
  return 145 * ceil_div(tiles(256, 256), cus) < 100 * ceil_div(tiles(128, 128), 2 * cus) ? kLarge : kSquare;
}

// A product that the large tiles compute in a few tiles more than whole rounds
// of the card leaves most CUs idle for a round, so its last rows go to smaller
// tiles in a launch of their own where that is shorter. Measured (us, against
// one launch): d = 2048, F = 1408 forward at 6000 tokens 119 (146), 9000 164
// (182), 12500 222 (240), 14000 254 (252), input gradient at 8300 170 (209),
// 17000 333 (370); 8-bit 4096 x 2816 at 3000 tokens 123 (155), 4200 162 (193).
// `cost`: hundredths of a round of large tiles, from the times above.
inline int cost(int M, int NB, bool mx8, bool swiglu, bool kmajor) {
  const int64_t cus = persistent_grid();
  switch (choose(M, NB, mx8, swiglu, kmajor)) {
    case kFew: return 20;
    case kSmall: return 25;
    case kNarrow: return 31;
    case kPair: return 45;
    case kHalf: return 50;
    case kSquare: return 69 * (int)ceil_div(ceil_div(M, 128) * ceil_div(NB, 128), 2 * cus);
    default: return 100 * (int)ceil_div(ceil_div(M, 256) * ceil_div(NB, 256), cus);
  }
}

// Rows of the first launch: M for one launch in all.
inline int head_rows(int M, int NB, bool mx8, bool swiglu, bool kmajor) {
  const int64_t cus = persistent_grid(), cols = ceil_div(NB, 256);
  const int64_t rounds = ceil_div(M, 256) * cols / cus;
  if (rounds == 0 || choose(M, NB, mx8, swiglu, kmajor) != kLarge) return M;
  const int64_t head = rounds * cus / cols * 256;
  if (head <= 0 || head >= M) return M;
  const int tail = cost(M - (int)head, NB, mx8, swiglu, kmajor) + 5;
  return 100 * rounds + tail < cost(M, NB, mx8, swiglu, kmajor) ? (int)head : M;
}

// Rows [from, from + count) of a product.
inline FfnTileParams rows(FfnTileParams p, bool mx8, int64_t from, int count) {
  p.A += from * p.lda;
  if (p.As) p.As += from * (p.K / 16);
  if (p.C) p.C += from * p.ldc;
  if (p.C2) p.C2 = reinterpret_cast<bf16_t *>(reinterpret_cast<char *>(p.C2) + from * p.F * (mx8 ? 1 : 2));
  if (p.C2s) p.C2s += from * (p.F / kMx8Block);
  if (p.H) p.H += from * p.ldc;
  if (p.add) p.add += from * p.ldc;
  p.M = count;
  return p;
}

template <typename Run>
hipError_t in_rounds(const FfnTileParams &p, int NB, bool mx8, bool swiglu, bool kmajor, Run run) {
  const int head = head_rows(p.M, NB, mx8, swiglu, kmajor);
  if (head == p.M) return run(p);
  const hipError_t err = run(rows(p, mx8, 0, head));
  return err != hipSuccess ? err : run(rows(p, mx8, head, p.M - head));
}

}  // namespace moe
