// Host launchers of the dense gated feed-forward block (ffn_kernel.h has the
// kernels and the mathematics): forward in bf16 and in the 8-bit block form,
// and the gradient of the input.
#include "ffn_few.h"
#include "ffn_kernel.h"
#include "ffn_wide.h"

namespace moe {

static FfnTileParams gateup_params(const FfnArgs &a) {
  FfnTileParams p{};
  p.A = (const bf16_t *)a.x;
  p.B = (const bf16_t *)a.w_gu;
  p.C = (bf16_t *)a.h;
  p.C2 = (bf16_t *)a.a;
  p.M = (int)a.T;
  p.N = a.F;
  p.F = a.F;
  p.K = a.mx8 ? a.d / 2 : a.d;
  p.lda = p.ldb = p.K;
  p.ldc = 2 * (int64_t)a.F;
  p.As = (const uint8_t *)a.x_scale;
  p.Bs = (const uint8_t *)a.w_gu_scale;
  p.C2s = (uint8_t *)a.a_scale;
  p.a32 = (float *)a.a32;
  return p;
}

static FfnTileParams down_params(const FfnArgs &a) {
  FfnTileParams p{};
  p.A = (const bf16_t *)a.a;
  p.B = (const bf16_t *)a.w_down;
  p.C = (bf16_t *)a.y;
  p.add = (const bf16_t *)a.add;
  p.M = (int)a.T;
  p.N = a.d;
  p.F = a.F;
  p.K = a.mx8 ? a.F / 2 : a.F;
  p.lda = p.ldb = p.K;
  p.ldc = a.d;
  p.As = (const uint8_t *)a.a_scale;
  p.Bs = (const uint8_t *)a.w_down_scale;
  return p;
}

template <bool BKM, int EPI>
static hipError_t wide(const FfnTileParams &t, hipStream_t s) {
  GemmParams p{};
  p.A = t.A;
  p.B = t.B;
  p.C = t.C;
  p.C2 = t.C2;
  p.H = EPI == EPI_SWIGLU_BWD ? t.H : t.add;
  p.M = t.M;
  p.N = t.N;
  p.K = t.K;
  p.F = t.F;
  p.lda = t.lda;
  p.ldb = t.ldb;
  p.ldc = t.ldc;
  return run_ffn_wide<BKM, EPI>(p, s);
}

template <bool BKM>
static hipError_t wide_store(const FfnTileParams &t, hipStream_t s) {
  return t.add ? wide<BKM, EPI_STORE_ADD>(t, s) : wide<BKM, EPI_STORE>(t, s);
}

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

static Tile choose(int M, int NB, bool mx8, bool swiglu, bool kmajor) {
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
static int cost(int M, int NB, bool mx8, bool swiglu, bool kmajor) {
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
static int head_rows(int M, int NB, bool mx8, bool swiglu, bool kmajor) {
  const int64_t cus = persistent_grid(), cols = ceil_div(NB, 256);
  const int64_t rounds = ceil_div(M, 256) * cols / cus;
  if (rounds == 0 || choose(M, NB, mx8, swiglu, kmajor) != kLarge) return M;
  const int64_t head = rounds * cus / cols * 256;
  if (head <= 0 || head >= M) return M;
  const int tail = cost(M - (int)head, NB, mx8, swiglu, kmajor) + 5;
  return 100 * rounds + tail < cost(M, NB, mx8, swiglu, kmajor) ? (int)head : M;
}

// Rows [from, from + count) of a product.
static FfnTileParams rows(FfnTileParams p, bool mx8, int64_t from, int count) {
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
static hipError_t in_rounds(const FfnTileParams &p, int NB, bool mx8, bool swiglu, bool kmajor, Run run) {
  const int head = head_rows(p.M, NB, mx8, swiglu, kmajor);
  if (head == p.M) return run(p);
  const hipError_t err = run(rows(p, mx8, 0, head));
  return err != hipSuccess ? err : run(rows(p, mx8, head, p.M - head));
}

// Each launch has a scope of its own: one record of the timer is one launch.
static hipError_t gateup_product(const FfnTileParams &p, Tile t, bool mx8, hipStream_t s) {
  LaunchScope scope("ffn_gateup_fwd", s);
  if (mx8) {
    switch (t) {
      case kFew: return run_ffn_few<true, FFN_SWIGLU_FWD>(p, s);
      case kNarrow: return run_ffn_tile<true, 64, 128, 32, 64, 2, 3, false, FFN_SWIGLU_FWD>(p, s);
      case kPair: return run_ffn_tile<true, 128, 128, 64, 64, 2, 2, false, FFN_SWIGLU_FWD>(p, s);
      case kLarge: return run_ffn_tile<true, 256, 256, 128, 64, 1, 2, false, FFN_SWIGLU_FWD>(p, s);
      default: return run_ffn_tile<true, 128, 128, 64, 64, 1, 2, false, FFN_SWIGLU_FWD>(p, s);
    }
  }
  switch (t) {
    case kFew: return run_ffn_few<false, FFN_SWIGLU_FWD>(p, s);
    case kSmall: return run_ffn_tile<false, 64, 64, 32, 64, 4, 2, false, FFN_SWIGLU_FWD>(p, s);
    case kNarrow: return run_ffn_tile<false, 64, 128, 32, 64, 2, 3, false, FFN_SWIGLU_FWD>(p, s);
    case kPair: return run_ffn_tile<false, 128, 128, 64, 64, 2, 2, false, FFN_SWIGLU_FWD>(p, s);
    case kHalf: return run_ffn_tile<false, 64, 128, 32, 64, 1, 3, false, FFN_SWIGLU_FWD>(p, s);
    case kLarge: return wide<false, EPI_SWIGLU_FWD>(p, s);
    default: return run_ffn_tile<false, 128, 128, 64, 64, 1, 2, false, FFN_SWIGLU_FWD>(p, s);
  }
}

static hipError_t gateup(const FfnTileParams &p, bool mx8, hipStream_t s) {
  const Tile t = choose(p.M, 2 * p.N, mx8, true, false);
  const hipError_t err = gateup_product(p, t, mx8, s);
  if (err != hipSuccess || !mx8 || t != kFew) return err;
  return launch_mx8_quantize(p.a32, p.C2, p.C2s, p.M, p.F, false, s);
}

static hipError_t down(const FfnTileParams &p, bool mx8, hipStream_t s) {
  LaunchScope scope("ffn_down_fwd", s);
  const Tile t = choose(p.M, p.N, mx8, false, false);
  if (mx8) {
    switch (t) {
      case kFew: return run_ffn_few<true, FFN_STORE>(p, s);
      case kSmall: return run_ffn_tile<true, 64, 64, 32, 64, 4, 2, false, FFN_STORE>(p, s);
      case kNarrow: return run_ffn_tile<true, 64, 128, 32, 64, 2, 3, false, FFN_STORE>(p, s);
      case kPair: return run_ffn_tile<true, 128, 128, 64, 64, 2, 2, false, FFN_STORE>(p, s);
      case kLarge: return run_ffn_tile<true, 256, 256, 128, 64, 1, 2, false, FFN_STORE>(p, s);
      default: return run_ffn_tile<true, 128, 128, 64, 64, 1, 2, false, FFN_STORE>(p, s);
    }
  }
  switch (t) {
    case kFew: return run_ffn_few<false, FFN_STORE>(p, s);
    case kSmall: return run_ffn_tile<false, 64, 64, 32, 64, 4, 2, false, FFN_STORE>(p, s);
    case kNarrow: return run_ffn_tile<false, 64, 128, 32, 64, 2, 3, false, FFN_STORE>(p, s);
    case kPair: return run_ffn_tile<false, 128, 128, 64, 64, 2, 2, false, FFN_STORE>(p, s);
    case kHalf: return run_ffn_tile<false, 64, 128, 32, 64, 1, 3, false, FFN_STORE>(p, s);
    case kLarge: return wide_store<false>(p, s);
    default: return run_ffn_tile<false, 128, 128, 64, 64, 1, 2, false, FFN_STORE>(p, s);
  }
}

hipError_t launch_ffn_dense_fwd(const FfnArgs &a, hipStream_t s) {
  const hipError_t err = in_rounds(gateup_params(a), 2 * a.F, a.mx8, true, false,
                                   [&](const FfnTileParams &p) { return gateup(p, a.mx8, s); });
  if (err != hipSuccess) return err;
  return in_rounds(down_params(a), a.d, a.mx8, false, false,
                   [&](const FfnTileParams &p) { return down(p, a.mx8, s); });
}

static hipError_t down_dgrad(const FfnTileParams &p, hipStream_t s) {
  LaunchScope scope("ffn_down_dgrad", s);
  switch (choose(p.M, p.N, false, false, true)) {
    case kNarrow: return run_ffn_tile<false, 64, 128, 32, 64, 2, 2, true, FFN_SWIGLU_BWD>(p, s);
    case kPair: return run_ffn_tile<false, 128, 128, 64, 64, 2, 2, true, FFN_SWIGLU_BWD>(p, s);
    case kLarge: return wide<true, EPI_SWIGLU_BWD>(p, s);
    default: return run_ffn_tile<false, 128, 128, 64, 64, 1, 2, true, FFN_SWIGLU_BWD>(p, s);
  }
}

static hipError_t gateup_dgrad(const FfnTileParams &p, hipStream_t s) {
  LaunchScope scope("ffn_gateup_dgrad", s);
  switch (choose(p.M, p.N, false, false, true)) {
    case kNarrow: return run_ffn_tile<false, 64, 128, 32, 64, 2, 2, true, FFN_STORE>(p, s);
    case kPair: return run_ffn_tile<false, 128, 128, 64, 64, 2, 2, true, FFN_STORE>(p, s);
    case kLarge: return wide_store<true>(p, s);
    default: return run_ffn_tile<false, 128, 128, 64, 64, 1, 2, true, FFN_STORE>(p, s);
  }
}

hipError_t launch_ffn_dense_dgrad(const FfnArgs &a, hipStream_t s) {
  FfnTileParams p{};
  p.A = (const bf16_t *)a.dy;
  p.B = (const bf16_t *)a.w_down;
  p.C = (bf16_t *)a.dh;
  p.H = (const bf16_t *)a.h;
  p.M = (int)a.T;
  p.N = a.F;
  p.F = a.F;
  p.K = a.d;
  p.lda = a.d;
  p.ldb = a.F;
  p.ldc = 2 * (int64_t)a.F;
  const hipError_t err =
      in_rounds(p, p.N, false, false, true, [&](const FfnTileParams &q) { return down_dgrad(q, s); });
  if (err != hipSuccess) return err;
  p = FfnTileParams{};
  p.A = (const bf16_t *)a.dh;
  p.B = (const bf16_t *)a.w_gu;
  p.C = (bf16_t *)a.dx;
  p.add = (const bf16_t *)a.add;
  p.M = (int)a.T;
  p.N = a.d;
  p.F = a.F;
  p.K = 2 * a.F;
  p.lda = 2 * (int64_t)a.F;
  p.ldb = a.d;
  p.ldc = a.d;
  return in_rounds(p, p.N, false, false, true, [&](const FfnTileParams &q) { return gateup_dgrad(q, s); });
}

}  // namespace moe
