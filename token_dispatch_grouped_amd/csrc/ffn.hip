// Host launchers of the dense gated feed-forward block (ffn_kernel.h has the
// kernels and the mathematics): forward in bf16 and in the 8-bit block form,
// and the gradient of the input.
#include "ffn_few.h"
#include "ffn_kernel.h"
#include "ffn_plan.h"
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
