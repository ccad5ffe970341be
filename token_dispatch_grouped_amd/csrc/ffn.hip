// Host launchers of the dense gated feed-forward block (ffn_kernel.h has the
// kernels and the mathematics): forward in bf16 and in the 8-bit block form,
// and the gradient of the input.
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

// Whether a product of M rows and N columns takes the 256 x 256 tile. A card
// of `cus` compute units runs one such tile per CU at a time, or two of the
// 128 x 128 ones; a round of the large tiles takes 1.45 times a round of the
// small ones and does twice the work (measured at K = 2048, N = 2816: 56-59
// against 38 us a round in bf16, 57 against 40 us in MX8). So the tile whose
// rounds take less time wins: the small one where the large leaves most CUs
// idle. n_small, n_large: output columns of a small and a large tile.
static bool large_tile(int M, int N, int n_small, int n_large) {
  const int64_t cus = persistent_grid();
  const int64_t small = ceil_div(M, 128) * ceil_div(N, n_small), large = ceil_div(M, 256) * ceil_div(N, n_large);
  return 145 * ceil_div(large, cus) < 100 * ceil_div(small, 2 * cus);
}

static hipError_t gateup(const FfnTileParams &p, bool mx8, hipStream_t s) {
  const bool large = large_tile(p.M, p.N, 64, 128);
  if (mx8)
    return large ? run_ffn_tile<true, 256, 256, 128, 64, false, FFN_SWIGLU_FWD>(p, s)
                 : run_ffn_tile<true, 128, 128, 64, 64, false, FFN_SWIGLU_FWD>(p, s);
  return large ? wide<false, EPI_SWIGLU_FWD>(p, s)
               : run_ffn_tile<false, 128, 128, 64, 64, false, FFN_SWIGLU_FWD>(p, s);
}

static hipError_t down(const FfnTileParams &p, bool mx8, hipStream_t s) {
  const bool large = large_tile(p.M, p.N, 128, 256);
  if (mx8)
    return large ? run_ffn_tile<true, 256, 256, 128, 64, false, FFN_STORE>(p, s)
                 : run_ffn_tile<true, 128, 128, 64, 64, false, FFN_STORE>(p, s);
  return large ? wide_store<false>(p, s) : run_ffn_tile<false, 128, 128, 64, 64, false, FFN_STORE>(p, s);
}

hipError_t launch_ffn_dense_fwd(const FfnArgs &a, hipStream_t s) {
  {
    LaunchScope scope("ffn_gateup_fwd", s);
    const hipError_t err = gateup(gateup_params(a), a.mx8, s);
    if (err != hipSuccess) return err;
  }
  LaunchScope scope("ffn_down_fwd", s);
  return down(down_params(a), a.mx8, s);
}

hipError_t launch_ffn_dense_dgrad(const FfnArgs &a, hipStream_t s) {
  {
    LaunchScope scope("ffn_down_dgrad", s);
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
    const hipError_t err = large_tile(p.M, p.N, 128, 256)
                               ? wide<true, EPI_SWIGLU_BWD>(p, s)
                               : run_ffn_tile<false, 128, 128, 64, 64, true, FFN_SWIGLU_BWD>(p, s);
    if (err != hipSuccess) return err;
  }
  LaunchScope scope("ffn_gateup_dgrad", s);
  FfnTileParams p{};
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
  return large_tile(p.M, p.N, 128, 256) ? wide_store<true>(p, s)
                                        : run_ffn_tile<false, 128, 128, 64, 64, true, FFN_STORE>(p, s);
}

}  // namespace moe
