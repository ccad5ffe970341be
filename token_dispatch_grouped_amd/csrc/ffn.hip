// Host launchers of the dense gated feed-forward block (ffn_kernel.h has the
// kernels and the mathematics): forward in bf16 and in the 8-bit block form,
// and the gradient of the input.
#include "ffn_kernel.h"

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

hipError_t launch_ffn_dense_fwd(const FfnArgs &a, hipStream_t s) {
  hipError_t err;
  {
    LaunchScope scope("ffn_gateup_fwd", s);
    const FfnTileParams p = gateup_params(a);
    err = a.mx8 ? run_ffn_tile<true, 128, 128, 64, 64, false, FFN_SWIGLU_FWD>(p, s)
                : run_ffn_tile<false, 128, 128, 64, 64, false, FFN_SWIGLU_FWD>(p, s);
  }
  if (err != hipSuccess) return err;
  LaunchScope scope("ffn_down_fwd", s);
  const FfnTileParams p = down_params(a);
  return a.mx8 ? run_ffn_tile<true, 128, 128, 64, 64, false, FFN_STORE>(p, s)
               : run_ffn_tile<false, 128, 128, 64, 64, false, FFN_STORE>(p, s);
}

hipError_t launch_ffn_dense_dgrad(const FfnArgs &a, hipStream_t s) {
  hipError_t err;
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
    err = run_ffn_tile<false, 128, 128, 64, 64, true, FFN_SWIGLU_BWD>(p, s);
  }
  if (err != hipSuccess) return err;
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
  return run_ffn_tile<false, 128, 128, 64, 64, true, FFN_STORE>(p, s);
}

}  // namespace moe
