// Weight gradients of the dense gated feed-forward block:
//   dw_gu [2F,d] (+)= dh^T x     dw_down [d,F]  (+)= dy^T a     (fp32)
// The grouped products' tile with both operands k-major, 256 x 256 or, for
// small gradients, 128 x 128. There are few output tiles and a long sum over
// the tokens, so the tokens are split into slices (ffn_wgrad_plan has the rule
// and what it was measured on): every (slice, tile) pair of either product is a
// workgroup of one launch. With one slice it writes dw or adds to it (7001
// tokens, adding: 167-173 us against 184 with a launch of its own for the sum,
// 160 overwriting; 128 tokens 19.5 against 32); otherwise it writes fp32 partial sums to the workspace
// and a second launch adds the slices in order (no atomics: the same bits run to run). The
// tiles of a slice are neighbours, so that the workgroups of an XCD share
// operand rows. At 32768 tokens, d = 2048, F = 1408: 550 us (1030 TFLOP/s) and
// 27 us for the sum of three slices.
//
// This file also holds the gate/up forward on the same tile, for the sake of
// the instruction scheduling that both are compiled with.
#include "ffn_wide.h"

namespace moe {

template hipError_t run_ffn_wide<false, EPI_SWIGLU_FWD>(GemmParams, hipStream_t);

struct WgradParams {
  GemmParams g[2];  // dw_gu, dw_down; total: the product's workgroups
  int T, chunk;
};

// B x B tiles: 8 wavefronts of 128 x 64 (B = 256), or 4 of 64 x 64 (B = 128).
template <int B, int EPI>
__global__ __launch_bounds__(B * 2) void ffn_wgrad_kernel(WgradParams w) {
  constexpr int WN = 64, NW = B / 32;
  __shared__ u32x4_t lds[2 * (B + B) * kStageK * 2 / 16];
  int lo, hi;
  xcd_range(blockIdx.x & 7, w.g[0].total + w.g[1].total, lo, hi);
  int id = lo + (int)(blockIdx.x >> 3);
  if (id >= hi) return;
  const int which = id >= w.g[0].total ? 1 : 0;
  if (which) id -= w.g[0].total;
  const GemmParams &p = w.g[which];
  const int tiles = p.m_tiles * p.n_tiles;
  const int slice = id / tiles, r = id - slice * tiles;
  const int mt = r / p.n_tiles, nt = r - mt * p.n_tiles;
  const int row0 = slice * w.chunk;
  const int kdim = min(w.chunk, w.T - row0);
  const int m0 = mt * B;
  auto none = [&](NextTile &nx) { nx.valid = false; };
  gg_tile<B, B, B / 2, WN, NW, true, true, EPI, true, kStageK, kStages>(
      p, lds, slice, m0, nt, min(B, p.M - m0), kdim, 0, p.A + (int64_t)row0 * p.lda + m0,
      p.B + (int64_t)row0 * p.ldb, false, none);
}

struct WgradReduce {
  const float *partial[2];
  float *dw[2];
  int64_t n4[2];  // 16-byte chunks of the gradient; 0: nothing to do
  int slices, accumulate;
};

__global__ __launch_bounds__(256) void ffn_wgrad_reduce_kernel(WgradReduce p) {
  int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int which = i >= p.n4[0] ? 1 : 0;
  if (which) i -= p.n4[0];
  if (i >= p.n4[which]) return;
  const f32x4_t *src = reinterpret_cast<const f32x4_t *>(p.partial[which]);
  f32x4_t *dst = reinterpret_cast<f32x4_t *>(p.dw[which]);
  f32x4_t v = {0.f, 0.f, 0.f, 0.f};
  if (p.accumulate) v = dst[i];
#pragma unroll 4
  for (int s = 0; s < p.slices; ++s) {
    const f32x4_t q = src[s * p.n4[which] + i];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += q[e];
  }
  dst[i] = v;
}

static hipError_t reduce(const WgradReduce &r, hipStream_t s) {
  const int64_t n = r.n4[0] + r.n4[1];
  if (n == 0) return hipSuccess;
  LaunchScope scope("ffn_wgrad_reduce", s);
  ffn_wgrad_reduce_kernel<<<(unsigned)ceil_div(n, 256), 256, 0, s>>>(r);
  return hipGetLastError();
}

hipError_t launch_ffn_dense_wgrad(const FfnArgs &a, hipStream_t s) {
  WgradParams w{};
  WgradReduce r{};
  w.T = (int)a.T;
  r.accumulate = a.accumulate ? 1 : 0;
  const FfnWgrad plan = ffn_wgrad_plan(a.T, a.d, a.F);
  const int slices = plan.slices;  // 0 without tokens
  r.slices = slices;
  w.chunk = plan.chunk;
  float *ws = static_cast<float *>(a.partial);
  for (int i = 0; i < 2; ++i) {
    GemmParams &p = w.g[i];
    p.A = (const bf16_t *)(i == 0 ? a.dh : a.dy);
    p.B = (const bf16_t *)(i == 0 ? a.x : a.a);
    p.M = i == 0 ? 2 * a.F : a.d;
    p.N = i == 0 ? a.d : a.F;
    p.lda = p.M;
    p.ldb = p.N;
    p.ldc = p.N;
    p.strideC = (int64_t)p.M * p.N;
    p.m_tiles = (p.M + plan.tile - 1) / plan.tile;
    p.n_tiles = (p.N + plan.tile - 1) / plan.tile;
    p.total = p.m_tiles * p.n_tiles * slices;
    float *dw = i == 0 ? a.dw_gu : a.dw_down;
    p.C = slices == 1 ? dw : ws;
    if (slices == 1) continue;
    r.partial[i] = ws;
    r.dw[i] = dw;
    r.n4[i] = p.strideC / 4;  // the sum of no slice is zero
    ws += slices * p.strideC;
  }
  const int total = w.g[0].total + w.g[1].total;
  if (total > 0) {
    LaunchScope scope("ffn_wgrad", s);
    const dim3 grid((unsigned)(ceil_div(total, 8) * 8));
    const bool add = slices == 1 && a.accumulate;
    if (plan.tile == 256) (add ? ffn_wgrad_kernel<256, EPI_ACC_F32> : ffn_wgrad_kernel<256, EPI_ST_F32>)<<<grid, 512, 0, s>>>(w);
    else (add ? ffn_wgrad_kernel<128, EPI_ACC_F32> : ffn_wgrad_kernel<128, EPI_ST_F32>)<<<grid, 256, 0, s>>>(w);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return reduce(r, s);
}

}  // namespace moe
