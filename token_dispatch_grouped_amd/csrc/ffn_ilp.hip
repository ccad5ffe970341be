// Weight gradients of the dense gated feed-forward block:
//   dw_down [d,F]  (+)= dy^T a     dw_gu [2F,d] (+)= dh^T x     (fp32)
// The grouped products' 256 x 256 tile with both operands k-major. There are
// few output tiles and a long sum over the tokens, so the tokens are split
// into slices: every (tile, slice) pair is a workgroup that writes fp32
// partial sums to the workspace, and a second kernel adds the slices in
// order (no atomics: results are the same bits run to run).
#include "ffn_wide.h"

namespace moe {

template hipError_t run_ffn_wide<false, EPI_SWIGLU_FWD>(GemmParams, hipStream_t);

constexpr int kWgBM = kGemmBM, kWgBN = kGemmBN;

template <int EPI>
__global__ __launch_bounds__(512, 1) void ffn_wgrad_kernel(GemmParams p, int T, int chunk) {
  __shared__ u32x4_t lds[2 * (kWgBM + kWgBN) * kStageK * 2 / 16];
  int lo, hi;
  xcd_range(blockIdx.x & 7, p.total, lo, hi);
  const int id = lo + (int)(blockIdx.x >> 3);
  if (id >= hi) return;
  const int tiles = p.m_tiles * p.n_tiles;
  const int slice = id / tiles, r = id - slice * tiles;
  const int mt = r / p.n_tiles, nt = r - mt * p.n_tiles;
  const int row0 = slice * chunk;
  const int kdim = min(chunk, T - row0);
  const int m0 = mt * kWgBM;
  auto none = [&](NextTile &nx) { nx.valid = false; };
  gg_tile<kWgBM, kWgBN, kWgBM / 2, kWgBN / 4, 8, true, true, EPI, true, kStageK, kStages>(
      p, lds, slice, m0, nt, min(kWgBM, p.M - m0), kdim, 0, p.A + (int64_t)row0 * p.lda + m0,
      p.B + (int64_t)row0 * p.ldb, false, none);
}

__global__ __launch_bounds__(256) void ffn_wgrad_reduce_kernel(const float *partial, float *dw, int64_t n4, int slices,
                                                               int accumulate) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n4) return;
  f32x4_t v = {0.f, 0.f, 0.f, 0.f};
  if (accumulate) v = reinterpret_cast<const f32x4_t *>(dw)[i];
  for (int s = 0; s < slices; ++s) {
    const f32x4_t q = reinterpret_cast<const f32x4_t *>(partial)[s * n4 + i];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += q[e];
  }
  reinterpret_cast<f32x4_t *>(dw)[i] = v;
}

static hipError_t wgrad(const char *name, const char *reduce_name, const void *A, const void *B, float *dw, int M,
                        int N, const FfnArgs &a, hipStream_t s) {
  GemmParams p{};
  p.A = (const bf16_t *)A;
  p.B = (const bf16_t *)B;
  p.M = M;
  p.N = N;
  p.lda = M;
  p.ldb = N;
  p.ldc = N;
  p.strideC = (int64_t)M * N;
  p.m_tiles = (M + kWgBM - 1) / kWgBM;
  p.n_tiles = (N + kWgBN - 1) / kWgBN;
  const FfnSlices sl = ffn_wgrad_slices(a.T, M, N);
  p.total = p.m_tiles * p.n_tiles * sl.slices;
  const dim3 grid((unsigned)(ceil_div(p.total, 8) * 8));
  {
    LaunchScope scope(name, s);
    if (sl.slices > 1) {
      p.C = a.partial;
      ffn_wgrad_kernel<EPI_ST_F32><<<grid, 512, 0, s>>>(p, (int)a.T, sl.chunk);
    } else {
      p.C = dw;
      if (a.accumulate) ffn_wgrad_kernel<EPI_ACC_F32><<<grid, 512, 0, s>>>(p, (int)a.T, sl.chunk);
      else ffn_wgrad_kernel<EPI_ST_F32><<<grid, 512, 0, s>>>(p, (int)a.T, sl.chunk);
    }
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || sl.slices == 1) return err;
  }
  LaunchScope scope(reduce_name, s);
  const int64_t n4 = (int64_t)M * N / 4;
  ffn_wgrad_reduce_kernel<<<(unsigned)ceil_div(n4, 256), 256, 0, s>>>((const float *)a.partial, dw, n4, sl.slices,
                                                                     a.accumulate ? 1 : 0);
  return hipGetLastError();
}

hipError_t launch_ffn_dense_wgrad(const FfnArgs &a, hipStream_t s) {
  if (a.T == 0) {  // no tokens: the gradients are zero
    const int64_t n = (int64_t)a.d * a.F / 4;
    LaunchScope scope("ffn_wgrad_zero", s);
    ffn_wgrad_reduce_kernel<<<(unsigned)ceil_div(n, 256), 256, 0, s>>>(nullptr, a.dw_down, n, 0, 0);
    ffn_wgrad_reduce_kernel<<<(unsigned)ceil_div(2 * n, 256), 256, 0, s>>>(nullptr, a.dw_gu, 2 * n, 0, 0);
    return hipGetLastError();
  }
  const hipError_t err = wgrad("ffn_down_wgrad", "ffn_down_wgrad_reduce", a.dy, a.a, a.dw_down, a.d, a.F, a, s);
  if (err != hipSuccess) return err;
  return wgrad("ffn_gateup_wgrad", "ffn_gateup_wgrad_reduce", a.dh, a.x, a.dw_gu, 2 * a.F, a.d, a, s);
}

}  // namespace moe
