// The dense product with bias, activation and residual:
//   z = x W^T + b,  y = act(z) + residual            x [T,K], W [N,K]
//   dz = dy act'(z)                                  (linear_dact)
//   dx = (dz W) act_in'(z_in) + add                  (linear_dgrad)
//   dW (+)= dz^T x, db (+)= sum over tokens of dz    (linear_wgrad)
// on the dense block's kernels (ffn_kernel.h, ffn_few.h), a form of its own for
// input gradients of few workgroups (linear_few_dx.h) and on large
// tiles of its own (linear_wide.h; the weight
// gradient's in ffn_ilp.hip), with epilogues of its own: bias, activation and
// residual are applied to the fp32 sums, so that z and y are each rounded once.
// The input gradient's epilogue applies the derivative of the activation that
// made x, so a chain of layers needs no elementwise pass between its products.
#include "act.h"
#include "ffn_few.h"
#include "ffn_kernel.h"
#include "ffn_plan.h"
#include "linear_dw.h"
#include "linear_few_dx.h"
#include "linear_wide.h"

namespace moe {

// The few-token kernel also where 32 columns and 48 tokens a workgroup leave a CU
// to each: a workgroup's wavefronts share the sum, which a tile takes stage by
// stage. us against the tiles: 64 columns, K 4096, 192 tokens 4.4, 14.9; 512
// columns, K 2048, 320 tokens 4.7, 9.4, 768 tokens (256 workgroups) 6.1, 9.7; 2048
// columns, K 8192, 192 tokens (256) 16.6, 30.5; 256 columns, K 4096, 1400 tokens (240)
// 16.0, 18.3. The slowest, 64 columns, K 4096, 3000 tokens (252 of 16 columns) 15.8,
// 15.1.
static bool few_workgroups(const FfnTileParams &p) {
  return p.N / 32 * ceil_div(ceil_div(p.M, 16), 3) <= persistent_grid();
}

static hipError_t forward(const FfnTileParams &p, hipStream_t s) {
  LaunchScope scope("linear_fwd", s);
  if (few_workgroups(p)) return run_ffn_few<false, FFN_LINEAR>(p, s);
  switch (choose(p.M, p.N, false, false, false)) {
    case kFew: return run_ffn_few<false, FFN_LINEAR>(p, s);
    case kSmall: return run_ffn_tile<false, 64, 64, 32, 64, 4, 2, false, FFN_LINEAR>(p, s);
    case kNarrow: return run_ffn_tile<false, 64, 128, 32, 64, 2, 3, false, FFN_LINEAR>(p, s);
    case kPair: return run_ffn_tile<false, 128, 128, 64, 64, 2, 2, false, FFN_LINEAR>(p, s);
    case kHalf: return run_ffn_tile<false, 64, 128, 32, 64, 1, 3, false, FFN_LINEAR>(p, s);
    case kLarge: return run_linear_wide<false>(p, s);
    default: return run_ffn_tile<false, 128, 128, 64, 64, 1, 2, false, FFN_LINEAR>(p, s);
  }
}

hipError_t launch_linear_fwd(const LinearArgs &a, hipStream_t s) {
  FfnTileParams p{};
  p.A = (const bf16_t *)a.x;
  p.B = (const bf16_t *)a.w;
  p.C = (bf16_t *)a.y;
  p.C2 = (bf16_t *)a.z;
  p.add = (const bf16_t *)a.add;
  p.bias = (const bf16_t *)a.bias;
  p.act = a.act;
  p.M = (int)a.T;
  p.N = p.F = a.N;
  p.K = a.K;
  p.lda = p.ldb = a.K;
  p.ldc = a.N;
  return in_rounds(p, p.N, false, false, false, [&](const FfnTileParams &q) { return forward(q, s); });
}

static hipError_t dgrad(const FfnTileParams &p, hipStream_t s) {
  LaunchScope scope("linear_dgrad", s);
  if (linear_few_dx_fits(p)) return run_linear_few_dx(p, s);
  switch (choose(p.M, p.N, false, false, true)) {
    case kNarrow: return run_ffn_tile<false, 64, 128, 32, 64, 2, 2, true, FFN_LINEAR_DX>(p, s);
    case kPair: return run_ffn_tile<false, 128, 128, 64, 64, 2, 2, true, FFN_LINEAR_DX>(p, s);
    case kLarge: return run_linear_wide<true>(p, s);
    default: return run_ffn_tile<false, 128, 128, 64, 64, 1, 2, true, FFN_LINEAR_DX>(p, s);
  }
}

hipError_t launch_linear_dgrad(const LinearArgs &a, hipStream_t s) {
  FfnTileParams p{};
  p.A = (const bf16_t *)a.dz;
  p.B = (const bf16_t *)a.w;
  p.C = (bf16_t *)a.dx;
  p.H = (const bf16_t *)a.z;
  p.add = (const bf16_t *)a.add;
  p.act = a.act;
  p.M = (int)a.T;
  p.N = p.F = a.K;
  p.K = a.N;
  p.lda = a.N;
  p.ldb = a.K;
  p.ldc = a.K;
  return in_rounds(p, p.N, false, false, true, [&](const FfnTileParams &q) { return dgrad(q, s); });
}

// ---------------------------------------------------------------------------
// dz = dy act'(z), a thread 16 bytes of each; dz may be dy or z.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void linear_dact_kernel(const bf16_t *dy, const bf16_t *z, bf16_t *dz, int64_t chunks,
                                                          int act) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= chunks) return;
  float g[8], v[8];
  Elem<bf16_t>::unpack(ld16(dy + c * 8), g);
  Elem<bf16_t>::unpack(ld16(z + c * 8), v);
  const ActSigmoid sg = act_sigmoid(act);
  with_act(act, [&](auto a) {
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] *= act_slope<decltype(a)::value>(v[i], sg);
  });
  st16(dz + c * 8, Elem<bf16_t>::pack(g));
}

hipError_t launch_linear_dact(const LinearArgs &a, hipStream_t s) {
  LaunchScope scope("linear_dact", s);
  const int64_t chunks = a.T * (a.N / 8);
  linear_dact_kernel<<<(unsigned)ceil_div(chunks, 256), 256, 0, s>>>((const bf16_t *)a.dy, (const bf16_t *)a.z,
                                                                      (bf16_t *)a.dz, chunks, a.act);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// db: column sums of dz. A workgroup sums a slice of the tokens of 64
// columns, 8 to a thread and 32 tokens abreast; a second launch adds the slices
// in order.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void linear_db_partial_kernel(const bf16_t *dz, float *partial, int T, int N,
                                                                int chunk) {
  __shared__ float s[32][65];
  const int col = threadIdx.x & 7, lane = threadIdx.x >> 3;
  const int c = blockIdx.x * 64 + col * 8;
  const int first = blockIdx.y * chunk, last = min(first + chunk, T);
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int t = first + lane; t < last; t += 32) {
    float v[8];
    Elem<bf16_t>::unpack(ld16(dz + (int64_t)t * N + c), v);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] += v[i];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) s[lane][col * 8 + i] = sum[i];
  __syncthreads();
  if (threadIdx.x >= 64) return;
  float v = 0.f;
#pragma unroll
  for (int l = 0; l < 32; ++l) v += s[l][threadIdx.x];
  partial[(int64_t)blockIdx.y * N + blockIdx.x * 64 + threadIdx.x] = v;
}

__global__ __launch_bounds__(64) void linear_db_reduce_kernel(const float *partial, float *db, int N, int slices,
                                                              int accumulate) {
  const int c = blockIdx.x * 64 + threadIdx.x;  // N is a multiple of 64
  float v = 0.f;
#pragma unroll 8
  for (int i = 0; i < slices; ++i) v += partial[(int64_t)i * N + c];
  db[c] = accumulate ? db[c] + v : v;
}

static hipError_t linear_db(const LinearArgs &a, hipStream_t s) {
  const int slices = linear_db_slices(a.T);
  if (slices > 0) {
    LaunchScope scope("linear_db", s);
    const int chunk = (int)(ceil_div(ceil_div(a.T, slices), 32) * 32);
    linear_db_partial_kernel<<<dim3((unsigned)(a.N / 64), (unsigned)slices), 256, 0, s>>>(
        (const bf16_t *)a.dz, a.db_partial, (int)a.T, a.N, chunk);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  LaunchScope scope("linear_db_reduce", s);
  linear_db_reduce_kernel<<<(unsigned)(a.N / 64), 64, 0, s>>>(a.db_partial, a.db, a.N, slices, a.accumulate ? 1 : 0);
  return hipGetLastError();
}

// The weight gradient's large tiles: db comes with them, one launch adds the
// slices of both. The small tiles (ffn_ilp.hip) leave db to the pass above.
hipError_t launch_linear_wgrad(const LinearArgs &a, hipStream_t s) {
  const FfnWgrad plan = linear_wgrad_plan(a.T, a.K, a.N);
  if (plan.tile != kPpTile) {
    const hipError_t err = launch_linear_dw(a, s);
    return err != hipSuccess || !a.db ? err : linear_db(a, s);
  }
  const bool direct = plan.slices == 1;
  if (plan.slices > 0) {
    LaunchScope scope("linear_wgrad", s);
    LinearDwParams p{};
    p.dz = (const bf16_t *)a.dz;
    p.x = (const bf16_t *)a.x;
    p.dw = direct ? a.dw : a.partial;
    p.db = !a.db ? nullptr : direct ? a.db : a.db_partial;
    p.T = (int)a.T;
    p.K = a.K;
    p.N = a.N;
    p.chunk = plan.chunk;
    p.slices = plan.slices;
    p.n_tiles = (a.N + kPpTile - 1) / kPpTile;
    p.k_tiles = (a.K + kPpTile - 1) / kPpTile;
    const int64_t total = (int64_t)p.n_tiles * p.k_tiles * plan.slices;
    const dim3 grid((unsigned)std::min<int64_t>(persistent_grid(), ceil_div(total, 8) * 8));
    if (direct && a.accumulate) linear_dw_kernel<true><<<grid, kPpThreads, 0, s>>>(p);
    else linear_dw_kernel<false><<<grid, kPpThreads, 0, s>>>(p);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  if (direct) return hipSuccess;
  LaunchScope scope("linear_wgrad_reduce", s);
  LinearDwReduce r{};
  r.dw_part = a.partial;
  r.db_part = a.db_partial;
  r.dw = a.dw;
  r.db = a.db;
  r.dw4 = (int64_t)a.N * a.K / 4;
  r.db4 = a.db ? a.N / 4 : 0;
  r.slices = plan.slices;
  r.accumulate = a.accumulate ? 1 : 0;
  linear_dw_reduce_kernel<<<(unsigned)ceil_div(r.dw4 + r.db4, 256), 256, 0, s>>>(r);
  return hipGetLastError();
}

}  // namespace moe
