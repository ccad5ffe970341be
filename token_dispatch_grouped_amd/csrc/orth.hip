// Orthogonalisation of a batch of matrices by Newton-Schulz products, and the
// optimiser step around it (Muon). orth_kernel.h has the products.
//
//   norm    per matrix sum(U^2) in 64 bits, as partial sums in a fixed order
//   prep    X0 = U / (|U| + eps) to two fp16 halves, short side first, padded
//           with zeros; the step also writes the momentum and clears the
//           gradient here
//   5 x     gram, poly, step; the last step's epilogue writes O, or w = w (1 -
//           lr wd) - lr scale O and its bf16 copy
//
// U is the matrix given, or  buf = mu buf + g,  U = g + mu buf (Nesterov) or
// buf; it is formed twice, in norm and in prep, from the same inputs.
#include "kernels.h"
#include "orth_kernel.h"
#include "validate.h"

namespace moe {

constexpr int kOrthThreads = 256;

struct OrthIo {
  const void *x;          // orthogonalise: fp32 or bf16
  float *grad, *mom;      // step
  float mu, grad_scale;
  int nesterov, zero_grad;
  int rows, cols;         // of the matrices given
  int parts;              // partial sums of a matrix
  double *partial;        // [batch, parts]
  float eps;
  int tall;               // rows > cols: X is the transpose
  half_t *hi, *lo;        // X [S, L] per matrix; lo may be NULL
  int64_t ldx, stride_x;
};

enum { SRC_F32 = 0, SRC_BF16 = 1, SRC_MUON = 2 };

// The inputs of U at 4 consecutive elements from `e` on (of the whole batch),
// `n` of them there (at least one); vec: they are one aligned vector.
template <int SRC>
struct OrthIn {
  float g[4], m[4];
  MOE_DEVICE void load(const OrthIo &p, int64_t e, int n, bool vec) {
    if constexpr (SRC == SRC_BF16) {
      const bf16_t *x = (const bf16_t *)p.x + e;
      if (vec) {
        const uint2 v = *reinterpret_cast<const uint2 *>(x);
        g[0] = __uint_as_float(v.x << 16);
        g[1] = __uint_as_float(v.x & 0xffff0000u);
        g[2] = __uint_as_float(v.y << 16);
        g[3] = __uint_as_float(v.y & 0xffff0000u);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) g[q] = q < n ? bf2f(x[q]) : 0.f;
      }
      return;
    }
    const float *x = SRC == SRC_F32 ? (const float *)p.x + e : p.grad + e;
    if (vec) {
      const f32x4_t v = *reinterpret_cast<const f32x4_t *>(x);
#pragma unroll
      for (int q = 0; q < 4; ++q) g[q] = v[q];
      if constexpr (SRC == SRC_MUON) {
        const f32x4_t w = *reinterpret_cast<const f32x4_t *>(p.mom + e);
#pragma unroll
        for (int q = 0; q < 4; ++q) m[q] = w[q];
      }
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        g[q] = q < n ? x[q] : 0.f;
        if (SRC == SRC_MUON) m[q] = q < n ? p.mom[e + q] : 0.f;
      }
    }
  }
  MOE_DEVICE void zero() {
#pragma unroll
    for (int q = 0; q < 4; ++q) g[q] = m[q] = 0.f;
  }
  // g becomes U, m the new momentum
  MOE_DEVICE void combine(const OrthIo &p) {
    if constexpr (SRC == SRC_MUON) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float gs = g[q] * p.grad_scale;
        m[q] = fmaf(p.mu, m[q], gs);
        g[q] = p.nesterov ? fmaf(p.mu, m[q], gs) : m[q];
      }
    }
  }
};

MOE_DEVICE double wave_sum64(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
  return v;
}

// Squares are summed in 64 bits: no gradient is too small or too large for it.
template <int SRC>
__global__ __launch_bounds__(kOrthThreads) void orth_norm_kernel(OrthIo p) {
  __shared__ double part[kOrthThreads / kWave];
  const int64_t n = (int64_t)p.rows * p.cols;
  const int64_t mat = blockIdx.x / p.parts;
  const int part_id = (int)(blockIdx.x - mat * p.parts);
  const int64_t chunk = ((n + p.parts - 1) / p.parts + 3) & ~(int64_t)3;
  const int64_t first = part_id * chunk, last = first + chunk < n ? first + chunk : n;
  const bool aligned = (n & 3) == 0;  // every matrix starts on a vector
  double sum = 0.0;
  auto add = [&](OrthIn<SRC> &in) {
    in.combine(p);
#pragma unroll
    for (int q = 0; q < 4; ++q) sum = fma((double)in.g[q], (double)in.g[q], sum);
  };
  const int64_t at = mat * n + threadIdx.x * 4;
  constexpr int kRow = kOrthThreads * 4;
  int64_t i = first;
  if (aligned) {  // whole rows of vectors, the loads of four in flight together
    for (; i + 4 * kRow <= last; i += 4 * kRow) {
      OrthIn<SRC> in[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) in[k].load(p, at + i + k * kRow, 4, true);
#pragma unroll
      for (int k = 0; k < 4; ++k) add(in[k]);
    }
  }
  // the rest, and matrices that start on no vector
  for (; i < last; i += 4 * kRow) {
    OrthIn<SRC> in[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t e = i + k * kRow + threadIdx.x * 4;
      const int left = (int)(last - e < 4 ? last - e : 4);
      in[k].zero();
      if (left > 0) in[k].load(p, mat * n + e, left, aligned && left == 4);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) add(in[k]);
  }
  sum = wave_sum64(sum);
  if ((threadIdx.x & (kWave - 1)) == 0) part[threadIdx.x / kWave] = sum;
  __syncthreads();
  if (threadIdx.x == 0) p.partial[blockIdx.x] = (part[0] + part[1]) + (part[2] + part[3]);
}

// X0 and the momentum. Rows and columns past the matrix's end are zeros (the
// padding of X). Where X is the matrix itself a workgroup takes 4096 elements of X
// on end, where it is the transpose, a 64 x 64 tile, turned in LDS.
constexpr int kPrepVectors = 4;  // of 4 elements, a thread's
template <int SRC, bool TALL>
__global__ __launch_bounds__(kOrthThreads) void orth_prep_kernel(OrthIo p) {
  __shared__ float tile[TALL ? 64 : 1][65];
  const int rt = (p.rows + 63) / 64, ct = (p.cols + 63) / 64;
  const int row_vectors = ct * 16, vectors = rt * 64 * row_vectors;  // of X, padded
  const int per = TALL ? rt * ct : (vectors + kPrepVectors * kOrthThreads - 1) / (kPrepVectors * kOrthThreads);
  const int64_t mat = blockIdx.x / per;
  const int t = (int)(blockIdx.x - mat * per);
  const int r0 = t / ct * 64, c0 = t % ct * 64;
  const int lane = threadIdx.x & (kWave - 1);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t base = mat * p.rows * p.cols;
  const bool vec = (p.cols & 3) == 0;
  OrthIn<SRC> in[kPrepVectors];
  int row[kPrepVectors], col[kPrepVectors], left[kPrepVectors];
#pragma unroll
  for (int k = 0; k < kPrepVectors; ++k) {
    const int i = (t * kPrepVectors + k) * kOrthThreads + threadIdx.x;
    row[k] = TALL ? r0 + ty + 16 * k : i / row_vectors;
    col[k] = TALL ? c0 + tx * 4 : (i - row[k] * row_vectors) * 4;
    left[k] = row[k] < p.rows ? min(4, p.cols - col[k]) : 0;
    in[k].zero();
    if (left[k] > 0) in[k].load(p, base + (int64_t)row[k] * p.cols + col[k], left[k], vec);
  }
  double sum = 0.0;
  for (int i = lane; i < p.parts; i += kWave) sum += p.partial[mat * p.parts + i];
  sum = wave_sum64(sum);
  // a matrix that holds an infinity or a NaN becomes NaN altogether
  const double scale = sum < __builtin_huge_val() ? (double)kOrthScale / (sqrt(sum) + (double)p.eps) : __builtin_nan("");
  auto put = [&](int64_t o, const float (&v)[4]) {
    *reinterpret_cast<uint2 *>(p.hi + mat * p.stride_x + o) = make_uint2(pack_h2(v[0], v[1]), pack_h2(v[2], v[3]));
    if (!p.lo) return;
    float l[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) l[q] = v[q] - h2f(f2h(v[q]));
    *reinterpret_cast<uint2 *>(p.lo + mat * p.stride_x + o) = make_uint2(pack_h2(l[0], l[1]), pack_h2(l[2], l[3]));
  };
#pragma unroll
  for (int k = 0; k < kPrepVectors; ++k) {
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (left[k] > 0) {
      const int64_t e = base + (int64_t)row[k] * p.cols + col[k];
      in[k].combine(p);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (q < left[k]) v[q] = (float)((double)in[k].g[q] * scale);
      if constexpr (SRC == SRC_MUON) {
        const float (&buf)[4] = in[k].m;
        if (vec) {
          *reinterpret_cast<f32x4_t *>(p.mom + e) = f32x4_t{buf[0], buf[1], buf[2], buf[3]};
          if (p.zero_grad) *reinterpret_cast<f32x4_t *>(p.grad + e) = f32x4_t{0.f, 0.f, 0.f, 0.f};
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (q < left[k]) {
              p.mom[e + q] = buf[q];
              if (p.zero_grad) p.grad[e + q] = 0.f;
            }
        }
      }
    }
    if constexpr (TALL) {
#pragma unroll
      for (int q = 0; q < 4; ++q) tile[ty + 16 * k][tx * 4 + q] = v[q];
    } else if (row[k] < rt * 64) {
      put((int64_t)row[k] * p.ldx + col[k], v);
    }
  }
  if constexpr (TALL) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = tile[tx * 4 + q][ty + 16 * k];
      put((int64_t)(c0 + ty + 16 * k) * p.ldx + r0 + tx * 4, v);
    }
  }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
//   small   64 x 64 tiles in 2 k groups (step: 64 x 128 in one), rings of 4 stages
//   pair    128 x 128 tiles, a ring of 4 stages, a workgroup a CU
//   square  128 x 128 tiles, a ring of 2 stages, two workgroups a CU
//   large   256 x 256 tiles
enum OrthTile { kSmall, kPair, kSquare, kLarge };

static OrthTile choose(int M, int N, int64_t batch, bool sym, bool both) {
  const int64_t cus = persistent_grid();
  const auto tiles = [&](int bm, int bn) {
    const int64_t m = ceil_div(M, bm), n = ceil_div(N, bn);
    return batch * (sym ? m * (m + 1) / 2 : m * n);
  };
  if (tiles(64, sym ? 64 : 128) <= cus) return kSmall;
  if (tiles(128, 128) <= cus) return kPair;
  if (both) return kSquare;
  return 145 * ceil_div(tiles(256, 256), cus) < 100 * ceil_div(tiles(128, 128), 2 * cus) ? kLarge : kSquare;
}

template <bool BOTH>
static hipError_t sym_product(OrthTileParams p, int64_t batch, bool gram, hipStream_t s) {
  const OrthTile t = choose(p.M, p.N, batch, true, BOTH);
  if (gram && t == kPair) {
    // long sums of tiles that leave CUs idle: slices of them, joined by a launch
    // of its own, which ends in the epilogue
    const int64_t m = ceil_div(p.M, 128);
    p.slices = orth_gram_slices(p.M, p.K, batch * m * (m + 1) / 2);
    if (p.slices > 1) {
      {
        LaunchScope scope("orth_gram", s);
        const hipError_t err = run_orth_tile<128, 128, 32, 64, 1, 2, ORTH_GRAM, BOTH>(p, batch, s);
        if (err != hipSuccess) return err;
      }
      LaunchScope scope("orth_gram_sum", s);
      return run_orth_sum<128, 32, 64, ORTH_GRAM, BOTH>(p, batch, s);
    }
  }
  LaunchScope scope(gram ? "orth_gram" : "orth_poly", s);
  if (gram) {
    switch (t) {
      case kSmall: return run_orth_tile<64, 64, 16, 64, 2, 4, ORTH_GRAM, BOTH>(p, batch, s);
      case kPair: return run_orth_tile<128, 128, 32, 64, 1, 4, ORTH_GRAM, BOTH>(p, batch, s);
      case kSquare: return run_orth_tile<128, 128, 32, 64, 1, 2, ORTH_GRAM, BOTH>(p, batch, s);
      default: return run_orth_wide<ORTH_GRAM>(p, batch, s);
    }
  }
  switch (t) {
    case kSmall: return run_orth_tile<64, 64, 16, 64, 2, 4, ORTH_POLY, BOTH>(p, batch, s);
    case kPair: return run_orth_tile<128, 128, 32, 64, 1, 4, ORTH_POLY, BOTH>(p, batch, s);
    case kSquare: return run_orth_tile<128, 128, 32, 64, 1, 2, ORTH_POLY, BOTH>(p, batch, s);
    default: return run_orth_wide<ORTH_POLY>(p, batch, s);
  }
}

template <int MODE, bool BOTH>
static hipError_t step_tiles(const OrthTileParams &p, int64_t batch, hipStream_t s) {
  switch (choose(p.M, p.N, batch, false, BOTH)) {
    case kSmall: return run_orth_tile<64, 128, 16, 64, 1, 4, MODE, BOTH>(p, batch, s);
    case kPair: return run_orth_tile<128, 128, 32, 64, 1, 4, MODE, BOTH>(p, batch, s);
    case kSquare: return run_orth_tile<128, 128, 32, 64, 1, 2, MODE, BOTH>(p, batch, s);
    default: return run_orth_wide<MODE>(p, batch, s);
  }
}

template <bool BOTH>
static hipError_t step_product(const OrthTileParams &p, int64_t batch, bool last, hipStream_t s) {
  LaunchScope scope(last ? "orth_last" : "orth_step", s);
  if (!last) return step_tiles<ORTH_STEP, BOTH>(p, batch, s);
  return p.out.param ? step_tiles<ORTH_LAST_MUON, BOTH>(p, batch, s) : step_tiles<ORTH_LAST, BOTH>(p, batch, s);
}

template <int SRC>
static hipError_t enter(const OrthIo &io, int64_t batch, hipStream_t s) {
  {
    LaunchScope scope("orth_norm", s);
    orth_norm_kernel<SRC><<<(unsigned)(batch * io.parts), kOrthThreads, 0, s>>>(io);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  LaunchScope scope("orth_prep", s);
  const int64_t tiles = ceil_div(io.rows, 64) * ceil_div(io.cols, 64);
  if (io.tall) {
    orth_prep_kernel<SRC, true><<<(unsigned)(batch * tiles), kOrthThreads, 0, s>>>(io);
  } else {
    const int64_t per = ceil_div(tiles * 1024, kPrepVectors * kOrthThreads);
    orth_prep_kernel<SRC, false><<<(unsigned)(batch * per), kOrthThreads, 0, s>>>(io);
  }
  return hipGetLastError();
}

hipError_t launch_orth(const OrthArgs &a, hipStream_t s) {
  const OrthWorkspace w = orth_workspace(a.batch, a.rows, a.cols);
  char *ws = static_cast<char *>(a.ws);
  half_t *hi[2] = {(half_t *)(ws + w.hi[0]), (half_t *)(ws + w.hi[1])};
  half_t *lo[2] = {(half_t *)(ws + w.lo[0]), (half_t *)(ws + w.lo[1])};
  half_t *A = (half_t *)(ws + w.a), *B = (half_t *)(ws + w.b);
  const bool both = orth_both_halves(w.S);
  half_t *Alo = both ? (half_t *)(ws + w.alo) : nullptr, *Blo = both ? (half_t *)(ws + w.blo) : nullptr;
  float *da = (float *)(ws + w.da), *db = (float *)(ws + w.db);
  OrthIo io{};
  io.x = a.x;
  io.grad = a.grad;
  io.mom = a.momentum;
  io.mu = a.mu;
  io.grad_scale = a.grad_scale;
  io.nesterov = a.nesterov ? 1 : 0;
  io.zero_grad = a.zero_grad ? 1 : 0;
  io.rows = a.rows;
  io.cols = a.cols;
  io.parts = w.parts;
  io.partial = (double *)(ws + w.partial);
  io.eps = a.eps;
  io.tall = a.rows > a.cols ? 1 : 0;
  io.hi = hi[0];
  io.lo = lo[0];
  io.ldx = w.L;
  io.stride_x = (int64_t)w.S * w.L;
  OrthOut out{};
  out.param = a.param;
  out.lowp = (bf16_t *)(a.param ? a.param_bf16 : a.o);
  out.rows = a.rows;
  out.cols = a.cols;
  out.tall = a.rows > a.cols ? 1 : 0;
  out.decay = a.decay;
  out.step_size = a.step_size;
  const bool muon = a.param != nullptr;
  hipError_t err = muon      ? enter<SRC_MUON>(io, a.batch, s)
                   : a.bf16 ? enter<SRC_BF16>(io, a.batch, s)
                            : enter<SRC_F32>(io, a.batch, s);
  int cur = 0;
  for (int k = 0; k < a.steps && err == hipSuccess; ++k) {
    OrthTileParams p{};
    p.ca = a.coef[0];
    p.cb = a.coef[1];
    p.cc = a.coef[2];
    p.S = w.S;
    p.A = p.B = hi[cur];
    p.C = A;
    p.sums = reinterpret_cast<f32x4_t *>(ws + w.sums);
    p.diag_out = da;
    p.M = p.N = w.S;
    p.K = w.L;
    p.lda = p.ldb = w.L;
    p.ldc = w.S;
    p.strideA = p.strideB = io.stride_x;
    p.strideC = (int64_t)w.S * w.S;
    if (both) {
      p.Alo = p.Blo = lo[cur];
      p.Clo = Alo;
    }
    err = both ? sym_product<true>(p, a.batch, true, s) : sym_product<false>(p, a.batch, true, s);
    if (err != hipSuccess) break;
    p.A = p.B = A;
    p.C = B;
    p.Alo = p.Blo = p.Xlo = Alo;
    p.Clo = Blo;
    p.diag = da;
    p.diag_out = db;
    p.K = w.S;
    p.lda = p.ldb = w.S;
    p.strideA = p.strideB = p.strideC;
    err = both ? sym_product<true>(p, a.batch, false, s) : sym_product<false>(p, a.batch, false, s);
    if (err != hipSuccess) break;
    p.A = B;
    p.Alo = Blo;
    p.B = hi[cur];
    p.Blo = p.Xlo = lo[cur];
    p.C = hi[cur ^ 1];
    p.Clo = k + (both ? 1 : 2) < a.steps ? lo[cur ^ 1] : nullptr;
    p.out = out;
    p.diag = db;
    p.N = w.L;
    p.ldb = p.ldc = w.L;
    p.strideB = p.strideC = io.stride_x;
    const bool last = k + 1 == a.steps;
    err = both ? step_product<true>(p, a.batch, last, s) : step_product<false>(p, a.batch, last, s);
    cur ^= 1;
  }
  return err;
}

}  // namespace moe
