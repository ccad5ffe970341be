// Layer norm with the residual's addition, and its backward pass. Bound by
// HBM as the RMS norm is (norm.hip, whose split of rows over threads, border
// for streams past the memory-side cache and shares of the backward pass
// these kernels take over): every kernel reads each input once and writes each
// output once, a row held in registers between the reductions and the scaling.
//
//   forward   r = round(x + residual);  m = mean(r);  rstd = 1 / sqrt(mean((r - m)^2) + eps)
//             y = (r - m) * rstd * w + b
//   backward  n = (r - m) * rstd, g = dy * w:
//             dx = rstd * (g - mean(g) - n * mean(g * n)) + dres
//             dw = sum over the rows of dy * n,  db = sum over the rows of dy
//
// The mean is summed twice, as m0 = sum(r) / d rounded to fp32 and delta =
// sum(r - m0) / d, so that rows whose mean is many times their spread keep
// the spread's digits: (r - m0) is exact there, and the variance is
// sum((r - m0)^2) / d - delta^2. Where delta is more than the spread, m0 + delta
// takes m0's place and the second sums are taken again.
#include "common.h"
#include "kernels.h"
#include "mx8.h"

namespace moe {

constexpr int kLnThreads = 256;
constexpr int64_t kLnCachedBytes = (int64_t)128 << 20;

template <bool NT>
MOE_DEVICE u32x4_t ln_ld(const void *p) {
  return NT ? ld16_nt(p) : ld16(p);
}
template <bool NT>
MOE_DEVICE void ln_st(void *p, const u32x4_t &v) {
  if (NT) st16_nt(p, v);
  else st16(p, v);
}

// Two sums over the TPR threads of a row, the same bits in every thread. TPR =
// 64 is one wavefront; 256 is the workgroup, through `part`, which must not be
// in use by an earlier sum.
typedef float LnPart[2][kLnThreads / kWave];
template <int TPR>
MOE_DEVICE void row_sums(float &a, float &b, LnPart &part) {
  a = wave_sum_dpp(a);
  b = wave_sum_dpp(b);
  if (TPR == kWave) return;
  if ((threadIdx.x & (kWave - 1)) == 0) {
    part[0][threadIdx.x / kWave] = a;
    part[1][threadIdx.x / kWave] = b;
  }
  __syncthreads();
  a = (part[0][0] + part[0][1]) + (part[0][2] + part[0][3]);
  b = (part[1][0] + part[1][1]) + (part[1][2] + part[1][3]);
}

// What normalises a row: n = ((r * scale - m0) - delta) * mul.
struct RowNorm {
  float scale, m0, delta, mul;
  float mean, rstd;  // what the backward pass reads
  MOE_DEVICE float operator()(float r) const { return (fmaf(r, scale, -m0) - delta) * mul; }
};

// The statistics of a row. each(f) calls f on every value of the row that the
// thread holds.
// A row whose sums pass fp32's range (|r| from about 2^60 on) is taken again
// over r 2^-80, where they do not: 65536 squares below 2^96 each. Spreads that
// get lost below that way are smaller than a step of such a row's values.
template <int TPR, typename Each>
MOE_DEVICE RowNorm row_norm(Each each, float inv_d, float eps, LnPart (&part)[4]) {
  constexpr float kDown = 0x1p-80f, kUp = 0x1p80f;
  RowNorm k;
  auto sums = [&](float scale, LnPart &pa, LnPart &pb, float &var) {
    float s = 0.f, none = 0.f;
    each([&](float r) { s = fmaf(r, scale, s); });
    row_sums<TPR>(s, none, pa);
    k.scale = scale;
    k.m0 = s * inv_d;
    float s2;
    // Again from m0 + delta where m0 is off by more than the spread (a row of one
    // value, or of steps of it): there the variance is what is left of two equal
    // terms, and n was a rounding of m0's error (1e4, where r is 1.6e15 throughout).
    for (bool again = false;; again = true) {
      float s1 = 0.f;
      s2 = 0.f;
      each([&](float r) {
        const float c = fmaf(r, scale, -k.m0);
        s1 += c;
        s2 = fmaf(c, c, s2);
      });
      row_sums<TPR>(s1, s2, again ? pa : pb);  // all have read pa by the sum in pb
      k.delta = s1 * inv_d;
      var = fmaxf(fmaf(s2, inv_d, -k.delta * k.delta), 0.f);
      if (again || !(var < k.delta * k.delta)) break;  // all threads of the row alike
      k.m0 += k.delta;
    }
    return s2;
  };
  float var;
  const float s2 = sums(1.f, part[0], part[1], var);
  k.mean = k.m0 + k.delta;
  k.rstd = 1.0f / sqrtf(var + eps);
  k.mul = k.rstd;
  if (!(s2 < __builtin_huge_valf())) {  // all threads of the row alike
    const float again = sums(kDown, part[2], part[3], var);
    if (!(again < __builtin_huge_valf())) var = __builtin_nanf("");  // an infinity or a NaN in the row
    k.mean = (k.m0 + k.delta) * kUp;
    const float sd = sqrtf(var) * kUp;
    k.rstd = sd < 0x1p60f ? 1.0f / sqrtf(fmaf(sd, sd, eps)) : 1.0f / sd;
    k.mul = k.rstd * kUp;
    if (k.mul == __builtin_huge_valf()) k.mul = 0x1p127f;  // a constant row with a tiny eps: 0, not 0 * inf
  }
  return k;
}

struct LnFwdParams {
  const void *x, *residual, *w, *b;
  void *r, *y;
  float *mean, *rstd;
  int64_t T;
  int d;
  float inv_d, eps;
};

// y of one chunk of V values
template <typename T>
MOE_DEVICE u32x4_t ln_affine(const RowNorm &k, const u32x4_t &r, const u32x4_t &w, const u32x4_t &b) {
  constexpr int V = Elem<T>::kVec;
  float rv[V], wv[V], bv[V];
  Elem<T>::unpack(r, rv);
  Elem<T>::unpack(w, wv);
  Elem<T>::unpack(b, bv);
#pragma unroll
  for (int i = 0; i < V; ++i) rv[i] = fmaf(k(rv[i]), wv[i], bv[i]);
  return Elem<T>::pack(rv);
}

// A row in TPR threads, NV chunks of 16 bytes each.
template <typename T, int TPR, int NV, bool NT>
__global__ __launch_bounds__(kLnThreads) void layernorm_fwd_kernel(LnFwdParams p) {
  constexpr int V = Elem<T>::kVec;
  __shared__ LnPart part[4];
  const int lane = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * (kLnThreads / TPR) + threadIdx.x / TPR;
  if (row >= p.T) return;  // whole wavefronts only, and no barrier below for TPR = 64
  const int n = p.d / V;
  const T *x = (const T *)p.x + row * p.d;
  const T *res = p.residual ? (const T *)p.residual + row * p.d : nullptr;
  u32x4_t xv[NV], rv[NV], wv[NV], bv[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = j * TPR + lane;
    const int cc = c < n ? c : 0;
    xv[j] = ln_ld<NT>(x + cc * V);
    if (res) rv[j] = ln_ld<NT>(res + cc * V);
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = j * TPR + lane;
    const int cc = c < n ? c : 0;
    wv[j] = ld16((const T *)p.w + cc * V);
    bv[j] = p.b ? ld16((const T *)p.b + cc * V) : u32x4_t{0u, 0u, 0u, 0u};
  }
  if (res) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = j * TPR + lane;
      float a[V], e[V];
      Elem<T>::unpack(xv[j], a);
      Elem<T>::unpack(rv[j], e);
#pragma unroll
      for (int i = 0; i < V; ++i) a[i] += e[i];
      xv[j] = Elem<T>::pack(a);  // rounded once: from here on r is what the row holds
      if (c < n) ln_st<NT>((T *)p.r + row * p.d + c * V, xv[j]);
    }
  }
  auto each = [&](auto f) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float a[V];
      Elem<T>::unpack(xv[j], a);
      if (j * TPR + lane < n) {
#pragma unroll
        for (int i = 0; i < V; ++i) f(a[i]);
      }
    }
  };
  const RowNorm k = row_norm<TPR>(each, p.inv_d, p.eps, part);
  if (lane == 0) {
    p.mean[row] = k.mean;
    p.rstd[row] = k.rstd;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = j * TPR + lane;
    if (c < n) ln_st<NT>((T *)p.y + row * p.d + c * V, ln_affine<T>(k, xv[j], wv[j], bv[j]));
  }
}

// Rows too long for registers: a workgroup per row, which reads it again from
// the caches for each pass. Every element is read and written by one thread,
// which reads its r back rather than x, so r may overwrite x.
template <typename T>
__global__ __launch_bounds__(kLnThreads) void layernorm_fwd_long_kernel(LnFwdParams p) {
  constexpr int V = Elem<T>::kVec;
  __shared__ LnPart part[4];
  const int64_t row = blockIdx.x;
  const int n = p.d / V;
  const T *src = (const T *)p.x + row * p.d;
  if (p.residual) {
    T *r = (T *)p.r + row * p.d;
    for (int c = threadIdx.x; c < n; c += kLnThreads) {
      float a[V], e[V];
      Elem<T>::unpack(ld16(src + c * V), a);
      Elem<T>::unpack(ld16((const T *)p.residual + row * p.d + c * V), e);
#pragma unroll
      for (int i = 0; i < V; ++i) a[i] += e[i];
      st16(r + c * V, Elem<T>::pack(a));
    }
    src = r;
  }
  auto each = [&](auto f) {
    for (int c = threadIdx.x; c < n; c += kLnThreads) {
      float a[V];
      Elem<T>::unpack(ld16(src + c * V), a);
#pragma unroll
      for (int i = 0; i < V; ++i) f(a[i]);
    }
  };
  const RowNorm k = row_norm<kLnThreads>(each, p.inv_d, p.eps, part);
  if (threadIdx.x == 0) {
    p.mean[row] = k.mean;
    p.rstd[row] = k.rstd;
  }
  for (int c = threadIdx.x; c < n; c += kLnThreads) {
    const u32x4_t b = p.b ? ld16((const T *)p.b + c * V) : u32x4_t{0u, 0u, 0u, 0u};
    st16((T *)p.y + row * p.d + c * V, ln_affine<T>(k, ld16(src + c * V), ld16((const T *)p.w + c * V), b));
  }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
struct LnBwdParams {
  const void *dy, *r, *w, *dres;
  const float *mean, *rstd;
  void *dx;
  float *partial;  // [gridDim.x, 2, d]: sums of dy * n, then of dy
  int64_t T;
  int d;
  float inv_d;
};

// n = (r - mean) * rstd as (r / 2 - mean / 2) * 2 rstd: the difference comes first
// and is rounded once, so that rows whose mean is many times their spread keep
// the spread's digits (r rstd - mean rstd would be off by a step of mean rstd), and
// by halves no difference passes fp32's range.
struct LnN {
  float half_mean, twice_rstd;
  MOE_DEVICE LnN(float mean, float rstd) : half_mean(0.5f * mean), twice_rstd(2.0f * rstd) {}
  MOE_DEVICE float operator()(float r) const { return fmaf(r, 0.5f, -half_mean) * twice_rstd; }
};

// The workgroups share the rows out evenly; a thread keeps the same columns
// of every row and holds their two sums in registers, which become one pair of
// partial rows per workgroup.
template <typename T, int TPR, int NV, bool NT>
__global__ __launch_bounds__(kLnThreads) void layernorm_bwd_kernel(LnBwdParams p) {
  constexpr int V = Elem<T>::kVec;
  constexpr int RPB = kLnThreads / TPR;
  __shared__ LnPart part[2];
  __shared__ float comb[RPB > 1 ? RPB - 1 : 1][RPB > 1 ? TPR * NV * V : 1];
  const int lane = threadIdx.x % TPR, slot = threadIdx.x / TPR;
  const int n = p.d / V;
  float dw[NV][V], db[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) dw[j][i] = db[j][i] = 0.f;
  u32x4_t wv[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = j * TPR + lane;
    wv[j] = ld16((const T *)p.w + (c < n ? c : 0) * V);
  }
  // the next row's loads are in flight while this one is finished
  u32x4_t gn[NV], rn[NV], en[NV];
  float rstd_n = 0.f, mean_n = 0.f;
  const int64_t step = (int64_t)gridDim.x * RPB;
  auto fetch = [&](int64_t row) {
    const int64_t base = row * p.d;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = j * TPR + lane;
      const int64_t o = base + (c < n ? c : 0) * V;
      gn[j] = ln_ld<NT>((const T *)p.dy + o);
      rn[j] = ln_ld<NT>((const T *)p.r + o);
      if (p.dres) en[j] = ln_ld<NT>((const T *)p.dres + o);
    }
    rstd_n = p.rstd[row];
    mean_n = p.mean[row];
  };
  int turn = 0;
  const int64_t row0 = (int64_t)blockIdx.x * RPB + slot;
  if (row0 < p.T) fetch(row0);
  for (int64_t row = row0; row < p.T; row += step) {
    const int64_t base = row * p.d;
    u32x4_t gv[NV], rv[NV], ev[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      gv[j] = gn[j];
      rv[j] = rn[j];
      ev[j] = en[j];
    }
    const float rstd = rstd_n;
    const LnN norm(mean_n, rstd_n);
    if (row + step < p.T) fetch(row + step);
    float sg = 0.f, sn = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = j * TPR + lane;
      float g[V], r[V], w[V];
      Elem<T>::unpack(gv[j], g);
      Elem<T>::unpack(rv[j], r);
      Elem<T>::unpack(wv[j], w);
      float a = 0.f, b = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float gn = g[i] * norm(r[i]);
        if (c < n) {
          dw[j][i] += gn;
          db[j][i] += g[i];
        }
        a = fmaf(g[i], w[i], a);
        b = fmaf(gn, w[i], b);
      }
      if (c < n) {
        sg += a;
        sn += b;
      }
    }
    // the two buffers alternate: a wavefront writes one again only after the
    // barrier of the sum in between, when every wavefront has read it
    row_sums<TPR>(sg, sn, part[turn]);
    turn ^= 1;
    const float mg = sg * p.inv_d, mn = sn * p.inv_d;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = j * TPR + lane;
      if (c >= n) continue;
      float g[V], r[V], w[V];
      Elem<T>::unpack(gv[j], g);
      Elem<T>::unpack(rv[j], r);
      Elem<T>::unpack(wv[j], w);
#pragma unroll
      for (int i = 0; i < V; ++i) g[i] = rstd * fmaf(-norm(r[i]), mn, fmaf(g[i], w[i], -mg));
      if (p.dres) {
        float e[V];
        Elem<T>::unpack(ev[j], e);
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] += e[i];
      }
      ln_st<NT>((T *)p.dx + base + c * V, Elem<T>::pack(g));
    }
  }
  float *out = p.partial + (int64_t)blockIdx.x * 2 * p.d;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    float(&sum)[NV][V] = q == 0 ? dw : db;
    // the slots' sums, in the order of the slots
    if (RPB > 1) {
      if (q == 1) __syncthreads();
      if (slot > 0) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < V; ++i) comb[slot - 1][(j * V + i) * TPR + lane] = sum[j][i];
      }
      __syncthreads();
      if (slot > 0) continue;
#pragma unroll
      for (int s = 0; s < RPB - 1; ++s)
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < V; ++i) sum[j][i] += comb[s][(j * V + i) * TPR + lane];
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = j * TPR + lane;
      if (c >= n) continue;
#pragma unroll
      for (int i = 0; i < V; i += 4)
        *reinterpret_cast<f32x4_t *>(out + q * p.d + c * V + i) =
            f32x4_t{sum[j][i], sum[j][i + 1], sum[j][i + 2], sum[j][i + 3]};
    }
  }
}

// Rows too long for registers: two passes over the row, the column sums kept
// in the workgroup's partial rows, each by the one thread that owns it. dx is
// written in the second pass by the thread that read the same element, so it
// may overwrite dy or dres.
template <typename T>
__global__ __launch_bounds__(kLnThreads) void layernorm_bwd_long_kernel(LnBwdParams p) {
  constexpr int V = Elem<T>::kVec;
  __shared__ LnPart part[2];
  const int n = p.d / V;
  float *out = p.partial + (int64_t)blockIdx.x * 2 * p.d;
  bool first = true;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
    const int64_t base = row * p.d;
    const float rstd = p.rstd[row];
    const LnN norm(p.mean[row], rstd);
    float sg = 0.f, sn = 0.f;
    for (int c = threadIdx.x; c < n; c += kLnThreads) {
      float g[V], r[V], w[V];
      Elem<T>::unpack(ld16((const T *)p.dy + base + c * V), g);
      Elem<T>::unpack(ld16((const T *)p.r + base + c * V), r);
      Elem<T>::unpack(ld16((const T *)p.w + c * V), w);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float gn = g[i] * norm(r[i]);
        float *o = out + c * V + i;
        o[0] = first ? gn : o[0] + gn;
        o[p.d] = first ? g[i] : o[p.d] + g[i];
        sg = fmaf(g[i], w[i], sg);
        sn = fmaf(gn, w[i], sn);
      }
    }
    first = false;
    row_sums<kLnThreads>(sg, sn, part[turn]);
    turn ^= 1;
    const float mg = sg * p.inv_d, mn = sn * p.inv_d;
    for (int c = threadIdx.x; c < n; c += kLnThreads) {
      float g[V], r[V], w[V];
      Elem<T>::unpack(ld16((const T *)p.dy + base + c * V), g);
      Elem<T>::unpack(ld16((const T *)p.r + base + c * V), r);
      Elem<T>::unpack(ld16((const T *)p.w + c * V), w);
#pragma unroll
      for (int i = 0; i < V; ++i) g[i] = rstd * fmaf(-norm(r[i]), mn, fmaf(g[i], w[i], -mg));
      if (p.dres) {
        float e[V];
        Elem<T>::unpack(ld16((const T *)p.dres + base + c * V), e);
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] += e[i];
      }
      st16((T *)p.dx + base + c * V, Elem<T>::pack(g));
    }
  }
}

// dw and db (+)= the sums of the partial rows, in a fixed order: 64 threads
// take every 64th pair of partial rows of 4 columns, then their sums are added
// in turn. Columns [0, d) of a pair are dw's, [d, 2d) db's.
__global__ __launch_bounds__(256) void layernorm_dw_reduce_kernel(const float *partial, float *dw, float *db, int rows,
                                                                  int d, int accumulate) {
  __shared__ f32x4_t s[64][5];
  const int col = threadIdx.x & 3, grp = threadIdx.x >> 2;
  const int c = blockIdx.x * 16 + col * 4;  // d is a multiple of 64
  f32x4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int b = grp; b < rows; b += 64) {
    const f32x4_t q = *reinterpret_cast<const f32x4_t *>(partial + (int64_t)b * 2 * d + c);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += q[e];
  }
  s[grp][col] = v;
  __syncthreads();
  if (threadIdx.x >= 16) return;
  float sum = 0.f;
#pragma unroll
  for (int g = 0; g < 64; ++g) sum += s[g][threadIdx.x >> 2][threadIdx.x & 3];
  const int o = blockIdx.x * 16 + threadIdx.x;
  float *out = o < d ? dw + o : db + (o - d);
  *out = accumulate ? *out + sum : sum;
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
// A wavefront a row from kNormWaveRows rows on, where the row is at most `most`
// chunks a thread; a workgroup a row otherwise.
static bool wave_rows(int64_t T, int chunks, int most) { return T >= kNormWaveRows && chunks <= most * kWave; }

template <typename T, bool NT>
static void fwd_dispatch(const LnFwdParams &p, hipStream_t s) {
  const int n = p.d / Elem<T>::kVec;
  const dim3 b(kLnThreads);
  if (wave_rows(p.T, n, 4)) {
    const dim3 g((unsigned)ceil_div(p.T, kLnThreads / kWave));
    if (n <= kWave) layernorm_fwd_kernel<T, kWave, 1, NT><<<g, b, 0, s>>>(p);
    else if (n <= 2 * kWave) layernorm_fwd_kernel<T, kWave, 2, NT><<<g, b, 0, s>>>(p);
    else layernorm_fwd_kernel<T, kWave, 4, NT><<<g, b, 0, s>>>(p);
    return;
  }
  const dim3 g((unsigned)p.T);
  if (n <= kLnThreads) layernorm_fwd_kernel<T, kLnThreads, 1, NT><<<g, b, 0, s>>>(p);
  else if (n <= 2 * kLnThreads) layernorm_fwd_kernel<T, kLnThreads, 2, NT><<<g, b, 0, s>>>(p);
  else if (n <= 4 * kLnThreads) layernorm_fwd_kernel<T, kLnThreads, 4, NT><<<g, b, 0, s>>>(p);
  else layernorm_fwd_long_kernel<T><<<g, b, 0, s>>>(p);
}

template <typename T>
static void fwd_streams(const LnFwdParams &p, hipStream_t s) {
  const int64_t bytes = p.T * p.d * (int64_t)sizeof(T) * (p.residual ? 4 : 2);
  if (bytes > kLnCachedBytes) fwd_dispatch<T, true>(p, s);
  else fwd_dispatch<T, false>(p, s);
}

hipError_t launch_layernorm_fwd(const LayerNormArgs &a, hipStream_t s) {
  LaunchScope scope("layernorm_fwd", s);
  LnFwdParams p{};
  p.x = a.x;
  p.residual = a.residual;
  p.w = a.w;
  p.b = a.b;
  p.r = a.r;
  p.y = a.y;
  p.mean = a.mean;
  p.rstd = a.rstd;
  p.T = a.T;
  p.d = a.d;
  p.inv_d = 1.0f / (float)a.d;
  p.eps = a.eps;
  if (a.bf16) fwd_streams<bf16_t>(p, s);
  else fwd_streams<float>(p, s);
  return hipGetLastError();
}

template <typename T, bool NT>
static void bwd_dispatch(const LnBwdParams &p, int blocks, hipStream_t s) {
  const int n = p.d / Elem<T>::kVec;
  const dim3 g((unsigned)blocks), b(kLnThreads);
  // 1024 values of a row in a wavefront: 16 a lane, in either type (fp32 rows of
  // 513 to 1024 values in a workgroup: 32768 x 768 65.9 us against 53.8, 7001 x 576
  // 16.3 against 13.5, 32768 x 1024 72.2 against 68.8)
  constexpr int kMost = 16 / Elem<T>::kVec;
  if (wave_rows(p.T, n, kMost)) {
    if (n <= kWave) layernorm_bwd_kernel<T, kWave, 1, NT><<<g, b, 0, s>>>(p);
    else if (n <= 2 * kWave) layernorm_bwd_kernel<T, kWave, 2, NT><<<g, b, 0, s>>>(p);
    else layernorm_bwd_kernel<T, kWave, kMost, NT><<<g, b, 0, s>>>(p);
    return;
  }
  if (n <= kLnThreads) layernorm_bwd_kernel<T, kLnThreads, 1, NT><<<g, b, 0, s>>>(p);
  else if (n <= 2 * kLnThreads) layernorm_bwd_kernel<T, kLnThreads, 2, NT><<<g, b, 0, s>>>(p);
  else if (n <= 4 * kLnThreads) layernorm_bwd_kernel<T, kLnThreads, 4, NT><<<g, b, 0, s>>>(p);
  else layernorm_bwd_long_kernel<T><<<g, b, 0, s>>>(p);
}

template <typename T>
static void bwd_streams(const LnBwdParams &p, int blocks, hipStream_t s) {
  const int64_t bytes = p.T * p.d * (int64_t)sizeof(T) * (p.dres ? 4 : 3);
  if (bytes > kLnCachedBytes) bwd_dispatch<T, true>(p, blocks, s);
  else bwd_dispatch<T, false>(p, blocks, s);
}

hipError_t launch_layernorm_bwd(const LayerNormArgs &a, hipStream_t s) {
  const int blocks = norm_bwd_blocks(a.T);
  if (blocks > 0) {
    LaunchScope scope("layernorm_bwd", s);
    LnBwdParams p{};
    p.dy = a.dy;
    p.r = a.r;
    p.w = a.w;
    p.dres = a.dres;
    p.mean = a.mean;
    p.rstd = a.rstd;
    p.dx = a.dx;
    p.partial = a.partial;
    p.T = a.T;
    p.d = a.d;
    p.inv_d = 1.0f / (float)a.d;
    if (a.bf16) bwd_streams<bf16_t>(p, blocks, s);
    else bwd_streams<float>(p, blocks, s);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  LaunchScope scope("layernorm_dw_reduce", s);
  layernorm_dw_reduce_kernel<<<(a.db ? 2 : 1) * a.d / 16, 256, 0, s>>>(a.partial, a.dw, a.db, blocks, a.d,
                                                                       a.accumulate ? 1 : 0);
  return hipGetLastError();
}

}  // namespace moe
