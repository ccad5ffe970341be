// RMS norm with the residual's addition, its backward pass, and the 8-bit
// block form of a matrix. All of it is bound by HBM: every kernel reads each
// input once and writes each output once, a row held in registers between
// the reduction over the row and its scaling.
//
//   forward   r = round(x + residual);  rstd = 1 / sqrt(mean(r^2) + eps);  y = r * rstd * w
//   backward  n = r * rstd, g = dy * w:  dx = rstd * (g - n * mean(g * n)) + dres
//             dw = sum over the rows of dy * n
// The norm reads the rounded r, the tensor that the backward pass and the
// next layer see, so that the gradient is the gradient of what was computed.
//
// Measured (a 1 GiB copy reaches 6.7 TB/s here): forward with residual, 32768
// x 2048 bf16, 87 us, 6.1 TB/s; backward 32768 x 4096 bf16 180 us, 6.0 TB/s;
// 5632 x 4096 bf16 to 8 bits 11.7 us, 6.0 TB/s; one row of 2048 2.1 us, the
// length of an all but empty kernel.
#include "common.h"
#include "kernels.h"
#include "mx8.h"

namespace moe {

constexpr int kNormThreads = 256;

// Streams of more than half the 256 MB memory-side cache pass it by (NT):
// 32768 x 2048 bf16 forward 87 us (93 through the cache), 32768 x 4096 backward
// 180 (200), 32768 x 2048 backward 88 (97); 16384 x 2048 to 8 bits, just above
// the border, 39.4 (38.7). Smaller ones stay in it for whoever reads them next,
// and are faster so (7001 x 1024 fp32 forward 10.5 against 12.2 us).
constexpr int64_t kNormCachedBytes = (int64_t)128 << 20;
template <bool NT>
MOE_DEVICE u32x4_t ld16s(const void *p) {
  return NT ? ld16_nt(p) : ld16(p);
}
template <bool NT>
MOE_DEVICE void st16s(void *p, const u32x4_t &v) {
  if (NT) st16_nt(p, v);
  else st16(p, v);
}

// Sum over the TPR threads of a row, the same bits in every thread. TPR = 64
// is one wavefront; 256 is the workgroup, through `part` (4 floats), which
// must not be in use by an earlier sum.
template <int TPR>
MOE_DEVICE float row_sum(float v, float *part) {
  v = wave_sum_dpp(v);
  if (TPR == kWave) return v;
  if ((threadIdx.x & (kWave - 1)) == 0) part[threadIdx.x / kWave] = v;
  __syncthreads();
  return (part[0] + part[1]) + (part[2] + part[3]);
}

// The squares of a row pass fp32's range from |r| of about 2^60 on, though rstd
// does not: such a row, whose sum is infinite, is summed again over r 2^-80.
// That sum stays below 2^112 (65536 values below 2^128), and the largest value
// of a row that needs it is at least 2^56, so that nothing that counts gets
// lost below. An infinity in the row leaves the sum infinite and rstd zero.
constexpr float kNormDown = 0x1p-80f;
MOE_DEVICE bool norm_again(float sum) { return sum == __builtin_huge_valf(); }
MOE_DEVICE float norm_rstd(float sum, float inv_d, float eps) { return 1.0f / sqrtf(fmaf(sum, inv_d, eps)); }
MOE_DEVICE float norm_rstd_down(float sum, float inv_d, float eps) {
  return kNormDown / sqrtf(fmaf(sum, inv_d, eps * kNormDown * kNormDown));
}

// One 16-byte chunk's worth of values to the 8-bit form. The 32 values of a
// block lie in 32 / kVec consecutive lanes, all of them active.
template <typename T>
MOE_DEVICE void store_mx8(const float *v, uint8_t *q, uint8_t *scale, int64_t row, int d, int chunk, bool valid) {
  constexpr int V = Elem<T>::kVec;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) m = umax(m, abs_bits(v[i]));
  m = group_umax<kMx8Block / V>(m);
  const uint32_t code = mx8_scale_code(m);
  const float inv = mx8_inv_scale(code);
  uint32_t w[V / 4];
#pragma unroll
  for (int i = 0; i < V / 4; ++i)
    w[i] = mx8_pack4(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
  if (!valid) return;
  uint8_t *p = q + row * d + (int64_t)chunk * V;
  if constexpr (V == 8) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
  } else {
    *reinterpret_cast<uint32_t *>(p) = w[0];
  }
  if (chunk % (kMx8Block / V) == 0) scale[row * (d / kMx8Block) + chunk / (kMx8Block / V)] = (uint8_t)code;
}

struct NormFwdParams {
  const void *x, *residual, *w;
  void *r, *y;
  uint8_t *y_scale;
  float *rstd;
  int64_t T;
  int d;
  float inv_d, eps;
};

// A row in TPR threads, NV chunks of 16 bytes each.
template <typename T, int TPR, int NV, bool MX8, bool NT>
__global__ __launch_bounds__(kNormThreads) void rmsnorm_fwd_kernel(NormFwdParams p) {
  constexpr int V = Elem<T>::kVec;
  __shared__ float part[2][kNormThreads / kWave];
  const int lane = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * (kNormThreads / TPR) + threadIdx.x / TPR;
  if (row >= p.T) return;  // whole wavefronts only, and no barrier below for TPR = 64
  const int n = p.d / V;
  const T *x = (const T *)p.x + row * p.d;
  const T *res = p.residual ? (const T *)p.residual + row * p.d : nullptr;
  u32x4_t xv[NV], rv[NV], wv[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = j * TPR + lane;
    const int cc = c < n ? c : 0;
    xv[j] = ld16s<NT>(x + cc * V);
    if (res) rv[j] = ld16s<NT>(res + cc * V);
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = j * TPR + lane;
    wv[j] = ld16((const T *)p.w + (c < n ? c : 0) * V);
  }
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = j * TPR + lane;
    if (res) {
      float a[V], b[V];
      Elem<T>::unpack(xv[j], a);
      Elem<T>::unpack(rv[j], b);
#pragma unroll
      for (int i = 0; i < V; ++i) a[i] += b[i];
      xv[j] = Elem<T>::pack(a);  // rounded once: from here on r is what the row holds
      if (c < n) st16s<NT>((T *)p.r + row * p.d + c * V, xv[j]);
    }
    float a[V];
    Elem<T>::unpack(xv[j], a);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) s = fmaf(a[i], a[i], s);
    if (c < n) sum += s;
  }
  sum = row_sum<TPR>(sum, part[0]);
  float rstd = norm_rstd(sum, p.inv_d, p.eps);
  if (norm_again(sum)) {  // all threads of the row alike
    float down = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float a[V];
      Elem<T>::unpack(xv[j], a);
      if (j * TPR + lane >= n) continue;
#pragma unroll
      for (int i = 0; i < V; ++i) down = fmaf(a[i] * kNormDown, a[i] * kNormDown, down);
    }
    rstd = norm_rstd_down(row_sum<TPR>(down, part[1]), p.inv_d, p.eps);
  }
  if (lane == 0) p.rstd[row] = rstd;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = j * TPR + lane;
    float a[V], w[V];
    Elem<T>::unpack(xv[j], a);
    Elem<T>::unpack(wv[j], w);
#pragma unroll
    for (int i = 0; i < V; ++i) a[i] = a[i] * rstd * w[i];
    if (MX8) {
      store_mx8<T>(a, (uint8_t *)p.y, p.y_scale, row, p.d, c, c < n);
    } else if (c < n) {
      st16s<NT>((T *)p.y + row * p.d + c * V, Elem<T>::pack(a));
    }
  }
}

// Rows too long for registers: a workgroup per row reads the row twice (the
// second time from the caches). Every element is read and written by one
// thread, which reads its r back rather than x, so r may overwrite x.
template <typename T, bool MX8>
__global__ __launch_bounds__(kNormThreads) void rmsnorm_fwd_long_kernel(NormFwdParams p) {
  constexpr int V = Elem<T>::kVec;
  __shared__ float part[2][kNormThreads / kWave];
  const int64_t row = blockIdx.x;
  const int n = p.d / V;
  const T *x = (const T *)p.x + row * p.d;
  float sum = 0.f;
  for (int c = threadIdx.x; c < n; c += kNormThreads) {
    u32x4_t v = ld16(x + c * V);
    float a[V];
    Elem<T>::unpack(v, a);
    if (p.residual) {
      float b[V];
      Elem<T>::unpack(ld16((const T *)p.residual + row * p.d + c * V), b);
#pragma unroll
      for (int i = 0; i < V; ++i) a[i] += b[i];
      v = Elem<T>::pack(a);
      st16((T *)p.r + row * p.d + c * V, v);
      Elem<T>::unpack(v, a);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) sum = fmaf(a[i], a[i], sum);
  }
  sum = row_sum<kNormThreads>(sum, part[0]);
  const T *src = p.residual ? (const T *)p.r + row * p.d : x;
  float rstd = norm_rstd(sum, p.inv_d, p.eps);
  if (norm_again(sum)) {
    float down = 0.f;
    for (int c = threadIdx.x; c < n; c += kNormThreads) {
      float a[V];
      Elem<T>::unpack(ld16(src + c * V), a);
#pragma unroll
      for (int i = 0; i < V; ++i) down = fmaf(a[i] * kNormDown, a[i] * kNormDown, down);
    }
    rstd = norm_rstd_down(row_sum<kNormThreads>(down, part[1]), p.inv_d, p.eps);
  }
  if (threadIdx.x == 0) p.rstd[row] = rstd;
  for (int c0 = 0; c0 < n; c0 += kNormThreads) {  // every lane takes every pass: blocks span lanes
    const int c = c0 + threadIdx.x;
    const int cc = c < n ? c : 0;
    float a[V], w[V];
    Elem<T>::unpack(ld16(src + cc * V), a);
    Elem<T>::unpack(ld16((const T *)p.w + cc * V), w);
#pragma unroll
    for (int i = 0; i < V; ++i) a[i] = a[i] * rstd * w[i];
    if (MX8) {
      store_mx8<T>(a, (uint8_t *)p.y, p.y_scale, row, p.d, c, c < n);
    } else if (c < n) {
      st16((T *)p.y + row * p.d + c * V, Elem<T>::pack(a));
    }
  }
}

// The 8-bit form of [rows, d]: chunks over the whole matrix (a row is a
// whole number of blocks).
template <typename T>
__global__ __launch_bounds__(kNormThreads) void mx8_quantize_kernel(const T *x, uint8_t *q, uint8_t *scale,
                                                                    int64_t chunks) {
  constexpr int V = Elem<T>::kVec;
  constexpr int LPB = kMx8Block / V;  // lanes per block
  const int64_t c = (int64_t)blockIdx.x * kNormThreads + threadIdx.x;
  const int64_t cc = c < chunks ? c : chunks - 1;
  float v[V];
  Elem<T>::unpack(ld16(x + cc * V), v);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) m = umax(m, abs_bits(v[i]));
  m = group_umax<LPB>(m);
  const uint32_t code = mx8_scale_code(m);
  const float inv = mx8_inv_scale(code);
  if (c >= chunks) return;
#pragma unroll
  for (int i = 0; i < V / 4; ++i)
    *reinterpret_cast<uint32_t *>(q + c * V + 4 * i) =
        mx8_pack4(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
  if (c % LPB == 0) scale[c / LPB] = (uint8_t)code;
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
struct NormBwdParams {
  const void *dy, *r, *w, *dres;
  const float *rstd;
  void *dx;
  float *partial;  // [gridDim.x, d]
  int64_t T;
  int d;
  float inv_d;
};

// The workgroups share the rows out evenly; a thread keeps the same columns
// of every row and holds their sums of dy * n in registers, which become one
// partial row per workgroup.
template <typename T, int TPR, int NV, bool NT>
__global__ __launch_bounds__(kNormThreads) void rmsnorm_bwd_kernel(NormBwdParams p) {
  constexpr int V = Elem<T>::kVec;
  constexpr int RPB = kNormThreads / TPR;
  __shared__ float part[2][kNormThreads / kWave];
  __shared__ float comb[RPB > 1 ? RPB - 1 : 1][RPB > 1 ? TPR * NV * V : 1];
  const int lane = threadIdx.x % TPR, slot = threadIdx.x / TPR;
  const int n = p.d / V;
  float dw[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) dw[j][i] = 0.f;
  u32x4_t wv[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = j * TPR + lane;
    wv[j] = ld16((const T *)p.w + (c < n ? c : 0) * V);
  }
  // the next row's loads are in flight while this one is finished
  u32x4_t gn[NV], rn[NV], en[NV];
  float rstd_n = 0.f;
  const int64_t step = (int64_t)gridDim.x * RPB;
  auto fetch = [&](int64_t row) {
    const int64_t base = row * p.d;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = j * TPR + lane;
      const int64_t o = base + (c < n ? c : 0) * V;
      gn[j] = ld16s<NT>((const T *)p.dy + o);
      rn[j] = ld16s<NT>((const T *)p.r + o);
      if (p.dres) en[j] = ld16s<NT>((const T *)p.dres + o);
    }
    rstd_n = p.rstd[row];
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
    if (row + step < p.T) fetch(row + step);
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = j * TPR + lane;
      float g[V], r[V], w[V];
      Elem<T>::unpack(gv[j], g);
      Elem<T>::unpack(rv[j], r);
      Elem<T>::unpack(wv[j], w);
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float gn = g[i] * (r[i] * rstd);
        if (c < n) dw[j][i] += gn;
        s = fmaf(gn, w[i], s);
      }
      if (c < n) dot += s;
    }
    // the two buffers alternate: a wavefront writes one again only after the
    // barrier of the sum in between, when every wavefront has read it
    dot = row_sum<TPR>(dot, part[turn]);
    turn ^= 1;
    const float mean = dot * p.inv_d;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = j * TPR + lane;
      if (c >= n) continue;
      float g[V], r[V], w[V];
      Elem<T>::unpack(gv[j], g);
      Elem<T>::unpack(rv[j], r);
      Elem<T>::unpack(wv[j], w);
#pragma unroll
      for (int i = 0; i < V; ++i) g[i] = rstd * fmaf(-(r[i] * rstd), mean, g[i] * w[i]);
      if (p.dres) {
        float e[V];
        Elem<T>::unpack(ev[j], e);
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] += e[i];
      }
      st16s<NT>((T *)p.dx + base + c * V, Elem<T>::pack(g));
    }
  }
  // the slots' sums, in the order of the slots
  if (RPB > 1) {
    if (slot > 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) comb[slot - 1][(j * V + i) * TPR + lane] = dw[j][i];
    }
    __syncthreads();
    if (slot > 0) return;
#pragma unroll
    for (int s = 0; s < RPB - 1; ++s)
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) dw[j][i] += comb[s][(j * V + i) * TPR + lane];
  }
  float *out = p.partial + (int64_t)blockIdx.x * p.d;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = j * TPR + lane;
    if (c >= n) continue;
#pragma unroll
    for (int i = 0; i < V; i += 4)
      *reinterpret_cast<f32x4_t *>(out + c * V + i) = f32x4_t{dw[j][i], dw[j][i + 1], dw[j][i + 2], dw[j][i + 3]};
  }
}

// Rows too long for registers: two passes over the row, the column sums kept
// in the workgroup's partial row, each by the one thread that owns it. dx is
// written in the second pass by the thread that read the same element, so it
// may overwrite dy or dres.
template <typename T>
__global__ __launch_bounds__(kNormThreads) void rmsnorm_bwd_long_kernel(NormBwdParams p) {
  constexpr int V = Elem<T>::kVec;
  __shared__ float part[2][kNormThreads / kWave];
  const int n = p.d / V;
  float *out = p.partial + (int64_t)blockIdx.x * p.d;
  bool first = true;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
    const int64_t base = row * p.d;
    const float rstd = p.rstd[row];
    float dot = 0.f;
    for (int c = threadIdx.x; c < n; c += kNormThreads) {
      float g[V], r[V], w[V];
      Elem<T>::unpack(ld16((const T *)p.dy + base + c * V), g);
      Elem<T>::unpack(ld16((const T *)p.r + base + c * V), r);
      Elem<T>::unpack(ld16((const T *)p.w + c * V), w);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float gn = g[i] * (r[i] * rstd);
        out[c * V + i] = first ? gn : out[c * V + i] + gn;
        dot = fmaf(gn, w[i], dot);
      }
    }
    first = false;
    dot = row_sum<kNormThreads>(dot, part[turn]);
    turn ^= 1;
    const float mean = dot * p.inv_d;
    for (int c = threadIdx.x; c < n; c += kNormThreads) {
      float g[V], r[V], w[V];
      Elem<T>::unpack(ld16((const T *)p.dy + base + c * V), g);
      Elem<T>::unpack(ld16((const T *)p.r + base + c * V), r);
      Elem<T>::unpack(ld16((const T *)p.w + c * V), w);
#pragma unroll
      for (int i = 0; i < V; ++i) g[i] = rstd * fmaf(-(r[i] * rstd), mean, g[i] * w[i]);
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

// dw (+)= the sum of the partial rows, in a fixed order: 64 threads take every
// 64th partial row of 4 columns, then their sums are added in turn.
__global__ __launch_bounds__(256) void rmsnorm_dw_reduce_kernel(const float *partial, float *dw, int rows, int d,
                                                                int accumulate) {
  __shared__ f32x4_t s[64][5];
  const int col = threadIdx.x & 3, grp = threadIdx.x >> 2;
  const int c = blockIdx.x * 16 + col * 4;  // d is a multiple of 64
  f32x4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int b = grp; b < rows; b += 64) {
    const f32x4_t q = *reinterpret_cast<const f32x4_t *>(partial + (int64_t)b * d + c);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += q[e];
  }
  s[grp][col] = v;
  __syncthreads();
  if (threadIdx.x >= 16) return;
  float sum = 0.f;
#pragma unroll
  for (int g = 0; g < 64; ++g) sum += s[g][threadIdx.x >> 2][threadIdx.x & 3];
  float *out = dw + blockIdx.x * 16 + threadIdx.x;
  *out = accumulate ? *out + sum : sum;
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
// Threads of a row: with few rows, as many as fill the row once (latency);
// otherwise one wavefront, which needs no barrier, up to 4 chunks a thread
// (32768 x 4096 bf16 forward 187 us with 8, 176 with a workgroup a row), in the
// backward pass, where a thread also holds column sums and the next row, up
// to 2 (217 against 212 us there).
static bool wave_rows(int64_t T, int chunks, int most) { return T >= kNormWaveRows && chunks <= most * kWave; }

template <typename T, bool MX8, bool NT>
static void fwd_dispatch(const NormFwdParams &p, hipStream_t s) {
  const int n = p.d / Elem<T>::kVec;
  if (wave_rows(p.T, n, 4)) {
    const dim3 g((unsigned)ceil_div(p.T, kNormThreads / kWave)), b(kNormThreads);
    if (n <= kWave) rmsnorm_fwd_kernel<T, kWave, 1, MX8, NT><<<g, b, 0, s>>>(p);
    else if (n <= 2 * kWave) rmsnorm_fwd_kernel<T, kWave, 2, MX8, NT><<<g, b, 0, s>>>(p);
    else rmsnorm_fwd_kernel<T, kWave, 4, MX8, NT><<<g, b, 0, s>>>(p);
    return;
  }
  const dim3 g((unsigned)p.T), b(kNormThreads);
  if (n <= kNormThreads) rmsnorm_fwd_kernel<T, kNormThreads, 1, MX8, NT><<<g, b, 0, s>>>(p);
  else if (n <= 2 * kNormThreads) rmsnorm_fwd_kernel<T, kNormThreads, 2, MX8, NT><<<g, b, 0, s>>>(p);
  else if (n <= 4 * kNormThreads) rmsnorm_fwd_kernel<T, kNormThreads, 4, MX8, NT><<<g, b, 0, s>>>(p);
  else rmsnorm_fwd_long_kernel<T, MX8><<<g, b, 0, s>>>(p);
}

template <typename T, bool MX8>
static void fwd_streams(const NormFwdParams &p, hipStream_t s) {
  const int64_t bytes = p.T * p.d * ((int64_t)sizeof(T) * (p.residual ? 3 : 1) + (MX8 ? 1 : sizeof(T)));
  if (bytes > kNormCachedBytes) fwd_dispatch<T, MX8, true>(p, s);
  else fwd_dispatch<T, MX8, false>(p, s);
}

hipError_t launch_rmsnorm_fwd(const RmsNormArgs &a, hipStream_t s) {
  LaunchScope scope("rmsnorm_fwd", s);
  NormFwdParams p{};
  p.x = a.x;
  p.residual = a.residual;
  p.w = a.w;
  p.r = a.r;
  p.y = a.y;
  p.y_scale = (uint8_t *)a.y_scale;
  p.rstd = a.rstd;
  p.T = a.T;
  p.d = a.d;
  p.inv_d = 1.0f / (float)a.d;
  p.eps = a.eps;
  if (a.bf16) {
    if (a.y_scale) fwd_streams<bf16_t, true>(p, s);
    else fwd_streams<bf16_t, false>(p, s);
  } else {
    if (a.y_scale) fwd_streams<float, true>(p, s);
    else fwd_streams<float, false>(p, s);
  }
  return hipGetLastError();
}

template <typename T, bool NT>
static void bwd_dispatch(const NormBwdParams &p, int blocks, hipStream_t s) {
  const int n = p.d / Elem<T>::kVec;
  const dim3 g((unsigned)blocks), b(kNormThreads);
  if (wave_rows(p.T, n, 2)) {
    if (n <= kWave) rmsnorm_bwd_kernel<T, kWave, 1, NT><<<g, b, 0, s>>>(p);
    else rmsnorm_bwd_kernel<T, kWave, 2, NT><<<g, b, 0, s>>>(p);
    return;
  }
  if (n <= kNormThreads) rmsnorm_bwd_kernel<T, kNormThreads, 1, NT><<<g, b, 0, s>>>(p);
  else if (n <= 2 * kNormThreads) rmsnorm_bwd_kernel<T, kNormThreads, 2, NT><<<g, b, 0, s>>>(p);
  else if (n <= 4 * kNormThreads) rmsnorm_bwd_kernel<T, kNormThreads, 4, NT><<<g, b, 0, s>>>(p);
  else rmsnorm_bwd_long_kernel<T><<<g, b, 0, s>>>(p);
}

template <typename T>
static void bwd_streams(const NormBwdParams &p, int blocks, hipStream_t s) {
  const int64_t bytes = p.T * p.d * (int64_t)sizeof(T) * (p.dres ? 4 : 3);
  if (bytes > kNormCachedBytes) bwd_dispatch<T, true>(p, blocks, s);
  else bwd_dispatch<T, false>(p, blocks, s);
}

hipError_t launch_rmsnorm_bwd(const RmsNormArgs &a, hipStream_t s) {
  const int blocks = norm_bwd_blocks(a.T);
  if (blocks > 0) {
    LaunchScope scope("rmsnorm_bwd", s);
    NormBwdParams p{};
    p.dy = a.dy;
    p.r = a.r;
    p.w = a.w;
    p.dres = a.dres;
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
  LaunchScope scope("rmsnorm_dw_reduce", s);
  rmsnorm_dw_reduce_kernel<<<a.d / 16, 256, 0, s>>>(a.partial, a.dw, blocks, a.d, a.accumulate ? 1 : 0);
  return hipGetLastError();
}

hipError_t launch_mx8_quantize(const void *x, void *q, void *scale, int64_t rows, int d, bool bf16, hipStream_t s) {
  LaunchScope scope("mx8_quantize", s);
  const int64_t chunks = rows * (d / (bf16 ? 8 : 4));
  const dim3 g((unsigned)ceil_div(chunks, kNormThreads)), b(kNormThreads);
  if (bf16) mx8_quantize_kernel<bf16_t><<<g, b, 0, s>>>((const bf16_t *)x, (uint8_t *)q, (uint8_t *)scale, chunks);
  else mx8_quantize_kernel<float><<<g, b, 0, s>>>((const float *)x, (uint8_t *)q, (uint8_t *)scale, chunks);
  return hipGetLastError();
}

}  // namespace moe
