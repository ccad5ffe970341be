// The dense product's weight gradient on the main loop of pingpong.h: 256 x 256
// tiles of dW = dz^T x, both operands k-major (a stage is 64 tokens), the tokens
// split into slices (linear_wgrad_plan), and in the same pass db, the sums of
// dz's columns: a wavefront adds up the one row block of its A fragments that no
// other of its tile row's wavefronts does (16 dot products with ones a stage,
// beside 64 MFMAs).
#pragma once

#include "gemm_common.h"
#include "pingpong.h"

namespace moe {

struct LinearDwParams {
  const bf16_t *dz, *x;  // [T, N], [T, K]
  float *dw, *db;        // dw: of a slice, db: [slices, N] or NULL
  int T, K, N, chunk, slices;
  int n_tiles, k_tiles;
};

// ADD (one slice): dw and db are added to.
template <bool ADD>
__global__ __launch_bounds__(kPpThreads, 2) void linear_dw_kernel(LinearDwParams p) {
  __shared__ u32x4_t lds[kPpLdsBytes / 16];
  const int tiles = p.n_tiles * p.k_tiles;
  int lo, hi;
  xcd_range(blockIdx.x & 7, (int64_t)tiles * p.slices, lo, hi);
  const int step = gridDim.x >> 3;
  const int first = lo + (int)(blockIdx.x >> 3);
  if (first >= hi) return;
  struct Place {
    int slice, n0, k0;
  };
  auto place = [&](int id) {
    const int slice = __builtin_amdgcn_readfirstlane(id / tiles);
    const int r = id - slice * tiles;
    const int nt = __builtin_amdgcn_readfirstlane(r / p.k_tiles);
    return Place{slice, nt * kPpTile, (r - nt * p.k_tiles) * kPpTile};
  };
  int load = first, put = first;
  auto get = [&]() {
    const Place at = place(load);
    const int64_t row0 = (int64_t)at.slice * p.chunk;
    load += step;
    PpTile t;
    t.A = p.dz + row0 * p.N + at.n0;
    t.B = p.x + row0 * p.K + at.k0;
    t.m_valid = min(kPpTile, p.N - at.n0);
    t.n_valid = min(kPpTile, p.K - at.k0);
    t.k_valid = min(p.chunk, p.T - (int)row0);
    return t;
  };
  float sum[2] = {0.f, 0.f};  // of the lane's row of block 0 of either half
  auto stage = [&](const bf16x8_t (&a0)[2], const bf16x8_t (&a1)[2]) {
    typedef __bf16 pair_t __attribute__((ext_vector_type(2)));
    const pair_t one = {(__bf16)1.f, (__bf16)1.f};
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const u32x4_t v0 = __builtin_bit_cast(u32x4_t, a0[ks]), v1 = __builtin_bit_cast(u32x4_t, a1[ks]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t u0 = v0[e], u1 = v1[e];
        sum[0] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(pair_t, u0), one, sum[0], false);
        sum[1] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(pair_t, u1), one, sum[1], false);
      }
    }
  };
  auto done = [&](PpAcc &acc) {
    const Place at = place(put);
    put += step;
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));  // no address below is formed above the main loop
    const int l16 = lane & 15, l4 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wn = wave & 3;
    const int n0 = at.n0 + (wave >> 2) * 128, k0 = at.k0 + wn * 64;
    if (p.db && at.k0 == 0) {
      float *db = p.db + (int64_t)at.slice * p.N;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v = sum[h];
        v += __shfl_xor(v, 16);
        v += __shfl_xor(v, 32);
        const int n = n0 + h * 64 + wn * 16 + l16;
        if (l4 == 0 && n < p.N) db[n] = ADD ? db[n] + v : v;
      }
    }
    sum[0] = sum[1] = 0.f;
    const int rows = min(128, p.N - n0);
    if (rows <= 0 || k0 >= p.K) return;  // 64 rows and columns exist or none
    const uint32_t pitch = (uint32_t)p.K * 4u;
    const TileRows dw(p.dw + ((int64_t)at.slice * p.N + n0) * p.K + k0, pitch, rows);
    const uint32_t off0 = (uint32_t)l16 * pitch + (uint32_t)l4 * 16u;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t off = off0 + (uint32_t)(h * 64 + (i ^ wn) * 16) * pitch;
        u32x4_t old[4];
        if constexpr (ADD) {
#pragma unroll
          for (int j = 0; j < 4; ++j) old[j] = dw.load(off + j * 64);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f32x4_t v = acc[h * 4 + i][j];
          if constexpr (ADD) v += __builtin_bit_cast(f32x4_t, old[j]);
          dw.store(off + j * 64, __builtin_bit_cast(u32x4_t, v));
        }
      }
  };
  pp_tiles<false, true, true>(lds, p.N, p.K, p.chunk / 64, (hi - first + step - 1) / step, get, done, stage);
}

// The sums of the slices, in order, and the gradient already there added to their
// sum (one rounding at its size, however many slices): chunks of 16 bytes of dw,
// then of db.
struct LinearDwReduce {
  const float *dw_part, *db_part;
  float *dw, *db;
  int64_t dw4, db4;  // chunks; db4 0: no db
  int slices, accumulate;
};

__global__ __launch_bounds__(256) void linear_dw_reduce_kernel(LinearDwReduce p) {
  int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const bool bias = i >= p.dw4;
  if (bias) i -= p.dw4;
  const int64_t n = bias ? p.db4 : p.dw4;
  if (i >= n) return;
  const f32x4_t *src = reinterpret_cast<const f32x4_t *>(bias ? p.db_part : p.dw_part) + i;
  f32x4_t *dst = reinterpret_cast<f32x4_t *>(bias ? p.db : p.dw) + i;
  f32x4_t old = {0.f, 0.f, 0.f, 0.f}, v = old;
  if (p.accumulate) old = *dst;
#pragma unroll 4
  for (int s = 0; s < p.slices; ++s) {
    const f32x4_t q = src[s * n];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += q[e];
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] += old[e];
  *dst = v;
}

}  // namespace moe
