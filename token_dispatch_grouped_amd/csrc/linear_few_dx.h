// The dense product's input gradient where few workgroups have work (few tokens,
// or few columns), dx = (dz W) act'(z) + add: bound by what a CU draws, the weights
// and the tokens' gradients, and by a kernel's start and end.
//
// The sum runs over W's rows, so a workgroup owns CB columns (64 or 32: 128 or 64
// bytes of every row) and 16 MF tokens, and each of its 8 wavefronts takes a run of
// steps of 32 rows through an LDS ring of its own, filled by the LDS DMA: no barrier
// until the partial sums meet, added in the order of the wavefronts. The
// fragments of W come out of transposing reads. The tiles, of 64 x 128 at least,
// make 16 workgroups of 2048 columns, each of which takes the stages of a sum over
// 8192 rows one after the other: 47 us at one token where 64 workgroups of 8
// wavefronts take 12.6 (a copy of the weights' bytes: 5.0); 2048 x 2048 12.0 and 3.8.
#pragma once

#include "act.h"
#include "ffn_kernel.h"

namespace moe {

template <int CB, int MF>
__global__ __launch_bounds__(512, 2) void linear_few_dx_kernel(FfnTileParams p) {
  constexpr int WAVES = 8, ROWS = 32;        // of W in a step
  constexpr int CF = CB / 16, CPR = CB / 8;  // column fragments, 16-byte chunks of a row
  constexpr int ROWB = CB * 2;
  constexpr int W_BYTES = ROWS * ROWB, STEP_BYTES = W_BYTES + MF * 1024;
  constexpr int NW = W_BYTES / 1024, PER = NW + MF;  // DMA instructions of a step
  constexpr int SLOTS = 20 * 1024 / STEP_BYTES < 4 ? 20 * 1024 / STEP_BYTES : 4;
  constexpr int WAVE_BYTES = SLOTS * STEP_BYTES;
  static_assert(SLOTS >= 2 && WAVES * WAVE_BYTES <= 160 * 1024, "LDS budget of one workgroup");
  static_assert(CF * MF * 1024 <= WAVE_BYTES, "the partial sums meet in the rings");
  __shared__ u32x4_t lds[WAVES * WAVE_BYTES / 16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i16 = lane & 15, g = lane >> 4;
  const int t0 = blockIdx.y * 16 * MF;
  // neighbouring half lines on one XCD, whose L2 then reads the line once
  int block = blockIdx.x;
  if (CB == 32 && gridDim.x % 16 == 0) block = ((block >> 4) * 8 + (block & 7)) * 2 + ((block >> 3) & 1);
  const int k0 = block * CB;

  // chunk c of row r of W at c ^ swz_w(r), the same for rows r and r + 4, which one
  // transposing read pairs; of a token's 64 bytes at c ^ (r / 4) % 4
  auto swz_w = [](int r) { return CB == 64 ? 2 * ((r >> 1) & 1) ^ 4 * ((r >> 3) & 1) : 2 * ((r >> 3) & 1); };
  const bf16_t *src[PER];
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    const int r = (i * 64 + lane) / CPR, c = lane % CPR ^ swz_w(r);
    src[i] = p.B + (int64_t)r * p.ldb + k0 + c * 8;
  }
#pragma unroll
  for (int m = 0; m < MF; ++m) {  // tokens past the last one feed dropped results
    const int r = lane >> 2, c = (lane & 3) ^ ((r >> 2) & 3);
    src[NW + m] = p.A + (int64_t)min(t0 + m * 16 + r, p.M - 1) * p.lda + c * 8;
  }
  const char *ring = reinterpret_cast<const char *>(lds) + wave * WAVE_BYTES;
  const uint32_t ring0 = (uint32_t)(uintptr_t)ring;

  const int n = p.K / ROWS;
  const int cnt = (n + WAVES - 1) / WAVES;
  const int first = min(wave * cnt, n);
  const int steps = min(cnt, n - first);
  auto issue = [&](int s) {
    const uint32_t dst = ring0 + (uint32_t)(s % SLOTS * STEP_BYTES);
    const int64_t row = (int64_t)(first + s) * ROWS;
#pragma unroll
    for (int i = 0; i < PER; ++i) dma16(src[i] + (i < NW ? row * p.ldb : row), dst + (uint32_t)(i * 1024));
  };
  auto wait_steps = [&](int younger) {  // until at most `younger` steps are in flight
    if (SLOTS > 3 && younger >= 3) wait_vm<3 * PER>();
    else if (SLOTS > 2 && younger >= 2) wait_vm<2 * PER>();
    else if (younger >= 1) wait_vm<PER>();
    else wait_vm<0>();
  };
  f32x4_t acc[CF][MF];
#pragma unroll
  for (int c = 0; c < CF; ++c)
#pragma unroll
    for (int m = 0; m < MF; ++m) acc[c][m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  // a fragment: 8 consecutive rows from 8 g on of column 16 c + i16
  const int k_lo = 8 * g + (i16 >> 2);
  uint32_t wat[CF];
#pragma unroll
  for (int c = 0; c < CF; ++c) {
    const int col = c * 16 + 4 * (i16 & 3);
    wat[c] = (uint32_t)(k_lo * ROWB + ((col >> 3) ^ swz_w(k_lo)) * 16 + ((col >> 2) & 1) * 8);
  }
  const uint32_t xat = (uint32_t)(W_BYTES + i16 * 64 + (g ^ ((i16 >> 2) & 3)) * 16);
#pragma unroll
  for (int s = 0; s < SLOTS; ++s)
    if (s < steps) issue(s);
  for (int s = 0; s < steps; ++s) {
    wait_steps(min(SLOTS, steps - s) - 1);
    const char *t = ring + s % SLOTS * STEP_BYTES;
    u32x4_t f[CF + MF];
#pragma unroll
    for (int c = 0; c < CF; ++c) {
      typedef __attribute__((__vector_size__(8 * sizeof(short)))) short i16x8_t;
      const i16x4_t lo = lds_read_tr16(t + wat[c]), hi = lds_read_tr16(t + wat[c] + 4 * ROWB);
      const i16x8_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      f[c] = __builtin_bit_cast(u32x4_t, v);
    }
#pragma unroll
    for (int m = 0; m < MF; ++m) f[CF + m] = *reinterpret_cast<const u32x4_t *>(t + xat + m * 1024);
    wait_lds();  // the slot's bytes are in registers
#pragma unroll
    for (int i = 0; i < CF + MF; ++i) asm volatile("" : "+v"(f[i]));
    if (s + SLOTS < steps) issue(s + SLOTS);
#pragma unroll
    for (int c = 0; c < CF; ++c)
#pragma unroll
      for (int m = 0; m < MF; ++m)
        acc[c][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, f[c]),
                                                            __builtin_bit_cast(bf16x8_t, f[CF + m]), acc[c][m], 0, 0, 0);
  }
  __syncthreads();  // every ring is done with
  auto red = [&](int w, int f, int l) -> f32x4_t & {
    return reinterpret_cast<f32x4_t *>(lds)[(w * CF * MF + f) * 64 + l];
  };
  // acc[c][m][v]: column 16 c + 4 g + v, token i16 of group m
#pragma unroll
  for (int c = 0; c < CF; ++c)
#pragma unroll
    for (int m = 0; m < MF; ++m) red(wave, c * MF + m, lane) = acc[c][m];
  __syncthreads();
  auto unpack = [](const bf16_t *a) {
    const uint2 b = *reinterpret_cast<const uint2 *>(a);
    return f32x4_t{__uint_as_float(b.x << 16), __uint_as_float(b.x & 0xffff0000u), __uint_as_float(b.y << 16),
                   __uint_as_float(b.y & 0xffff0000u)};
  };
  const ActSigmoid sg = act_sigmoid(p.act);
  for (int it = threadIdx.x; it < CF * MF * 64; it += WAVES * 64) {
    const int f = it >> 6, l = it & 63;
    const int t = t0 + f % MF * 16 + (l & 15);
    if (t >= p.M) continue;
    const int64_t o = (int64_t)t * p.ldc + k0 + f / MF * 16 + (l >> 4) * 4;
    f32x4_t v = red(0, f, l);
#pragma unroll
    for (int w = 1; w < WAVES; ++w) {
      const f32x4_t q = red(w, f, l);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += q[e];
    }
    if (p.act) {
      const f32x4_t z = unpack(p.H + o);
      with_act(p.act, [&](auto act) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] *= act_slope<decltype(act)::value>(z[e], sg);
      });
    }
    if (p.add) {
      const f32x4_t a = unpack(p.add + o);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += a[e];
    }
    *reinterpret_cast<uint2 *>(p.C + o) = make_uint2(pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]));
  }
}

// 32 columns a workgroup while each has a CU, 64 otherwise; then as few tokens as
// leave a CU to each.
template <int CB>
static void few_dx(const FfnTileParams &p, hipStream_t s) {
  const unsigned gx = (unsigned)(p.N / CB);  // p.N: a multiple of 64
  const int64_t groups = ceil_div(p.M, 16);
  const auto fits = [&](int mf) { return gx * ceil_div(groups, mf) <= persistent_grid(); };
  const auto grid = [&](int mf) { return dim3(gx, (unsigned)ceil_div(groups, mf)); };
  if (groups == 1 || fits(1)) linear_few_dx_kernel<CB, 1><<<grid(1), 512, 0, s>>>(p);
  else if (groups == 2 || fits(2)) linear_few_dx_kernel<CB, 2><<<grid(2), 512, 0, s>>>(p);
  else linear_few_dx_kernel<CB, 3><<<grid(3), 512, 0, s>>>(p);
}

// Taken while 64 columns and 48 tokens a workgroup leave a CU to each; from there on
// the tiles win. us against the tiles: 8192 columns, 2048 rows, 96 tokens (256
// workgroups) 9.7, 14.9, 128 tokens (384) 17.0, 15.6; 4096 x 4096, 192 tokens (256)
// 16.7, 27.9, 256 tokens (384) 29.3, 27.9; 2048 columns, 8192 rows, 320 tokens (224)
// 26.8, 53.1, 400 tokens (288) 49.8, 52.1; 16384 columns, 2048 rows, one token (256)
// 12.4, 15.5, 65536 columns, 256 rows (1024) 8.3, 7.2.
inline bool linear_few_dx_fits(const FfnTileParams &p) {
  return p.N / 64 * ceil_div(ceil_div(p.M, 16), 3) <= persistent_grid();
}

inline hipError_t run_linear_few_dx(const FfnTileParams &p, hipStream_t s) {
  if (p.N / 32 * ceil_div(ceil_div(p.M, 16), 3) <= persistent_grid()) few_dx<32>(p, s);
  else few_dx<64>(p, s);
  return hipGetLastError();
}

}  // namespace moe
