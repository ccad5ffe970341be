// The dense block's forward products for few tokens (decode steps): bound by
// reading the weights, each once, and by the latency of a few launches.
//
// What counts is that every CU draws on the memory at once and has enough in
// flight. A workgroup owns 16 weight rows (64 rows, 88 workgroups for F =
// 2816, took 14 us at one token where 16 take 6), or 32 where 16 would make
// more workgroups than CUs, and 16 MF tokens; each of its
// wavefronts takes a run of the k steps (a step is 128 contiguous bytes of
// every row) through an LDS ring of its own, filled by the LDS DMA in whole
// 128-byte lines: no barrier until the partial sums meet, added in the order
// of the wavefronts. (Loads straight into MFMA operands touch 16 half lines
// each: 5.2 against 3.9 us at one token, 12 against 7 us at 64.) The 16-row
// MFMA holds weight rows as its first operand: a lane ends with 4 consecutive
// output columns of one token.
//
// A gate/up fragment is 8 gate rows and the 8 up rows that go with them. Its 8
// columns of a are a quarter of a block of the 8-bit form, so there a is
// written in fp32 and quantised by a kernel of its own.
//
// Measured: one token, 2048 x 1408, bf16: gate/up 4.0 us (2.9 TB/s of
// weights), down 3.5 us, of which some 2 us are a kernel's start and end; 48
// tokens, 4096 x 2816, 8-bit: gate/up 8.4 us (2.8 TB/s), down 5.6 us (2.1 TB/s).
// Bound by the launches and each kernel's start, and by what a CU draws.
#pragma once

#include "ffn_kernel.h"

namespace moe {

template <bool F8, int NR, int MF, int WAVES, int EPI>
__global__ __launch_bounds__(WAVES * 64, 2) void ffn_few_kernel(FfnTileParams p) {
  constexpr int UNITS = 64;                    // 16-bit units of k per step: 128 bytes of a row
  constexpr int ROWS = 16 * NR + 16 * MF;      // weight rows, then tokens
  constexpr int NDMA = ROWS / 8;               // 8 rows of 128 bytes per DMA instruction
  constexpr int NSC = F8 ? (ROWS + 63) / 64 : 0;  // scale instructions: one dword per lane
  constexpr int PER = NDMA + NSC;              // instructions per step
  constexpr int STEP_BYTES = ROWS * 128 + NSC * 256;
  // two workgroups of 4 wavefronts or one of 8 fit a CU's 160 KB; 32 weight
  // rows with 48 tokens, 4 wavefronts alone
  constexpr int BUDGET = (NR == 2 && MF == 3 ? 40 : 20) * 1024;
  constexpr int SLOTS = BUDGET / STEP_BYTES < 4 ? BUDGET / STEP_BYTES : 4;
  constexpr int WAVE_BYTES = SLOTS * STEP_BYTES;
  static_assert(SLOTS >= 2 && WAVES * WAVE_BYTES <= 160 * 1024, "LDS budget of one workgroup");
  static_assert(NR * MF * 1024 <= WAVE_BYTES, "the partial sums meet in the rings");
  __shared__ u32x4_t lds[WAVES * WAVE_BYTES / 16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i16 = lane & 15, g = lane >> 4;
  const int t0 = blockIdx.y * 16 * MF;
  const int n0 = blockIdx.x * NR * (EPI == FFN_SWIGLU_FWD ? 8 : 16);  // first output column

  // source row of row r of a step: weight rows, then tokens (rows past the
  // last one feed dropped results)
  auto weight_row = [&](int r) {
    return EPI == FFN_SWIGLU_FWD ? n0 + r / 16 * 8 + (r & 7) + (r & 8 ? p.F : 0) : n0 + r;
  };
  auto token_row = [&](int r) { return min(t0 + r, p.M - 1); };
  const bf16_t *src[NDMA];
#pragma unroll
  for (int i = 0; i < NDMA; ++i) {
    const int r = i * 8 + lane / 8, c = (lane % 8) ^ (r & 7);
    src[i] = (i < 2 * NR ? p.B + (int64_t)weight_row(r) * p.ldb : p.A + (int64_t)token_row(r - 16 * NR) * p.lda) + c * 8;
  }
  const uint8_t *ssrc[NSC + 1];
#pragma unroll
  for (int i = 0; i < NSC; ++i) {
    const int64_t sld = p.K / 16;  // scales of a row
    const int r = min(i * 64 + lane, ROWS - 1);
    ssrc[i] = r < 16 * NR ? p.Bs + weight_row(r) * sld : p.As + token_row(r - 16 * NR) * sld;
  }
  const char *ring = reinterpret_cast<const char *>(lds) + wave * WAVE_BYTES;
  const uint32_t ring0 = (uint32_t)(uintptr_t)ring;

  // the wavefront's run of steps, in a ring of its own: no barrier until the
  // sums meet
  const int n = p.K / UNITS;
  const int cnt = (n + WAVES - 1) / WAVES;
  const int first = min(wave * cnt, n);
  const int steps = min(cnt, n - first);
  auto issue = [&](int s) {
    const uint32_t dst = ring0 + (uint32_t)(s % SLOTS * STEP_BYTES);
#pragma unroll
    for (int i = 0; i < NDMA; ++i) dma16(src[i] + (first + s) * UNITS, dst + (uint32_t)(i * 1024));
#pragma unroll
    for (int i = 0; i < NSC; ++i) dma4(ssrc[i] + (first + s) * 4, dst + (uint32_t)(ROWS * 128 + i * 256));
  };
  auto wait_steps = [&](int younger) {  // until at most `younger` steps are in flight
    if (SLOTS > 3 && younger >= 3) wait_vm<3 * PER>();
    else if (SLOTS > 2 && younger >= 2) wait_vm<2 * PER>();
    else if (younger >= 1) wait_vm<PER>();
    else wait_vm<0>();
  };
  // A lane reads bytes 16 g and 64 + 16 g of a row's 128: the scaled MFMA's
  // own k order (its first 16 bytes belong to the step's blocks 0 and 1, the
  // others to blocks 2 and 3). In bf16 the two are two products, whose k
  // order is any order that both operands share.
  f32x4_t acc[NR][MF];
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int m = 0; m < MF; ++m) acc[r][m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < SLOTS; ++s)
    if (s < steps) issue(s);
  for (int s = 0; s < steps; ++s) {
    wait_steps(min(SLOTS, steps - s) - 1);
    const char *t = ring + s % SLOTS * STEP_BYTES;
    u32x4_t f[NR + MF][2];
    int sc[NR + MF];
#pragma unroll
    for (int m = 0; m < NR + MF; ++m) {
      const int r = m * 16 + i16;
#pragma unroll
      for (int c = 0; c < 2; ++c)
        f[m][c] = *reinterpret_cast<const u32x4_t *>(t + r * 128 + (((c * 4 + g) ^ (r & 7)) * 16));
      if (F8) sc[m] = *reinterpret_cast<const uint8_t *>(t + ROWS * 128 + r * 4 + g);
    }
    wait_lds();  // the slot's bytes are in registers
#pragma unroll
    for (int m = 0; m < NR + MF; ++m) asm volatile("" : "+v"(f[m][0]), "+v"(f[m][1]));
    if (s + SLOTS < steps) issue(s + SLOTS);
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int m = 0; m < MF; ++m) {
        const u32x4_t *w = f[r], *x = f[NR + m];
        if constexpr (F8) {
          auto join = [](const u32x4_t &a, const u32x4_t &c) {
            return i32x8_t{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)c[0], (int)c[1], (int)c[2], (int)c[3]};
          };
          acc[r][m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(w[0], w[1]), join(x[0], x[1]), acc[r][m],
                                                                       0, 0, 0, sc[r], 0, sc[NR + m]);
        } else {
#pragma unroll
          for (int c = 0; c < 2; ++c)
            acc[r][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w[c]),
                                                                __builtin_bit_cast(bf16x8_t, x[c]), acc[r][m], 0, 0, 0);
        }
      }
  }
  __syncthreads();  // every ring is done with
  auto red = [&](int w, int f, int l) -> f32x4_t & {  // fragment f = r * MF + m
    return reinterpret_cast<f32x4_t *>(lds)[(w * NR * MF + f) * 64 + l];
  };
  // acc[r][m][v]: weight row 4 g + v of fragment r, token i16 of group m
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int m = 0; m < MF; ++m) red(wave, r * MF + m, lane) = acc[r][m];
  __syncthreads();
  auto total = [&](int f, int l) {
    f32x4_t v = red(0, f, l);
#pragma unroll
    for (int w = 1; w < WAVES; ++w) {
      const f32x4_t q = red(w, f, l);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += q[e];
    }
    return v;
  };
  auto store4 = [](bf16_t *dst, const f32x4_t &v) {
    *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]));
  };
  // a thread finishes 4 columns of a token at a time
  constexpr int TPG = EPI == FFN_SWIGLU_FWD ? 32 : 64;  // threads of a fragment
  for (int it = threadIdx.x; it < NR * MF * TPG; it += WAVES * 64) {
    const int l = it % TPG, f = it / TPG;
    const int t = t0 + f % MF * 16 + (l & 15);
    if (t >= p.M) continue;
    const int c = n0 + f / MF * (EPI == FFN_SWIGLU_FWD ? 8 : 16) + (l >> 4) * 4;
    f32x4_t v = total(f, l);
    if constexpr (EPI == FFN_STORE) {
      const int64_t o = (int64_t)t * p.ldc + c;
      if (p.add) {
        const uint2 b = *reinterpret_cast<const uint2 *>(p.add + o);
        v[0] += __uint_as_float(b.x << 16);
        v[1] += __uint_as_float(b.x & 0xffff0000u);
        v[2] += __uint_as_float(b.y << 16);
        v[3] += __uint_as_float(b.y & 0xffff0000u);
      }
      store4(p.C + o, v);
    } else {
      const f32x4_t uv = total(f, l + 32);
      if (p.C) {
        store4(p.C + (int64_t)t * p.ldc + c, v);
        store4(p.C + (int64_t)t * p.ldc + p.F + c, uv);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = silu_f(v[e]) * uv[e];
      if (F8) *reinterpret_cast<f32x4_t *>(p.a32 + (int64_t)t * p.F + c) = v;
      else store4(p.C2 + (int64_t)t * p.F + c, v);
    }
  }
}

// 16 weight rows a workgroup, while that is no more workgroups than CUs (8
// wavefronts, one a CU) or there are few tokens (4 wavefronts, two a CU, so
// that none waits for a second round); otherwise 32 rows, which read every
// token half as often.
template <bool F8, int MF, int EPI>
static void few_rows(const FfnTileParams &p, int groups, hipStream_t s) {
  const unsigned gx = (unsigned)(p.N / (EPI == FFN_SWIGLU_FWD ? 8 : 16));  // p.N: a multiple of 64
  const unsigned gy = (unsigned)((groups + MF - 1) / MF);
  if ((int64_t)gx * gy <= persistent_grid()) {
    ffn_few_kernel<F8, 1, MF, 8, EPI><<<dim3(gx, gy), 512, 0, s>>>(p);
  } else if constexpr (MF == 1) {
    ffn_few_kernel<F8, 1, MF, 4, EPI><<<dim3(gx, gy), 256, 0, s>>>(p);
  } else if constexpr (MF == 2) {
    ffn_few_kernel<F8, 2, MF, 8, EPI><<<dim3(gx / 2, gy), 512, 0, s>>>(p);
  } else {
    ffn_few_kernel<F8, 2, MF, 4, EPI><<<dim3(gx / 2, gy), 256, 0, s>>>(p);
  }
}

template <bool F8, int EPI>
hipError_t run_ffn_few(const FfnTileParams &p, hipStream_t s) {
  const int groups = (p.M + 15) / 16;
  if (groups == 1) few_rows<F8, 1, EPI>(p, groups, s);
  else if (groups == 2) few_rows<F8, 2, EPI>(p, groups, s);
  else few_rows<F8, 3, EPI>(p, groups, s);
  return hipGetLastError();
}

}  // namespace moe
