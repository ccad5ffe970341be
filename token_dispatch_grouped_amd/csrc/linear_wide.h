// The dense product's large tiles: forward and input gradient on the main loop
// of pingpong.h, epilogues in fp32.
#pragma once

#include "act.h"
#include "ffn_kernel.h"
#include "pingpong.h"

namespace moe {

// Epilogue of a wavefront's 128 x 64 of a tile, from row m0 and column col0 on;
// rows: that exist of it. Global memory is read and written in whole rows of a
// 32 x 64 block (8 lanes of 16 bytes), which the wavefront's own LDS scr turns
// into the accumulators' order and back; the loads of all blocks are in flight
// together, in the registers that the main loop's fragments have left. ADD:
// there is an addend; ACT (input gradient): there is an activation below.
template <bool DX, bool ADD, bool ACT>
MOE_DEVICE void linear_epilogue(const FfnTileParams &p, PpAcc &acc, char *scr, int m0, int rows, int col0) {
  if (col0 >= p.N || rows <= 0) return;  // 64 columns exist or none
  int lane = threadIdx.x & 63;
  // opaque: no address below is formed above the main loop and held there
  asm volatile("" : "+v"(lane));
  const RowBlock blk(scr, lane);
  const ActSigmoid sg = act_sigmoid(p.act);
  auto unpack = [](const uint2 &v) {
    return f32x4_t{__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                   __uint_as_float(v.y & 0xffff0000u)};
  };
  const uint32_t pitch = (uint32_t)p.ldc * 2u, off0 = (uint32_t)blk.rr * pitch + (uint32_t)blk.rc * 16u;
  auto off = [&](int b, int k) { return off0 + (uint32_t)(b * 32 + k * 8) * pitch; };
  const int64_t at0 = (int64_t)m0 * p.ldc + col0;
  // the first tensor read: z, or without one the addend; the second: the addend beside z
  constexpr bool TWO = DX && ACT && ADD;
  u32x4_t gf[4][4], gs[2][4];
  (void)gf;
  (void)gs;
  const TileRows first((DX && ACT ? p.H : p.add) + at0, pitch, rows), second(p.add + at0, pitch, rows);
  if constexpr (ADD || (DX && ACT)) {
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int k = 0; k < 4; ++k) gf[b][k] = first.load(off(b, k));
  }
  if constexpr (TWO) {
#pragma unroll
    for (int k = 0; k < 4; ++k) gs[0][k] = second.load(off(0, k));
  }
  uint2 bias[4];
  (void)bias;
  if (!DX && p.bias) {
#pragma unroll
    for (int j = 0; j < 4; ++j) bias[j] = *reinterpret_cast<const uint2 *>(p.bias + col0 + j * 16 + 4 * blk.l4);
  }
  const TileRows y(p.C + at0, pitch, rows), z(p.C2 + at0, pitch, p.C2 ? rows : 0);
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    if (b * 32 >= rows) break;
    if constexpr (TWO) {
      if (b + 1 < 4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) gs[(b + 1) & 1][k] = second.load(off(b + 1, k));
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    auto rows_out = [&](const TileRows &dst) {
      blk.rows_out(
          [&](int i, int j) {
            const f32x4_t &a = acc[b * 2 + i][j];
            return make_uint2(pack_bf2(a[0], a[1]), pack_bf2(a[2], a[3]));
          },
          [&](int k, const u32x4_t &v) { dst.store(off(b, k), v); });
    };
    if constexpr (DX && ACT) {
      with_act(p.act, [&](auto act) {
        blk.in_order(gf[b], [&](int i, int j, const uint2 &v) {
          const f32x4_t zv = unpack(v);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[b * 2 + i][j][e] *= act_slope<decltype(act)::value>(zv[e], sg);
        });
      });
    }
    if constexpr (!DX) {
      if (p.bias) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f32x4_t v = unpack(bias[j]);
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[b * 2 + i][j][e] += v[e];
        }
      }
      if (p.C2) rows_out(z);
      with_act(p.act, [&](auto act) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              acc[b * 2 + i][j][e] = act_value<decltype(act)::value>(acc[b * 2 + i][j][e], sg);
      });
    }
    if constexpr (ADD)
      blk.in_order(TWO ? gs[b & 1] : gf[b], [&](int i, int j, const uint2 &v) {
        const f32x4_t a = unpack(v);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[b * 2 + i][j][e] += a[e];
      });
    rows_out(y);
  }
}

template <bool DX, bool ADD, bool ACT>
__global__ __launch_bounds__(kPpThreads, 2) void linear_wide_kernel(FfnTileParams p) {
  __shared__ u32x4_t lds[(kPpLdsBytes + 8 * RowBlock::kBytes) / 16];  // all 160 KB
  int lo, hi;
  xcd_range(blockIdx.x & 7, (int64_t)p.m_tiles * p.n_tiles, lo, hi);
  const int step = gridDim.x >> 3;
  const int first = lo + (int)(blockIdx.x >> 3);
  if (first >= hi) return;
  PpCursor load, put;
  load.start(p.m_tiles, p.n_tiles, first);
  put = load;
  auto get = [&]() {
    const int m0 = load.mt * kPpTile, n0 = load.nt * kPpTile;
    PpTile t;
    t.A = p.A + (int64_t)m0 * p.lda;
    t.B = p.B + (DX ? (int64_t)n0 : (int64_t)n0 * p.ldb);
    t.m_valid = min(kPpTile, p.M - m0);
    t.n_valid = min(kPpTile, p.N - n0);
    load.step(p.m_tiles, p.n_tiles, step);
    return t;
  };
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  char *scr = reinterpret_cast<char *>(lds) + kPpLdsBytes + wave * RowBlock::kBytes;
  auto done = [&](PpAcc &acc) {
    const int m0 = put.mt * kPpTile + (wave >> 2) * 128;
    const FfnTileParams &p = late_args<FfnTileParams>();
    linear_epilogue<DX, ADD, ACT>(p, acc, scr, m0, min(128, p.M - m0), put.nt * kPpTile + (wave & 3) * 64);
    put.step(p.m_tiles, p.n_tiles, step);
  };
  pp_tiles<false, DX>(lds, p.lda, p.ldb, p.K / 64, (hi - first + step - 1) / step, get, done);
}

template <bool DX>
hipError_t run_linear_wide(FfnTileParams p, hipStream_t s) {
  p.m_tiles = (p.M + kPpTile - 1) / kPpTile;
  p.n_tiles = (p.N + kPpTile - 1) / kPpTile;
  const int64_t total = (int64_t)p.m_tiles * p.n_tiles;
  const int64_t grid = std::min<int64_t>(persistent_grid(), ceil_div(total, 8) * 8);
  const dim3 g((unsigned)grid);
  if constexpr (DX) {
    if (p.act && p.add) linear_wide_kernel<true, true, true><<<g, kPpThreads, 0, s>>>(p);
    else if (p.act) linear_wide_kernel<true, false, true><<<g, kPpThreads, 0, s>>>(p);
    else if (p.add) linear_wide_kernel<true, true, false><<<g, kPpThreads, 0, s>>>(p);
    else linear_wide_kernel<true, false, false><<<g, kPpThreads, 0, s>>>(p);
  } else {
    if (p.add) linear_wide_kernel<false, true, false><<<g, kPpThreads, 0, s>>>(p);
    else linear_wide_kernel<false, false, false><<<g, kPpThreads, 0, s>>>(p);
  }
  return hipGetLastError();
}

}  // namespace moe
