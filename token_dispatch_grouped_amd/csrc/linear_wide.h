// The dense product's large tiles: forward and input gradient on the main loop
// of pingpong.h, epilogues in fp32.
#pragma once

#include "act.h"
#include "ffn_kernel.h"
#include "pingpong.h"

namespace moe {

// Epilogue of a wavefront's 128 x 64 of a tile, from row m0 + row0 and column
// col0 on; m_valid: rows of the tile that exist. Global memory is read and
// written in whole rows of a 32 x 64 block (8 lanes of 16 bytes), which the
// wavefront's own LDS scr turns into the accumulators' order and back; the loads
// of a block are in flight together, at clamped addresses.
template <bool DX>
MOE_DEVICE void linear_epilogue(const FfnTileParams &p, PpAcc &acc, char *scr, int m0, int m_valid, int row0, int col0) {
  if (col0 >= p.N) return;  // 64 columns exist or none
  int lane = threadIdx.x & 63;
  // opaque: no address below is formed above the main loop and held there
  asm volatile("" : "+v"(lane));
  const RowBlock blk(scr, lane);
  const ActSigmoid sg = act_sigmoid(p.act);
  auto unpack = [](const uint2 &v) {
    return f32x4_t{__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                   __uint_as_float(v.y & 0xffff0000u)};
  };
  uint2 bias[4];
  (void)bias;
  if (!DX && p.bias) {
#pragma unroll
    for (int j = 0; j < 4; ++j) bias[j] = *reinterpret_cast<const uint2 *>(p.bias + col0 + j * 16 + 4 * blk.l4);
  }
  u32x4_t gz[2][4], ga[2][4];  // a block's and the next one's
  (void)gz;
  auto load = [&](int b) {
    auto row_at = [&](int k) {
      const int r = row0 + b * 32 + k * 8 + blk.rr;
      return (int64_t)(m0 + (r < m_valid ? r : 0)) * p.ldc + col0 + blk.rc * 8;
    };
    if (DX && p.act) {
#pragma unroll
      for (int k = 0; k < 4; ++k) gz[b & 1][k] = ld16(p.H + row_at(k));
    }
    if (p.add) {
#pragma unroll
      for (int k = 0; k < 4; ++k) ga[b & 1][k] = ld16(p.add + row_at(k));
    }
  };
  load(0);
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const int rb = row0 + b * 32;
    if (rb >= m_valid) break;
    // the lane's row k * 8 + rr of the block
    auto row_ok = [&](int k) { return rb + k * 8 + blk.rr < m_valid; };
    auto row_at = [&](int k) { return (int64_t)(m0 + rb + k * 8 + blk.rr) * p.ldc + col0 + blk.rc * 8; };
    if (b + 1 < 4) load(b + 1);
    __builtin_amdgcn_sched_barrier(0);
    auto rows_out = [&](bf16_t *dst) {
      blk.rows_out(
          [&](int i, int j) {
            const f32x4_t &a = acc[b * 2 + i][j];
            return make_uint2(pack_bf2(a[0], a[1]), pack_bf2(a[2], a[3]));
          },
          [&](int k, const u32x4_t &v) {
            if (row_ok(k)) st16(dst + row_at(k), v);
          });
    };
    if constexpr (DX) {
      with_act(p.act, [&](auto act) {
        blk.in_order(gz[b & 1], [&](int i, int j, const uint2 &v) {
          const f32x4_t z = unpack(v);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[b * 2 + i][j][e] *= act_slope<decltype(act)::value>(z[e], sg);
        });
      });
    } else {
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
      if (p.C2) rows_out(p.C2);
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
    if (p.add)
      blk.in_order(ga[b & 1], [&](int i, int j, const uint2 &v) {
        const f32x4_t a = unpack(v);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[b * 2 + i][j][e] += a[e];
      });
    rows_out(p.C);
  }
}

template <bool DX>
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
    const int m0 = put.mt * kPpTile;
    linear_epilogue<DX>(p, acc, scr, m0, min(kPpTile, p.M - m0), (wave >> 2) * 128, put.nt * kPpTile + (wave & 3) * 64);
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
  linear_wide_kernel<DX><<<dim3((unsigned)grid), kPpThreads, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace moe
