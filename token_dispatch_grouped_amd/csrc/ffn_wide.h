// The dense block's products on the grouped products' 256 x 256 tile, for
// row counts that fill the card with it: the same main loop, DMA ring and
// epilogues (gg_tile), one group of p.M rows instead of an offsets table.
// Persistent, one workgroup per CU, each XCD walking a contiguous share of
// the tiles; the next tile's first stage is issued during the epilogue.
// Bound by the main loop's operand stream from L2 to LDS. Measured at d =
// 2048, F = 1408: 16384 tokens gate/up with SwiGLU 179 us (1.06 PFLOP/s), down
// 89 us (1.06) and 106-111 us with an addend; 7001 tokens down's input gradient
// 70 us, gate/up's with an addend 86 us (0.94), one round of tiles each.
#pragma once

#include "gemm_bf16_kernel.h"

namespace moe {

template <bool BKM, int EPI>
__global__ __launch_bounds__(512, 1) void ffn_wide_kernel(GemmParams p) {
  constexpr int BM = kGemmBM, BN = kGemmBN, WM = BM / 2, WN = BN / 4;
  constexpr int STAGE_BYTES = (BM + BN) * kStageK * 2;
  static_assert(BM * BN * 2 <= 2 * STAGE_BYTES, "the epilogues stage within the ring");
  __shared__ u32x4_t lds[2 * STAGE_BYTES / 16];
  const int per = kGroupM * p.n_tiles;
  int lo, hi;
  xcd_range(blockIdx.x & 7, (int64_t)p.m_tiles * p.n_tiles, lo, hi);
  const int nW = gridDim.x >> 3;
  auto decode = [&](int bid, int &m0, int &n_tile, int &m_valid) {
    const int grp = bid / per, rem = bid - grp * per;
    const int rows = min(kGroupM, p.m_tiles - grp * kGroupM);  // of the last group fewer
    n_tile = rem / rows;
    m0 = (grp * kGroupM + (rem - n_tile * rows)) * BM;
    m_valid = min(BM, p.M - m0);
  };
  bool pre = false;  // this tile's stage 0 is already in flight
  for (int bid = lo + (int)(blockIdx.x >> 3); bid < hi; bid += nW) {
    int m0, n_tile, m_valid;
    decode(bid, m0, n_tile, m_valid);
    bool nvalid = false;
    auto next_tile = [&](NextTile &nx) {
      int nm0 = 0;
      nx.valid = bid + nW < hi;
      if (nx.valid) decode(bid + nW, nm0, nx.n_tile, nx.m_valid);
      nx.Ab = p.A + (int64_t)nm0 * p.lda;
      nx.Bb = p.B;
      nvalid = nx.valid;
    };
    gg_tile<BM, BN, WM, WN, 8, false, BKM, EPI, false, kStageK, kStages>(
        p, lds, 0, m0, n_tile, m_valid, p.K, m0, p.A + (int64_t)m0 * p.lda, p.B, pre, next_tile);
    pre = nvalid;
    __syncthreads();  // the epilogue's LDS reads are done before the next tile's DMA
  }
}

template <bool BKM, int EPI>
hipError_t run_ffn_wide(GemmParams p, hipStream_t s) {
  p.m_tiles = (p.M + kGemmBM - 1) / kGemmBM;
  p.n_tiles = EPI == EPI_SWIGLU_FWD ? (p.N + kGemmBN / 2 - 1) / (kGemmBN / 2) : (p.N + kGemmBN - 1) / kGemmBN;
  const int64_t L = (int64_t)p.m_tiles * p.n_tiles;
  const int grid = (int)std::min<int64_t>(persistent_grid(), (L + 7) / 8 * 8);
  ffn_wide_kernel<BKM, EPI><<<dim3((unsigned)grid), 512, 0, s>>>(p);
  return hipGetLastError();
}

extern template hipError_t run_ffn_wide<false, EPI_SWIGLU_FWD>(GemmParams, hipStream_t);

}  // namespace moe
