// The products of the Newton-Schulz iteration on the gfx950 matrix cores, for
// a batch of matrices X [S, L] (S <= L, both padded with zeros to multiples of
// 64), one step of which is
//   gram   A = X X^T            [S, S], symmetric
//   poly   B = b A + c A A      [S, S], symmetric
//   step   X' = a X + B X       [S, L]
//
// Operands are fp16 and sums fp32. fp16 keeps 11 bits where bf16 keeps 8, at
// the same rate; its range is no limit here, because every tensor's largest
// singular value is known (about 1, checked on the host for other
// coefficients): each is stored times 2^12, so that elements from 2^-26 to 8
// are normal numbers. Three roundings that would still show are avoided:
//   X is held as a high and a low half (22 bits). The products read the high
//     one; the term a X, which carries X while B X is small, reads both.
//   The diagonals of A and B, where nearly orthogonal rows put all their
//     weight, are held apart in fp32 (DA, DB), the matrices' own diagonals
//     being zero:  A A = A'A' + (DA_i + DA_j) A'_ij + DA_i^2 [i = j]  and
//     a X + B X = (a + DB_i) X + B'X.
// Measured on a 704 x 1024 matrix against fp64: 5e-4 of the norm, 1.4e-3
// without, 1e-2 with everything in bf16; where a few directions hold all the
// weight, 4e-4, 3e-2 and 2e-1.
//
// The kernel is the dense block's tile (ffn_kernel.h): a ring of 64-deep
// stages filled by the LDS DMA, 32 x 32 x 16 MFMAs with swapped operands, KG
// groups of wavefronts sharing a tile's stages where tiles are few. The two
// symmetric products compute the tiles on and below the diagonal and store
// each twice.
#pragma once

#include "gemm_bf16_kernel.h"

namespace moe {

enum { ORTH_GRAM = 0, ORTH_POLY = 1, ORTH_STEP = 2 };

typedef uint16_t half_t;  // fp16 storage (bit pattern)
typedef __attribute__((__vector_size__(8 * sizeof(_Float16)))) _Float16 f16x8_t;

constexpr float kOrthScale = 4096.f;           // what every fp16 tensor is multiplied with
constexpr float kOrthUnscale = 1.f / 4096.f;

struct OrthTileParams {
  const half_t *A, *B;      // operands, per matrix
  half_t *C;                // GRAM: A', POLY: B', STEP: high half of X'
  half_t *Clo;              // STEP: low half of X'
  const half_t *Xlo;        // STEP: low half of X (its high half is B)
  const float *diag;        // POLY: DA, STEP: DB (with a added)
  float *diag_out;          // GRAM: DA, POLY: DB + a
  float ca, cb, cc;         // coefficients a, b, c
  int M, N, K;              // all multiples of 64
  int64_t lda, ldb, ldc;
  int64_t strideA, strideB, strideC;  // from one matrix to the next
  int S;                    // stride of the diagonals
  int m_tiles, n_tiles, tiles;        // tiles: of one matrix
  int64_t total;            // tiles of all matrices
};

MOE_DEVICE uint32_t pack_h2(float a, float b) {  // nearest-even
  typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
  const f16x2_t v = {(_Float16)a, (_Float16)b};
  return __builtin_bit_cast(uint32_t, v);
}
MOE_DEVICE half_t f2h(float a) { return __builtin_bit_cast(half_t, (_Float16)a); }
MOE_DEVICE float h2f(half_t a) { return (float)__builtin_bit_cast(_Float16, a); }
MOE_DEVICE void unpack_h2(uint32_t v, float &a, float &b) {
  a = h2f((half_t)(v & 0xffffu));
  b = h2f((half_t)(v >> 16));
}

// vdst's upper lanes trade places with vsrc's lower ones.
MOE_DEVICE void orth_swap32(uint32_t &a, uint32_t &b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}

template <int BM, int BN, int WM, int WN, int KG, int STAGES, int MODE>
__global__ __launch_bounds__(KG * (BM / WM) * (BN / WN) * 64, 2) void orth_tile_kernel(OrthTileParams p) {
  constexpr bool BKM = MODE == ORTH_STEP;  // X is [k, n] there
  constexpr bool SYM = MODE != ORTH_STEP;
  static_assert(!SYM || BM == BN, "symmetric products have square tiles");
  constexpr int WAVES_M = BM / WM, WAVES_N = BN / WN, NW = WAVES_M * WAVES_N, NT = NW * 64;  // of a k group
  constexpr int FM = WM / 32, FN = WN / 32;
  constexpr int BK = 64, KS = 4;
  static_assert((KS * FM) % 2 == 0, "the A fragments alternate between two sets across stages");
  using OpA = Operand<BM, false, NW, BK>;
  using OpB = Operand<BN, BKM, NW, BK>;
  constexpr int STAGE_BYTES = OpA::BYTES + OpB::BYTES;
  constexpr int PER_STAGE = OpA::NDMA + OpB::NDMA;
  static_assert(KG * STAGES * STAGE_BYTES <= 160 * 1024, "LDS budget of one workgroup");
  static_assert((KG - 1) * BM * BN * 4 <= KG * STAGES * STAGE_BYTES, "the groups' sums meet in the rings");
  __shared__ u32x4_t lds[KG * STAGES * STAGE_BYTES / 16];

  // each XCD takes a contiguous share of the tiles, matrix by matrix
  const int64_t lo = (int64_t)(blockIdx.x & 7) * p.total >> 3, hi = (int64_t)((blockIdx.x & 7) + 1) * p.total >> 3;
  const int64_t id = lo + (int64_t)(blockIdx.x >> 3);
  if (id >= hi) return;
  const int mat = (int)(id / p.tiles);
  const int t = (int)(id - (int64_t)mat * p.tiles);
  int mt, nt;
  if (SYM) {  // t = mt (mt + 1) / 2 + nt, nt <= mt
    mt = (int)((sqrtf(8.f * (float)t + 1.f) - 1.f) * 0.5f);
    while ((mt + 1) * (mt + 2) / 2 <= t) ++mt;
    while (mt * (mt + 1) / 2 > t) --mt;
    nt = t - mt * (mt + 1) / 2;
  } else {  // groups of row tiles, column tile outer
    const int per = kGroupM * p.n_tiles;
    const int grp = t / per, rem = t - grp * per;
    const int rows = min(kGroupM, p.m_tiles - grp * kGroupM);
    nt = rem / rows;
    mt = grp * kGroupM + (rem - nt * rows);
  }
  const int m0 = mt * BM, n0 = nt * BN;
  const int m_valid = min(BM, p.M - m0), n_valid = min(BN, p.N - n0);

  const int kg = KG == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / NT);
  const char *ldsc = reinterpret_cast<const char *>(lds) + kg * (STAGES * STAGE_BYTES);
  const int tid = KG == 1 ? threadIdx.x : threadIdx.x % NT;
  const int lane = tid & 63, wave = tid >> 6;
  const int wm = wave / WAVES_N, wn = wave % WAVES_N;
  const int l32 = lane & 31, lhi = lane >> 5;
  const int wave_u = __builtin_amdgcn_readfirstlane(wave);

  const half_t *Ab = p.A + mat * p.strideA + (int64_t)m0 * p.lda;
  const half_t *Bb = p.B + mat * p.strideB + (BKM ? (int64_t)n0 : (int64_t)n0 * p.ldb);
  OpA opa;
  OpB opb;
  opa.init(Ab, p.lda, m_valid, wave, lane, [&](int r) { return r < m_valid ? r : m_valid - 1; });
  opb.init(Bb, p.ldb, n_valid, wave, lane, [&](int r) { return BKM || r < n_valid ? r : n_valid - 1; });

  const uint32_t lds0 = (uint32_t)(uintptr_t)ldsc;
  auto issue = [&](int kt) {  // the group's stage kt
    const uint32_t sb = lds0 + (uint32_t)(kt % STAGES * STAGE_BYTES);
    const int ks = kt * KG + kg;
    opa.issue(ks * BK, p.lda, p.K, sb, wave_u);
    opb.issue(ks * BK, p.ldb, p.K, sb + OpA::BYTES, wave_u);
  };
  auto load_a = [&](int slot, int ks, int i) {
    return __builtin_bit_cast(f16x8_t, opa.frag(ldsc + slot * STAGE_BYTES, wm * WM + i * 32, ks, lane));
  };
  auto load_b = [&](int slot, int ks, int j) {
    return __builtin_bit_cast(f16x8_t, opb.frag(ldsc + slot * STAGE_BYTES + OpA::BYTES, wn * WN + j * 32, ks, lane));
  };

  f32x16_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

  const int stages = p.K / BK;
  const int nk = (stages - kg + KG - 1) / KG;  // the group's own
  const int nk_max = (stages + KG - 1) / KG;   // barriers are the workgroup's
  f16x8_t fa[2], fb[2][FN];
  auto mma = [&](int i, int set_a, int set_b) {
#pragma unroll
    for (int j = 0; j < FN; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fb[set_b][j], fa[set_a], acc[i][j], 0, 0, 0);
  };
  // wait until at most `younger` whole stages are still in flight
  auto wait_stages = [&](int younger) {
    if (STAGES > 3 && younger >= 3) wait_vm<3 * PER_STAGE>();
    else if (STAGES > 2 && younger >= 2) wait_vm<2 * PER_STAGE>();
    else if (younger >= 1) wait_vm<PER_STAGE>();
    else wait_vm<0>();
  };
  for (int st = 0; st < STAGES; ++st)
    if (st < nk) issue(st);
  wait_stages(min(nk, STAGES) - 1);
  barrier();
  fa[0] = load_a(0, 0, 0);
#pragma unroll
  for (int j = 0; j < FN; ++j) fb[0][j] = load_b(0, 0, j);

  constexpr int NG = KS * FM;
  for (int kt = 0; kt < nk_max; ++kt) {
    const int slot = kt % STAGES;
    const bool mine = KG == 1 || kt < nk;  // uniform over the group
    if (mine) {
#pragma unroll
      for (int g = 0; g < NG - 1; ++g) {
        const int ks = g / FM, i = g % FM;
        fa[(g + 1) & 1] = load_a(slot, (g + 1) / FM, (g + 1) % FM);
        if (i == 0 && ks + 1 < KS) {
#pragma unroll
          for (int j = 0; j < FN; ++j) fb[(ks + 1) & 1][j] = load_b(slot, ks + 1, j);
        }
        mma(i, g & 1, ks & 1);
      }
    }
    // every fragment of this stage is in registers: its slot takes stage
    // kt + STAGES once all wavefronts are here, and stage kt + 1 has landed
    __builtin_amdgcn_sched_barrier(0);
    wait_lds();
    wait_stages(min(STAGES - 2, nk - 2 - kt));
    barrier();
    if (kt + STAGES < nk) issue(kt + STAGES);
    // the first fragments of the next stage (on the last pass a harmless
    // read of a stale slot)
    const int nslot = (kt + 1) % STAGES;
    fa[0] = load_a(nslot, 0, 0);
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[0][j] = load_b(nslot, 0, j);
    if (mine) mma(FM - 1, 1, (KS - 1) & 1);
  }

  if constexpr (KG > 1) {
    // the groups' sums, added in the order of the groups by the first one
    __syncthreads();  // every ring is done with
    f32x4_t *sum = reinterpret_cast<f32x4_t *>(lds);
    auto at = [&](int g, int f, int q) -> f32x4_t & { return sum[((g * FM * FN + f) * 4 + q) * NT + tid]; };
    if (kg > 0) {
#pragma unroll
      for (int f = 0; f < FM * FN; ++f)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x16_t &a = acc[f / FN][f % FN];
          at(kg - 1, f, q) = f32x4_t{a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]};
        }
    }
    __syncthreads();
    if (kg > 0) return;
#pragma unroll
    for (int g = 0; g < KG - 1; ++g)
#pragma unroll
      for (int f = 0; f < FM * FN; ++f)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x4_t v = at(g, f, q);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[f / FN][f % FN][4 * q + e] += v[e];
        }
  }

  // Epilogue. acc[i][j][4g + q] is row i*32 + l32, column j*32 + 8g + 4*lhi + q
  // of the wavefront's sub-tile; chunk (j, gp) of a lane is the 8 columns from
  // j*32 + 16*gp + 8*lhi.
  auto pack_chunk = [&](const float *v) -> u32x4_t {  // v: groups 2gp (4 values) and 2gp + 1
    uint32_t e0 = pack_h2(v[0], v[1]), e1 = pack_h2(v[2], v[3]);
    uint32_t o0 = pack_h2(v[4], v[5]), o1 = pack_h2(v[6], v[7]);
    orth_swap32(e0, o0);
    orth_swap32(e1, o1);
    return u32x4_t{e0, e1, o0, o1};
  };
  auto unpack_chunk = [&](const u32x4_t &c, float *v) {  // the inverse
    uint32_t e0 = c[0], e1 = c[1], o0 = c[2], o1 = c[3];
    orth_swap32(e0, o0);
    orth_swap32(e1, o1);
    unpack_h2(e0, v[0], v[1]);
    unpack_h2(e1, v[2], v[3]);
    unpack_h2(o0, v[4], v[5]);
    unpack_h2(o1, v[6], v[7]);
  };
  int el32 = l32, ehi = lhi;
  // opaque: no address below is formed above the main loop and held there
  asm volatile("" : "+v"(el32), "+v"(ehi));
  const int row_l = wm * WM + el32;
  half_t *C = p.C + mat * p.strideC;
  const u32x4_t zero = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int r = row_l + i * 32;
    const bool rok = r < m_valid;
    const int gr = m0 + (rok ? r : 0);
    const int64_t ro = (int64_t)gr * p.ldc;
    const float dr = MODE == ORTH_GRAM ? 0.f : p.diag[(int64_t)mat * p.S + gr];
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int gp = 0; gp < 2; ++gp) {
        const int cb = n0 + wn * WN + j * 32 + 16 * gp;  // of the chunk pair
        const int c = cb + 8 * ehi;
        const bool ok = rok && c < p.N;
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = acc[i][j][8 * gp + q] * kOrthUnscale;
        if constexpr (MODE == ORTH_STEP) {
          const half_t *xh = p.B + mat * p.strideB;
          float h[8], l[8];
          unpack_chunk(ok ? ld16(xh + ro + c) : zero, h);
          unpack_chunk(ok ? ld16(p.Xlo + mat * p.strideC + ro + c) : zero, l);
#pragma unroll
          for (int q = 0; q < 8; ++q) v[q] = fmaf(dr, h[q] + l[q], v[q]);
          const u32x4_t o = pack_chunk(v);
#pragma unroll
          for (int q = 0; q < 8; ++q) l[q] = v[q] - h2f(f2h(v[q]));
          const u32x4_t ol = pack_chunk(l);
          if (ok) {
            st16(C + ro + c, o);
            st16(p.Clo + mat * p.strideC + ro + c, ol);
          }
        } else {
          // column of v[q]: groups 2gp (q < 4) and 2gp + 1, 8 apart
          auto col = [&](int q) { return cb + 8 * (q >> 2) + 4 * ehi + (q & 3); };
          if constexpr (MODE == ORTH_POLY) {
            float a[8];
            unpack_chunk(ok ? ld16(p.A + mat * p.strideA + ro + c) : zero, a);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const int cc = col(q);
              const float dc = p.diag[(int64_t)mat * p.S + (cc < p.N ? cc : 0)];
              if (cc == m0 + r) a[q] = 0.5f * dr;  // (DA_i + DA_j) a = DA_i^2 on the diagonal, and b a below
              const float bb = cc == m0 + r ? 2.f * p.cb : p.cb;
              v[q] = fmaf(bb, a[q], p.cc * fmaf((dr + dc) * kOrthUnscale, a[q], v[q]));
            }
          }
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (col(q) == m0 + r) {
              if (rok) p.diag_out[(int64_t)mat * p.S + gr] = MODE == ORTH_GRAM ? v[q] : fmaf(v[q], kOrthUnscale, p.ca);
              v[q] = 0.f;
            }
          const u32x4_t o = pack_chunk(v);
          if (ok) st16(C + ro + c, o);
          if (mt != nt && rok) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const int cc = col(q);
              if (cc < p.N) C[(int64_t)cc * p.ldc + gr] = f2h(v[q]);
            }
          }
        }
      }
  }
}

template <int BM, int BN, int WM, int WN, int KG, int STAGES, int MODE>
hipError_t run_orth_tile(OrthTileParams p, int64_t batch, hipStream_t s) {
  constexpr int NT = KG * (BM / WM) * (BN / WN) * 64;
  p.m_tiles = (p.M + BM - 1) / BM;
  p.n_tiles = (p.N + BN - 1) / BN;
  p.tiles = MODE == ORTH_STEP ? p.m_tiles * p.n_tiles : p.m_tiles * (p.m_tiles + 1) / 2;
  p.total = batch * p.tiles;
  const unsigned grid = (unsigned)(ceil_div(p.total, 8) * 8);
  orth_tile_kernel<BM, BN, WM, WN, KG, STAGES, MODE><<<dim3(grid), NT, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace moe
