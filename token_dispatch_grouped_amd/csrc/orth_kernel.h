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
//     one; the term a X, which carries X while B X is small, reads both (the
//     last step, where little is left to carry, the high one).
//   The diagonals of A and B, where nearly orthogonal rows put all their
//     weight, are held apart in fp32 (DA, DB), the matrices' own diagonals
//     being zero:  A A = A'A' + (DA_i + DA_j) A'_ij + DA_i^2 [i = j]  and
//     a X + B X = (a + DB_i) X + B'X.
// Measured on a 704 x 1024 matrix against fp64: 5e-4 of the norm, 1.3e-3
// without, 1e-2 with everything in bf16; where a few directions hold nearly
// all the weight, 8e-4, 3e-2 and 2e-1. Where the short side is short those
// roundings are larger (fewer terms average them) and the products cheap: there
// (orth_both_halves) X, A' and B' are held in two halves throughout and each
// product is high x high + high x low + low x high, 2e-7 of the norm.
//
// The kernel is the dense block's tile (ffn_kernel.h): a ring of stages of 64 k (32 in
// both halves) filled by the LDS DMA, MFMAs with swapped operands, KG
// groups of wavefronts sharing a tile's stages where tiles are few. The two
// symmetric products compute the tiles on and below the diagonal and store
// each twice.
#pragma once

#include "mx8.h"
#include "pingpong.h"

namespace moe {

// LAST: the step whose result goes out, as o or into the weights (MUON)
enum { ORTH_GRAM = 0, ORTH_POLY = 1, ORTH_STEP = 2, ORTH_LAST = 3, ORTH_LAST_MUON = 4 };
constexpr bool orth_step(int mode) { return mode >= ORTH_STEP; }

typedef uint16_t half_t;  // fp16 storage (bit pattern)

constexpr float kOrthScale = 4096.f;           // what every fp16 tensor is multiplied with
constexpr float kOrthUnscale = 1.f / 4096.f;

// Where the last step's result goes: [batch, rows, cols], X itself or, tall, its
// transpose.
struct OrthOut {
  float *param;      // MUON: param = param * decay - step_size * X
  uint16_t *lowp;    // bf16: X, or MUON: the new param, or NULL
  int rows, cols, tall;
  float decay, step_size;
};

struct OrthTileParams {
  const half_t *A, *B;      // operands, per matrix
  half_t *C;                // GRAM: A', POLY: B', STEP: high half of X'
  half_t *Clo;              // STEP: low half of X', or NULL (the last X); BOTH: of every result
  const half_t *Xlo;        // STEP: low half of X (its high half is B), or NULL; BOTH, POLY: of A
  const float *diag;        // POLY: DA, STEP: DB (with a added)
  float *diag_out;          // GRAM: DA, POLY: DB + a
  float ca, cb, cc;         // coefficients a, b, c
  int M, N, K;              // all multiples of 64
  int64_t lda, ldb, ldc;
  int64_t strideA, strideB, strideC;  // from one matrix to the next
  int S;                    // stride of the diagonals
  int m_tiles, n_tiles, tiles;        // tiles: of one matrix
  int64_t total;            // tiles of all matrices
  int slices;               // GRAM: of the sum, whole stages each, in `sums`
  f32x4_t *sums;            // [tile, slice, fragment, thread]
  OrthOut out;              // LAST
  const half_t *Alo, *Blo;  // BOTH: the operands' low halves
};

MOE_DEVICE uint32_t pack_h2(float a, float b) {  // nearest-even
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
  const f32x2_t v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2_t));
}
MOE_DEVICE half_t f2h(float a) { return __builtin_bit_cast(half_t, (_Float16)a); }
MOE_DEVICE float h2f(half_t a) { return (float)__builtin_bit_cast(_Float16, a); }
MOE_DEVICE void unpack_h2(uint32_t v, float &a, float &b) {
  a = h2f((half_t)(v & 0xffffu));
  b = h2f((half_t)(v >> 16));
}

// A 4 x 4 transpose over lanes 4n .. 4n + 3: d0, d1 hold a lane's columns 0 .. 3 of
// fp16 as pairs; after it lane k of the four holds column k, its pairs the
// lanes' rows.
MOE_DEVICE void orth_quad_transpose(uint32_t &d0, uint32_t &d1, int lane) {
  const uint32_t t0 = dpp_u<kDppXor1>(d0), t1 = dpp_u<kDppXor1>(d1);
  const bool odd = lane & 1, upper = lane & 2;
  // even lanes: (own low, other's low); odd ones: (other's high, own high)
  const uint32_t p0 = odd ? __builtin_amdgcn_perm(d0, t0, 0x07060302u) : __builtin_amdgcn_perm(t0, d0, 0x05040100u);
  const uint32_t p1 = odd ? __builtin_amdgcn_perm(d1, t1, 0x07060302u) : __builtin_amdgcn_perm(t1, d1, 0x05040100u);
  const uint32_t r = dpp_u<kDppXor2>(upper ? p0 : p1);
  d0 = upper ? r : p0;
  d1 = upper ? p1 : r;
}

// The same for fp32: v[e] becomes row e of column `lane & 3`.
MOE_DEVICE void orth_quad_transpose(float (&v)[4], int lane) {
  const bool odd = lane & 1, upper = lane & 2;
  auto dpp = [](float x, auto ctrl) { return __uint_as_float(dpp_u<decltype(ctrl)::value>(__float_as_uint(x))); };
  constexpr std::integral_constant<int, kDppXor1> x1{};
  constexpr std::integral_constant<int, kDppXor2> x2{};
  const float r0 = dpp(odd ? v[0] : v[1], x1), r1 = dpp(odd ? v[2] : v[3], x1);
  // p: columns (0 or 1), s: columns (2 or 3), rows of the lane pair
  const float p0 = odd ? r0 : v[0], p1 = odd ? v[1] : r0, s0 = odd ? r1 : v[2], s1 = odd ? v[3] : r1;
  const float t0 = dpp(upper ? p0 : s0, x2), t1 = dpp(upper ? p1 : s1, x2);
  v[0] = upper ? t0 : p0;
  v[1] = upper ? t1 : p1;
  v[2] = upper ? s0 : t0;
  v[3] = upper ? s1 : t1;
}

// Epilogue of a wavefront's sub-tile of FM x 4 blocks of 16 x 16, from row m0 +
// row0 and column col0 on (FM 1: 16 rows); m_valid: rows of the tile that exist, mirror: store
// the transpose as well.
//
// Global memory is read and written in whole rows of a block of 32 rows, which the
// wavefront's own LDS scr turns into the accumulators' order and back. (Straight
// from registers an instruction touches 32 rows, 32 bytes of each, and the
// step's epilogue took 400 of 730 us.) The loads of a row block and the next one
// are in flight together.
template <int FM, int MODE, bool BOTH = false>
MOE_DEVICE void orth_epilogue(const OrthTileParams &p, f32x4_t (&acc)[FM][4], char *scr, int mat, int m0, int m_valid,
                              int row0, int col0, bool mirror) {
  constexpr int H = FM > 1 ? 2 : 1, RB = (FM + 1) / 2;  // blocks of 16 rows in a row block (of 32, or 16); row blocks
  static_assert(FM == 1 || FM % 2 == 0, "whole row blocks");
  constexpr bool STEP = orth_step(MODE);
  constexpr bool LAST = MODE == ORTH_LAST || MODE == ORTH_LAST_MUON;
  int lane = threadIdx.x & 63;
  // opaque: no address below is formed above the main loop and held there
  asm volatile("" : "+v"(lane));
  const RowBlock blk(scr, lane);
  const int l16 = blk.l16, l4 = blk.l4, rr = blk.rr, rc = blk.rc;
  auto unpack = [](const uint2 &v) {
    f32x4_t x;
    float a, b;
    unpack_h2(v.x, a, b);
    x[0] = a;
    x[1] = b;
    unpack_h2(v.y, a, b);
    x[2] = a;
    x[3] = b;
    return x;
  };
  auto pack = [](const f32x4_t &a) { return make_uint2(pack_h2(a[0], a[1]), pack_h2(a[2], a[3])); };
  // the part's rows in every tensor of X's (A's) shape: 32 of a block and 64
  // columns exist or none
  const int rows = col0 < p.N ? m_valid - row0 : 0;
  if (rows <= 0) return;
  const int r0 = m0 + row0;
  const int64_t at0 = (int64_t)r0 * p.ldc + col0;
  const uint32_t pitch = (uint32_t)p.ldc * 2u, off0 = (uint32_t)rr * pitch + (uint32_t)rc * 16u;
  auto off = [&](int i, int k) { return off0 + (uint32_t)(i * 32 + k * 8) * pitch; };
  const bool low = BOTH ? MODE != ORTH_GRAM : STEP && !LAST && p.Xlo;
  const TileRows src((STEP ? p.B + mat * p.strideB : p.A + mat * p.strideA) + at0, pitch, rows);  // X, or POLY: A
  const TileRows srclo(p.Xlo + mat * p.strideC + at0, pitch, low ? rows : 0);
  const TileRows dst(p.C + mat * p.strideC + at0, pitch, rows), dstlo(p.Clo + mat * p.strideC + at0, pitch, p.Clo ? rows : 0);
  const float *diag = p.diag + (int64_t)mat * p.S;
  const OrthOut &out = p.out;
  const bool ovec = (out.cols & 3) == 0;
  u32x4_t gh[2][4], gl[2][4];  // of a row block and the next one
  f32x4_t pv[2][4];
  (void)gh;
  (void)gl;
  (void)pv;
  // the part's place in the matrices given, and its 32 x 32 fp32 blocks there:
  // row k * 8 + rr, 4 columns from rc * 4 on
  const int64_t obase = mat * (int64_t)out.rows * out.cols;
  const int orow0 = out.tall ? col0 : r0, ocol0 = out.tall ? r0 : col0;
  auto out_at = [&](int i, int j, int k, int &left) -> int64_t {
    const int orow = orow0 + (out.tall ? j : i) * 32 + k * 8 + rr, ocol = ocol0 + (out.tall ? i : j) * 32 + rc * 4;
    left = orow < out.rows && (H > 1 || (out.tall ? rc * 4 : k * 8 + rr) < 16) ? out.cols - ocol : 0;
    return obase + (left > 0 ? (int64_t)orow * out.cols + ocol : 0);
  };
  auto load_rows = [&](int i) {
    if constexpr (MODE != ORTH_GRAM) {
#pragma unroll
      for (int k = 0; k < 2 * H; ++k) gh[i & 1][k] = src.load(off(i, k));
    }
    if constexpr (MODE == ORTH_STEP || (BOTH && MODE != ORTH_GRAM)) {
#pragma unroll
      for (int k = 0; k < 2 * H; ++k) gl[i & 1][k] = srclo.load<2>(off(i, k));  // zeros where there is none
    }
  };
  auto load_param = [&](int i, int j) {
    if constexpr (MODE == ORTH_LAST_MUON) {
      if (!ovec) return;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        int left;
        pv[j][k] = *reinterpret_cast<const f32x4_t *>(out.param + out_at(i, j, k, left));
      }
    }
  };
  load_rows(0);
  load_param(0, 0);
  load_param(0, 1);
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    if (i * 32 >= rows) break;
    const int br = r0 + i * 32;
    if (i + 1 < RB) load_rows(i + 1);
    float dr[2] = {0.f, 0.f};
    if constexpr (MODE != ORTH_GRAM) {
      dr[0] = diag[br + l16];
      if (H > 1) dr[1] = diag[br + 16 + l16];
    }
    __builtin_amdgcn_sched_barrier(0);
    // acc -> the new values, in place
    auto acc_at = [&](int h, int j) -> f32x4_t & { return acc[i * 2 + h][j]; };
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc_at(h, j)[e] *= kOrthUnscale;
    auto col = [&](int j) { return col0 + j * 16 + 4 * l4; };  // of acc_at(., j)[0]
    if constexpr (STEP) {
      auto add = [&](int h, int j, const uint2 &g) {
        const f32x4_t v = unpack(g);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc_at(h, j)[e] = fmaf(dr[h], v[e], acc_at(h, j)[e]);
      };
      blk.template in_order<H>(gh[i & 1], add);
      if constexpr (MODE == ORTH_STEP || BOTH) {
        if (low) blk.template in_order<H>(gl[i & 1], add);
      }
    } else if constexpr (MODE == ORTH_POLY) {
      blk.template in_order<H>(gh[i & 1], [&](int h, int j, const uint2 &g) {
        const f32x4_t v = unpack(g);
        const f32x4_t dc = *reinterpret_cast<const f32x4_t *>(diag + col(j));
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc_at(h, j)[e] =
              fmaf(p.cb, v[e], p.cc * fmaf((dr[h] + dc[e]) * kOrthUnscale, v[e], acc_at(h, j)[e]));
      });
      if constexpr (BOTH)
        blk.template in_order<H>(gl[i & 1], [&](int h, int j, const uint2 &g) {
          const f32x4_t v = unpack(g);
          const f32x4_t dc = *reinterpret_cast<const f32x4_t *>(diag + col(j));
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc_at(h, j)[e] = fmaf(fmaf(p.cc, (dr[h] + dc[e]) * kOrthUnscale, p.cb), v[e], acc_at(h, j)[e]);
        });
    }
    if constexpr (!STEP) {
      if (br < col0 + 64 && col0 < br + 16 * H) {  // a block on the diagonal
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (col(j) + e == br + h * 16 + l16) {
                float x = acc_at(h, j)[e];
                // A' is zero there: b DA_i + c DA_i^2 is still to come
                if (MODE == ORTH_POLY)
                  x = fmaf(fmaf(p.cc * dr[h] * kOrthUnscale + p.cb, dr[h], x), kOrthUnscale, p.ca);
                p.diag_out[(int64_t)mat * p.S + br + h * 16 + l16] = x;
                acc_at(h, j)[e] = 0.f;
              }
      }
    }
    auto mirror_out = [&](half_t *C) {
      if (mirror) {
        // transposed: 64 columns of 32 (16) rows in scr, 64 bytes each, 16-byte
        // chunks swizzled by bits 1 and 2 of the column
        auto at = [&](int c, int ch) { return scr + c * 64 + ((ch ^ ((c >> 1) & 3)) * 16); };
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint2 d = pack(acc_at(h, j));
            orth_quad_transpose(d.x, d.y, lane);
            const int r4 = h * 4 + (l16 >> 2);  // rows 4 r4 .. of column 16 j + 4 l4 + (lane & 3)
            *reinterpret_cast<uint2 *>(at(j * 16 + 4 * l4 + (lane & 3), r4 >> 1) + (r4 & 1) * 8) = d;
          }
#pragma unroll
        for (int k = 0; k < 2 * H; ++k) {
          const int c = k * (32 / H) + (lane / (2 * H)), ch = lane % (2 * H);
          const u32x4_t v = *reinterpret_cast<const u32x4_t *>(at(c, ch));
          st16(C + mat * p.strideC + (int64_t)(col0 + c) * p.ldc + br + ch * 8, v);
        }
      }
    };
    if constexpr (!STEP) mirror_out(p.C);
    if constexpr (!LAST) {
      auto rows_out = [&](const TileRows &to) {
        blk.template rows_out<H>([&](int h, int j) { return pack(acc_at(h, j)); },
                     [&](int k, const u32x4_t &v) { to.store<2>(off(i, k), v); });
      };
      rows_out(dst);
      if ((STEP || BOTH) && p.Clo) {
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const f32x4_t hi = unpack(pack(acc_at(h, j)));
#pragma unroll
            for (int e = 0; e < 4; ++e) acc_at(h, j)[e] -= hi[e];
          }
        if constexpr (!STEP) mirror_out(p.Clo);
        rows_out(dstlo);
      }
    } else {
#pragma unroll
      for (int j2 = 0; j2 < 2; ++j2) {
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = acc_at(h, j2 * 2 + x)[e] * kOrthUnscale;
            if (out.tall) orth_quad_transpose(v, lane);
            const u32x4_t w = {__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
            if (out.tall) blk.at16(x * 16 + 4 * l4 + (lane & 3), h * 4 + (l16 >> 2)) = w;
            else blk.at16(h * 16 + l16, x * 4 + l4) = w;
          }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const u32x4_t w = blk.at16(k * 8 + rr, rc);
          float x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(w[e]);
          int left;
          const int64_t o = out_at(i, j2, k, left);
          if (left <= 0) continue;
          if (ovec) {
            if constexpr (MODE == ORTH_LAST_MUON) {
#pragma unroll
              for (int e = 0; e < 4; ++e) x[e] = fmaf(-out.step_size, x[e], pv[j2][k][e] * out.decay);
              *reinterpret_cast<f32x4_t *>(out.param + o) = f32x4_t{x[0], x[1], x[2], x[3]};
            }
            if (out.lowp)
              *reinterpret_cast<uint2 *>(out.lowp + o) = make_uint2(pack_bf2(x[0], x[1]), pack_bf2(x[2], x[3]));
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (e >= left) break;
              if constexpr (MODE == ORTH_LAST_MUON) {
                x[e] = fmaf(-out.step_size, x[e], out.param[o + e] * out.decay);
                out.param[o + e] = x[e];
              }
              if (out.lowp) out.lowp[o + e] = f2bf(x[e]);
            }
          }
        }
        if (i + 1 < RB) load_param(i + 1, j2);
      }
    }
  }
}

// A place in the order of the tiles: matrix by matrix; of a symmetric product
// the tiles on and below the diagonal, row by row.
template <bool SYM>
struct OrthCursor {
  int mat, mt, nt;
  PpCursor c;  // step

  MOE_DEVICE void start(const OrthTileParams &p, int64_t id) {
    mat = __builtin_amdgcn_readfirstlane((int)(id / p.tiles));
    const int t = __builtin_amdgcn_readfirstlane((int)(id - (int64_t)mat * p.tiles));
    if (SYM) {  // t = mt (mt + 1) / 2 + nt, nt <= mt
      mt = (int)((sqrtf(8.f * (float)t + 1.f) - 1.f) * 0.5f);
      while ((mt + 1) * (mt + 2) / 2 <= t) ++mt;
      while (mt * (mt + 1) / 2 > t) --mt;
      mt = __builtin_amdgcn_readfirstlane(mt);
      nt = t - mt * (mt + 1) / 2;
    } else {
      c.start(p.m_tiles, p.n_tiles, t);
      mt = c.mt;
      nt = c.nt;
    }
  }
  MOE_DEVICE void step(const OrthTileParams &p, int n) {
    if (SYM) {
      nt += n;
      while (nt > mt) {
        nt -= mt + 1;
        if (++mt == p.m_tiles) {
          mt = 0;
          ++mat;
        }
      }
    } else {
      mat += c.step(p.m_tiles, p.n_tiles, n);
      mt = c.mt;
      nt = c.nt;
    }
  }
};

// BOTH: every operand in both its halves. A stage is then 32 k, the high half's
// chunks (k-major: rows) in front of the low half's, and three products of them are
// taken: high x high, high x low, low x high (low x low is below fp32's rounding).
template <int BM, int BN, int WM, int WN, int KG, int STAGES, int MODE, bool BOTH>
__global__ __launch_bounds__(KG * (BM / WM) * (BN / WN) * 64, 2) void orth_tile_kernel(OrthTileParams p) {
  constexpr bool BKM = orth_step(MODE);  // X is [k, n] there
  constexpr bool SYM = !orth_step(MODE);
  static_assert(!SYM || BM == BN, "symmetric products have square tiles");
  constexpr int WAVES_M = BM / WM, WAVES_N = BN / WN, NW = WAVES_M * WAVES_N, NT = NW * 64;  // of a k group
  constexpr int FM = WM / 16, FN = WN / 16;
  constexpr int BK = 64, KS = 2;   // of a stage in LDS
  constexpr int STEP_K = BOTH ? 32 : BK;  // of the sum
  static_assert(FN == 4, "the epilogue's rows are 64 columns");
  static_assert((KS * FM) % 2 == 0, "the A fragments alternate between two sets across stages");
  using OpA = Operand<BM, false, NW, BK>;
  using OpB = Operand<BN, BKM, NW, BK>;
  constexpr int STAGE_BYTES = OpA::BYTES + OpB::BYTES;
  constexpr int PER_STAGE = OpA::NDMA + OpB::NDMA;
  static_assert(KG * STAGES * STAGE_BYTES <= 160 * 1024, "LDS budget of one workgroup");
  static_assert((KG - 1) * BM * BN * 4 + NW * RowBlock::kBytes <= KG * STAGES * STAGE_BYTES,
                "the groups' sums meet in the rings, the epilogue's scratch behind them");
  __shared__ u32x4_t lds[KG * STAGES * STAGE_BYTES / 16];

  // each XCD takes a contiguous share of the tiles, matrix by matrix
  const int slices = MODE == ORTH_GRAM && KG == 1 ? p.slices : 1;
  const int64_t parts = p.total * slices;
  const int64_t lo = (int64_t)(blockIdx.x & 7) * parts >> 3, hi = (int64_t)((blockIdx.x & 7) + 1) * parts >> 3;
  const int64_t part = lo + (int64_t)(blockIdx.x >> 3);
  if (part >= hi) return;
  const int64_t id = slices == 1 ? part : part / slices;
  OrthCursor<SYM> at;
  at.start(p, id);
  const int mat = at.mat, mt = at.mt, nt = at.nt;
  // the slice's stages
  const int all = p.K / STEP_K, slice = (int)(part - id * slices);
  const int first_stage = slice * all / slices, stages = (slice + 1) * all / slices - first_stage;
  const int m0 = mt * BM, n0 = nt * BN;
  const int m_valid = min(BM, p.M - m0), n_valid = min(BN, p.N - n0);

  const int kg = KG == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / NT);
  const char *ldsc = reinterpret_cast<const char *>(lds) + kg * (STAGES * STAGE_BYTES);
  const int tid = KG == 1 ? threadIdx.x : threadIdx.x % NT;
  const int lane = tid & 63, wave = tid >> 6;
  const int wm = wave / WAVES_N, wn = wave % WAVES_N;
  const int wave_u = __builtin_amdgcn_readfirstlane(wave);

  const half_t *Ab = p.A + mat * p.strideA + (int64_t)m0 * p.lda + first_stage * STEP_K;
  const half_t *Bb = p.B + mat * p.strideB + (BKM ? (int64_t)n0 : (int64_t)n0 * p.ldb + first_stage * STEP_K);
  OpA opa;
  OpB opb;
  opa.init(Ab, p.lda, m_valid, wave, lane, [&](int r) { return r < m_valid ? r : m_valid - 1; });
  opb.init(Bb, p.ldb, n_valid, wave, lane, [&](int r) { return BKM || r < n_valid ? r : n_valid - 1; });
  // the chunks' order is pingpong.h's, whose fragments are these; lo: from a high half to its low one
  auto reorder = [&](auto &op, int valid, bool km, int64_t lo) {
    using Op = std::remove_reference_t<decltype(op)>;
#pragma unroll
    for (int i = 0; i < Op::NDMA; ++i) {
      const int r = (i * NW + wave) * Op::RPI + lane / Op::CPR, phys = lane % Op::CPR;
      if constexpr (BOTH) {
        if (km) {
          if (r & 32) op.ptr[i] += lo;
          op.krow[i] = r & 31;
        } else if ((phys ^ pp_swz(r)) & 4) {
          op.ptr[i] += lo - 32;
        }
      }
      if (km) op.ptr[i] += min((phys ^ pp_swz_km(r)) * 8, valid - 8) - min((phys ^ (4 * (r & 3))) * 8, valid - 8);
      else op.ptr[i] += ((phys ^ pp_swz(r)) - (phys ^ swz(r))) * 8;
    }
  };
  reorder(opa, m_valid, false, p.Alo - p.A);
  reorder(opb, n_valid, BKM, p.Blo - p.B);

  const uint32_t lds0 = (uint32_t)(uintptr_t)ldsc;
  auto issue = [&](int kt) {  // the group's stage kt
    const uint32_t sb = lds0 + (uint32_t)(kt % STAGES * STAGE_BYTES);
    const int ks = kt * KG + kg;
    opa.issue(ks * STEP_K, p.lda, p.K, sb, wave_u);
    opb.issue(ks * STEP_K, p.ldb, p.K, sb + OpA::BYTES, wave_u);
  };
  // 8 consecutive k of row lane & 15 from 8 (lane >> 4) on
  auto rows16 = [&](const char *tile, int rb, int ks) {
    const int r = rb + (lane & 15), c = ks * 4 + (lane >> 4);
    return __builtin_bit_cast(f16x8_t, *reinterpret_cast<const u32x4_t *>(tile + (r * 8 + (c ^ pp_swz(r))) * 16));
  };
  auto cols16 = [&](const char *tile, int cb, int ks) {  // of column lane & 15, k-major
    typedef __attribute__((__vector_size__(8 * sizeof(short)))) short i16x8_t;
    const int b = lane & 15, col = cb + 4 * (b & 3), k_lo = 8 * (lane >> 4) + (b >> 2);
    const char *a = tile + (ks * 32 + k_lo) * OpB::ROWB + ((col >> 3) ^ pp_swz_km(k_lo)) * 16 + ((col >> 2) & 1) * 8;
    const i16x4_t lo = lds_read_tr16(a), hi = lds_read_tr16(a + 4 * OpB::ROWB);
    const i16x8_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    return __builtin_bit_cast(f16x8_t, v);
  };
  auto load_a = [&](int slot, int ks, int i) { return rows16(ldsc + slot * STAGE_BYTES, wm * WM + i * 16, ks); };
  auto load_b = [&](int slot, int ks, int j) {
    const char *tile = ldsc + slot * STAGE_BYTES + OpA::BYTES;
    if constexpr (BKM) return cols16(tile, wn * WN + j * 16, ks);
    else return rows16(tile, wn * WN + j * 16, ks);
  };

  f32x4_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  const int nk = (stages - kg + KG - 1) / KG;  // the group's own
  const int nk_max = (stages + KG - 1) / KG;   // barriers are the workgroup's
  f16x8_t fa[2], fb[2][FN];
  auto mma = [&](int i, int set_a, int set_b) {
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = mfma16(fb[set_b][j], fa[set_a], acc[i][j]);
  };
  // wait until at most `younger` whole stages are still in flight
  auto wait_stages = [&](int younger) {
    static_assert(STAGES <= 8, "one wait for each number of younger stages");
    switch (min(younger, STAGES - 1)) {
      case 7: return wait_vm<(STAGES > 7 ? 7 : 0) * PER_STAGE>();
      case 6: return wait_vm<(STAGES > 6 ? 6 : 0) * PER_STAGE>();
      case 5: return wait_vm<(STAGES > 5 ? 5 : 0) * PER_STAGE>();
      case 4: return wait_vm<(STAGES > 4 ? 4 : 0) * PER_STAGE>();
      case 3: return wait_vm<(STAGES > 3 ? 3 : 0) * PER_STAGE>();
      case 2: return wait_vm<(STAGES > 2 ? 2 : 0) * PER_STAGE>();
      case 1: return wait_vm<PER_STAGE>();
      default: return wait_vm<0>();
    }
  };
  for (int st = 0; st < STAGES; ++st)
    if (st < nk) issue(st);
  wait_stages(min(nk, STAGES) - 1);
  barrier();
  // BOTH: A's low half first, so that the products behind the barrier need the low
  // half of B alone, whose registers the next stage does not fill yet
  auto a_half = [](int g) { return BOTH ? 1 - g / FM : g / FM; };
  fa[0] = load_a(0, a_half(0), 0);
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
        fa[(g + 1) & 1] = load_a(slot, a_half(g + 1), (g + 1) % FM);
        if (i == 0 && ks + 1 < KS) {
#pragma unroll
          for (int j = 0; j < FN; ++j) fb[(ks + 1) & 1][j] = load_b(slot, ks + 1, j);
        }
        mma(i, g & 1, BOTH ? 0 : ks & 1);
        if (BOTH && ks == 1) mma(i, g & 1, 1);
      }
      if constexpr (BOTH) mma(FM - 1, 1, 0);
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
    fa[0] = load_a(nslot, a_half(0), 0);
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[0][j] = load_b(nslot, 0, j);
    if (mine) mma(FM - 1, 1, (KS - 1) & 1);
  }

  __syncthreads();  // every ring is done with
  if constexpr (KG > 1) {
    // the groups' sums, added in the order of the groups by the first one
    f32x4_t *sum = reinterpret_cast<f32x4_t *>(lds);
    auto at = [&](int g, int f) -> f32x4_t & { return sum[(g * FM * FN + f) * NT + tid]; };
    if (kg > 0) {
#pragma unroll
      for (int f = 0; f < FM * FN; ++f) at(kg - 1, f) = acc[f / FN][f % FN];
    }
    __syncthreads();
    if (kg > 0) return;
#pragma unroll
    for (int g = 0; g < KG - 1; ++g)
#pragma unroll
      for (int f = 0; f < FM * FN; ++f) {
        const f32x4_t v = at(g, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[f / FN][f % FN][e] += v[e];
      }
  }
  if (slices > 1) {
#pragma unroll
    for (int f = 0; f < FM * FN; ++f) p.sums[(part * FM * FN + f) * NT + tid] = acc[f / FN][f % FN];
    return;
  }
  // scratch: behind the groups' sums
  char *scr = reinterpret_cast<char *>(lds) + (KG - 1) * BM * BN * 4 + wave * RowBlock::kBytes;
  orth_epilogue<FM, MODE, BOTH>(p, acc, scr, mat, m0, m_valid, wm * WM, n0 + wn * WN, mt != nt);
}

// The slices' sums of a symmetric product's tiles, added in order, to the epilogue, in
// the threads' places that the tiles' kernel has.
template <int BM, int WM, int WN, int MODE, bool BOTH>
__global__ __launch_bounds__((BM / WM) * (BM / WN) * 64, 2) void orth_sum_kernel(OrthTileParams p) {
  constexpr int WAVES_N = BM / WN, NW = BM / WM * WAVES_N, NT = NW * 64, FM = WM / 16, FN = WN / 16;
  __shared__ u32x4_t lds[NW * RowBlock::kBytes / 16];
  const int64_t id = blockIdx.x;
  OrthCursor<true> at;
  at.start(p, id);
  const int m0 = at.mt * BM, n0 = at.nt * BM;
  const int tid = threadIdx.x, wave = tid >> 6, wm = wave / WAVES_N, wn = wave % WAVES_N;
  f32x4_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const f32x4_t *src = p.sums + id * p.slices * FM * FN * NT + tid;
#pragma unroll 2
  for (int s = 0; s < p.slices; ++s) {
#pragma unroll
    for (int f = 0; f < FM * FN; ++f) {
      const f32x4_t v = src[(int64_t)(s * FM * FN + f) * NT];
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[f / FN][f % FN][e] += v[e];
    }
  }
  char *scr = reinterpret_cast<char *>(lds) + wave * RowBlock::kBytes;
  orth_epilogue<FM, MODE, BOTH>(p, acc, scr, at.mat, m0, min(BM, p.M - m0), wm * WM, n0 + wn * WN, at.mt != at.nt);
}

template <int BM, int BN, int WM, int WN, int KG, int STAGES, int MODE, bool BOTH>
hipError_t run_orth_tile(OrthTileParams p, int64_t batch, hipStream_t s) {
  constexpr int NT = KG * (BM / WM) * (BN / WN) * 64;
  p.m_tiles = (p.M + BM - 1) / BM;
  p.n_tiles = (p.N + BN - 1) / BN;
  p.tiles = orth_step(MODE) ? p.m_tiles * p.n_tiles : p.m_tiles * (p.m_tiles + 1) / 2;
  p.total = batch * p.tiles;
  if (MODE != ORTH_GRAM || KG > 1 || p.slices < 1) p.slices = 1;
  const unsigned grid = (unsigned)(ceil_div(p.total * p.slices, 8) * 8);
  orth_tile_kernel<BM, BN, WM, WN, KG, STAGES, MODE, BOTH><<<dim3(grid), NT, 0, s>>>(p);
  return hipGetLastError();
}

// Behind run_orth_tile with slices, on the same tiles.
template <int BM, int WM, int WN, int MODE, bool BOTH>
hipError_t run_orth_sum(OrthTileParams p, int64_t batch, hipStream_t s) {
  p.m_tiles = p.n_tiles = (p.M + BM - 1) / BM;
  p.tiles = p.m_tiles * (p.m_tiles + 1) / 2;
  p.total = batch * p.tiles;
  orth_sum_kernel<BM, WM, WN, MODE, BOTH><<<dim3((unsigned)p.total), (BM / WM) * (BM / WN) * 64, 0, s>>>(p);
  return hipGetLastError();
}

// Large products: 256 x 256 tiles on the main loop of pingpong.h, persistent,
// each XCD walking a contiguous share of the tiles.
template <int MODE>
__global__ __launch_bounds__(kPpThreads, 2) void orth_wide_kernel(OrthTileParams p) {
  __shared__ u32x4_t lds[(kPpLdsBytes + 8 * RowBlock::kBytes) / 16];  // all 160 KB
  const int64_t lo = (int64_t)(blockIdx.x & 7) * p.total >> 3, hi = (int64_t)((blockIdx.x & 7) + 1) * p.total >> 3;
  const int step = gridDim.x >> 3;
  const int64_t first = lo + (blockIdx.x >> 3);
  if (first >= hi) return;
  const int count = (int)((hi - first + step - 1) / step);
  OrthCursor<!orth_step(MODE)> load, put;
  load.start(p, first);
  put = load;
  auto get = [&]() {
    const int m0 = load.mt * kPpTile, n0 = load.nt * kPpTile;
    PpTile t;
    t.A = p.A + load.mat * p.strideA + (int64_t)m0 * p.lda;
    t.B = p.B + load.mat * p.strideB + (orth_step(MODE) ? (int64_t)n0 : (int64_t)n0 * p.ldb);
    t.m_valid = min(kPpTile, p.M - m0);
    t.n_valid = min(kPpTile, p.N - n0);
    load.step(p, step);
    return t;
  };
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  char *scr = reinterpret_cast<char *>(lds) + kPpLdsBytes + wave * RowBlock::kBytes;
  auto done = [&](PpAcc &acc) {
    const int m0 = put.mt * kPpTile;
    const OrthTileParams &p = late_args<OrthTileParams>();
    orth_epilogue<8, MODE>(p, acc, scr, put.mat, m0, min(kPpTile, p.M - m0), (wave >> 2) * 128,
                              put.nt * kPpTile + (wave & 3) * 64, put.mt != put.nt);
    put.step(p, step);
  };
  pp_tiles<true, orth_step(MODE)>(lds, p.lda, p.ldb, p.K / 64, count, get, done);
}

template <int MODE>
hipError_t run_orth_wide(OrthTileParams p, int64_t batch, hipStream_t s) {
  p.m_tiles = (p.M + kPpTile - 1) / kPpTile;
  p.n_tiles = (p.N + kPpTile - 1) / kPpTile;
  p.tiles = orth_step(MODE) ? p.m_tiles * p.n_tiles : p.m_tiles * (p.m_tiles + 1) / 2;
  p.total = batch * p.tiles;
  const int64_t grid = std::min<int64_t>(persistent_grid(), ceil_div(p.total, 8) * 8);
  orth_wide_kernel<MODE><<<dim3((unsigned)grid), kPpThreads, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace moe
