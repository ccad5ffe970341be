// The dense gated feed-forward block's products on the gfx950 matrix cores:
// C[m, n] = sum_k A(m, k) B(n, k), one group of rows, no routing tables.
//
//   gate/up   [hg | hu] = X W_gu^T, a = silu(hg) hu     A = x [T,d]    B = w_gu [2F,d]
//   down      y  = a W_down^T + add                     A = a [T,F]    B = w_down [d,F]
//   dgrad     da = dy W_down -> dh                      A = dy [T,d]   B k-major = w_down
//             dx = dh W_gu + add                        A = dh [T,2F]  B k-major = w_gu
//
// Elements are bf16, or the 8-bit block form (F8), whose scales go into the
// scaled MFMA. A stage is 128 bytes of k of every tile row (64 bf16 or 128
// e4m3 values) in an LDS ring of STAGES slots filled by the LDS DMA, with the operand
// layout, swizzle and fragment reads of the grouped products (Operand): an
// e4m3 row is moved as a bf16 row of half its length. The scales of a stage
// are one dword per tile row (4 blocks of 32), a 4-byte DMA of each thread.
//
// With few tiles, KG groups of wavefronts share a tile's stages out among
// them, each in a ring of its own, and add their sums at the end: more
// wavefronts to hide the latency of a stage, and fewer stages in a row.
//
// Within a stage the wavefront walks (k step, row block) groups: FN MFMAs on
// one A fragment while the next A fragment (and, once per k step, the next
// step's B fragments) is read, so only two A and two sets of B fragments
// are held beside the accumulators.
//
// Measured (256 x 256 tiles, d = 4096, F = 2816, 8192 tokens, 8-bit): gate/up
// 188 us (2.0 PFLOP/s), down 96 us (2.0 PFLOP/s). Bound by moving the operands:
// a 64 KB stage takes 1.85 us of a CU, in bf16 and in 8 bits alike.
//
// The 8-bit products: the matrix core adds the 32 products of a block aligned
// to the largest of them and cuts off what lies below 2^-13 of it; sums over
// blocks are fp32.
//
// The MFMA is issued with its operands swapped: a lane holds 4 consecutive
// columns of one row, its partner lane (+ 32) the next 4; v_permlane32_swap
// turns two such groups into 16-byte chunks, so the epilogues read and write
// global memory straight from registers.
#pragma once

#include "gemm_bf16_kernel.h"
#include "mx8.h"

namespace moe {

enum { FFN_SWIGLU_FWD = 0, FFN_STORE = 1, FFN_SWIGLU_BWD = 2 };

struct FfnTileParams {
  const bf16_t *A, *B;         // F8: e4m3 bytes; lda, ldb count pairs of them
  const uint8_t *As, *Bs;      // F8: scales [rows, K / 32]
  bf16_t *C;                   // STORE: the output; SWIGLU_FWD: h or NULL; SWIGLU_BWD: dh
  bf16_t *C2;                  // SWIGLU_FWD: a (bf16, or e4m3 bytes when C2s is given)
  uint8_t *C2s;                // SWIGLU_FWD, F8: scales of a
  float *a32;                  // SWIGLU_FWD, F8, few tokens: a in fp32
  const bf16_t *H;             // SWIGLU_BWD: saved h
  const bf16_t *add;           // STORE: [M, N] added before the rounding, or NULL; may be C
  int M, N, K;                 // N: columns of C (SWIGLU: F); K: 16-bit units of a row
  int64_t lda, ldb, ldc;
  int F;
  int n_tiles, m_tiles;
};

typedef __attribute__((__vector_size__(8 * sizeof(int)))) int i32x8_t;

// vdst's upper lanes trade places with vsrc's lower ones.
MOE_DEVICE void swap32(uint32_t &a, uint32_t &b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}

// 4 bytes per lane from global `g` into LDS at `lds_addr` + 4 * lane.
MOE_DEVICE void dma4(const void *g, uint32_t lds_addr) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dword %1, off" ::"s"(lds_addr), "v"(g) : "memory", "m0");
}

// Fragment of one MFMA: 16 k values of bf16, or 64 of e4m3 (two blocks of 32
// with their scales), 8 or 32 of them in a lane.
template <bool F8>
struct FfnFrag {
  typedef bf16x8_t type;
};
template <>
struct FfnFrag<true> {
  typedef i32x8_t type;
};

template <bool F8, int BM, int BN, int WM, int WN, int KG, int STAGES, bool BKM, int EPI>
__global__ __launch_bounds__(KG * (BM / WM) * (BN / WN) * 64, 2) void ffn_tile_kernel(FfnTileParams p) {
  constexpr int WAVES_M = BM / WM, WAVES_N = BN / WN, NW = WAVES_M * WAVES_N, NT = NW * 64;  // of a k group
  constexpr int FM = WM / 32, FN = WN / 32;
  constexpr int BK = 64;               // 16-bit units of k per stage
  constexpr int KS = F8 ? 2 : 4;       // k steps per stage
  static_assert(!F8 || (BM + BN <= NT && !BKM), "one scale dword per thread and stage");
  static_assert(EPI != FFN_SWIGLU_FWD || FN % 2 == 0, "gate/up pairs need an even fragment count");
  static_assert((KS * FM) % 2 == 0, "the A fragments alternate between two sets across stages");
  using OpA = Operand<BM, false, NW, BK>;
  using OpB = Operand<BN, BKM, NW, BK>;
  constexpr int SCALE_BYTES = F8 ? NT * 4 : 0;
  constexpr int STAGE_BYTES = OpA::BYTES + OpB::BYTES + SCALE_BYTES;
  constexpr int PER_STAGE = OpA::NDMA + OpB::NDMA + (F8 ? 1 : 0);
  static_assert(KG * STAGES * STAGE_BYTES <= 160 * 1024, "LDS budget of one workgroup");
  static_assert((KG - 1) * BM * BN * 4 <= KG * STAGES * STAGE_BYTES, "the groups' sums meet in the rings");
  __shared__ u32x4_t lds[KG * STAGES * STAGE_BYTES / 16];

  // each XCD takes a contiguous share of the tiles: groups of kGroupM row
  // tiles (the last one of fewer, so that all XCDs have as many tiles: 700
  // tokens, 2048 x 1408, 40 -> 28 us), column tile outer, so its resident
  // workgroups share operands
  const int per = kGroupM * p.n_tiles;
  int lo, hi;
  xcd_range(blockIdx.x & 7, (int64_t)p.m_tiles * p.n_tiles, lo, hi);
  const int id = lo + (int)(blockIdx.x >> 3);
  if (id >= hi) return;
  const int grp = id / per, rem = id - grp * per;
  const int rows = min(kGroupM, p.m_tiles - grp * kGroupM);
  const int n_tile = rem / rows;
  const int m0 = (grp * kGroupM + (rem - n_tile * rows)) * BM;
  const int m_valid = min(BM, p.M - m0);

  // group kg of NW wavefronts computes the whole tile over its share of the
  // stages (kg, kg + KG, ...) in a ring of its own
  const int kg = KG == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / NT);
  const char *ldsc = reinterpret_cast<const char *>(lds) + kg * (STAGES * STAGE_BYTES);
  const int tid = KG == 1 ? threadIdx.x : threadIdx.x % NT;
  const int lane = tid & 63, wave = tid >> 6;
  const int wm = wave / WAVES_N, wn = wave % WAVES_N;
  const int l32 = lane & 31, lhi = lane >> 5;
  const int wave_u = __builtin_amdgcn_readfirstlane(wave);

  // B rows of a gate/up tile interleave gate and up rows per wavefront column
  auto b_row = [&](int r) {
    if (EPI == FFN_SWIGLU_FWD) {
      const int wcol = r / WN, q = r % WN;
      const int gi = n_tile * (BN / 2) + wcol * (WN / 2) + q % (WN / 2);
      const int gc = gi < p.N ? gi : p.N - 1;  // past-the-end columns are masked on output
      return q < WN / 2 ? gc : p.F + gc;
    }
    const int c = n_tile * BN + r;
    return c < p.N ? c : p.N - 1;
  };
  OpA opa;
  OpB opb;
  opa.init(p.A + (int64_t)m0 * p.lda, p.lda, m_valid, wave, lane, [&](int r) { return r < m_valid ? r : m_valid - 1; });
  if (BKM) opb.init(p.B + n_tile * BN, p.ldb, p.N - n_tile * BN, wave, lane, [](int r) { return r; });
  else opb.init(p.B, p.ldb, p.N, wave, lane, b_row);
  const uint8_t *sptr = nullptr;  // F8: this thread's row of scales
  if (F8) {
    const int64_t sld = p.K / 16;  // K 16-bit units are 2K values, 2K / 32 blocks
    const int t = tid < BM + BN ? tid : BM + BN - 1;  // any threads beyond repeat the last row's
    sptr = t < BM ? p.As + (int64_t)(m0 + (t < m_valid ? t : m_valid - 1)) * sld : p.Bs + (int64_t)b_row(t - BM) * sld;
  }

  const uint32_t lds0 = (uint32_t)(uintptr_t)ldsc;
  auto issue = [&](int kt) {  // the group's stage kt
    const uint32_t sb = lds0 + (uint32_t)(kt % STAGES * STAGE_BYTES);
    const int ks = kt * KG + kg;
    opa.issue(ks * BK, p.lda, p.K, sb, wave_u);
    opb.issue(ks * BK, p.ldb, p.K, sb + OpA::BYTES, wave_u);
    if (F8) dma4(sptr + ks * 4, sb + OpA::BYTES + OpB::BYTES + (uint32_t)(wave_u * 256));
  };

  typedef typename FfnFrag<F8>::type frag_t;
  auto load8 = [&](const char *tile, int rb, int ks) -> i32x8_t {
    // the scaled MFMA's k order: a lane half's first 16 bytes are the half-th
    // 16 of block 0, its last 16 those of block 1, and it is the lower half
    // that names block 0's scale, the upper one block 1's
    const int r = rb + l32, c = ks * 4 + lhi, z = kc_swz<8>(r);
    const u32x4_t a = *reinterpret_cast<const u32x4_t *>(tile + (r * 8 + (c ^ z)) * 16);
    const u32x4_t b = *reinterpret_cast<const u32x4_t *>(tile + (r * 8 + ((c + 2) ^ z)) * 16);
    return i32x8_t{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
  };
  auto load_a = [&](int slot, int ks, int i) -> frag_t {
    const char *t = ldsc + slot * STAGE_BYTES;
    if constexpr (F8) return load8(t, wm * WM + i * 32, ks);
    else return opa.frag(t, wm * WM + i * 32, ks, lane);
  };
  auto load_b = [&](int slot, int ks, int j) -> frag_t {
    const char *t = ldsc + slot * STAGE_BYTES + OpA::BYTES;
    if constexpr (F8) return load8(t, wn * WN + j * 32, ks);
    else return opb.frag(t, wn * WN + j * 32, ks, lane);
  };
  // byte b of a scale dword is block b of the stage; a lane's half owns bytes
  // lhi and lhi + 2, which a shift brings to bytes 0 and 2
  auto load_scale = [&](int slot, int row) -> int {
    const char *t = ldsc + slot * STAGE_BYTES + OpA::BYTES + OpB::BYTES;
    return (int)(*reinterpret_cast<const uint32_t *>(t + row * 4) >> (8 * lhi));
  };

  f32x16_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

  const int stages = p.K / BK;                       // K is a multiple of BK
  const int nk = (stages - kg + KG - 1) / KG;        // the group's own
  const int nk_max = (stages + KG - 1) / KG;         // barriers are the workgroup's
  frag_t fa[2], fb[2][FN];
  int sa[FM], sb[FN];
  (void)sa;
  (void)sb;
  auto mma = [&](int i, int set_a, int set_b, int ks) {
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      if constexpr (F8) {
        if (ks == 0)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[set_b][j], fa[set_a], acc[i][j], 0, 0, 0,
                                                                      sb[j], 0, sa[i]);
        else
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[set_b][j], fa[set_a], acc[i][j], 0, 0, 2,
                                                                      sb[j], 2, sa[i]);
      } else {
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[set_b][j], fa[set_a], acc[i][j], 0, 0, 0);
      }
    }
  };

  // wait until at most `younger` whole stages are still in flight
  auto wait_stages = [&](int younger) {
    if (STAGES > 4 && younger >= 4) wait_vm<4 * PER_STAGE>();
    else if (STAGES > 3 && younger >= 3) wait_vm<3 * PER_STAGE>();
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
  if (F8) {
#pragma unroll
    for (int i = 0; i < FM; ++i) sa[i] = load_scale(0, wm * WM + i * 32 + l32);
#pragma unroll
    for (int j = 0; j < FN; ++j) sb[j] = load_scale(0, BM + wn * WN + j * 32 + l32);
  }

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
      mma(i, g & 1, ks & 1, ks);
      if (F8) __builtin_amdgcn_sched_barrier(0);  // reads run one group ahead, not more
    }
    }
    // every fragment of this stage is in registers: its slot takes stage
    // kt + STAGES once all wavefronts are here, and stage kt + 1 has landed
    if constexpr (F8) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) asm volatile("" : "+v"(acc[i][j]));  // no product sinks below the branch
    }
    __builtin_amdgcn_sched_barrier(0);
    wait_lds();
    wait_stages(min(STAGES - 2, nk - 2 - kt));  // issued so far: up to stage min(kt + STAGES, nk) - 1
    barrier();
    if (kt + STAGES < nk) issue(kt + STAGES);
    // the first fragments of the next stage (on the last pass a harmless
    // read of a stale slot)
    const int nslot = (kt + 1) % STAGES;
    fa[0] = load_a(nslot, 0, 0);
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[0][j] = load_b(nslot, 0, j);
    int nsa[FM], nsb[FN];
    if (F8) {
#pragma unroll
      for (int i = 0; i < FM; ++i) nsa[i] = load_scale(nslot, wm * WM + i * 32 + l32);
#pragma unroll
      for (int j = 0; j < FN; ++j) nsb[j] = load_scale(nslot, BM + wn * WN + j * 32 + l32);
    }
    if (mine) mma(FM - 1, 1, (KS - 1) & 1, KS - 1);
    if (F8) {
#pragma unroll
      for (int i = 0; i < FM; ++i) sa[i] = nsa[i];
#pragma unroll
      for (int j = 0; j < FN; ++j) sb[j] = nsb[j];
    }
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
    uint32_t e0 = pack_bf2(v[0], v[1]), e1 = pack_bf2(v[2], v[3]);
    uint32_t o0 = pack_bf2(v[4], v[5]), o1 = pack_bf2(v[6], v[7]);
    swap32(e0, o0);
    swap32(e1, o1);
    return u32x4_t{e0, e1, o0, o1};
  };
  auto unpack_chunk = [&](const u32x4_t &c, float *v) {  // the inverse
    uint32_t e0 = c[0], e1 = c[1], o0 = c[2], o1 = c[3];
    swap32(e0, o0);
    swap32(e1, o1);
    const u32x4_t w = {e0, e1, o0, o1};
    Elem<bf16_t>::unpack(w, v);
  };
  int el32 = l32, ehi = lhi;
  // opaque: no address below is formed above the main loop and held there
  asm volatile("" : "+v"(el32), "+v"(ehi));
  const int row_l = wm * WM + el32;
  if constexpr (EPI == FFN_STORE) {
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int r = row_l + i * 32;
      const bool rok = r < m_valid;
      const int64_t ro = (int64_t)(m0 + (rok ? r : 0)) * p.ldc;
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int gp = 0; gp < 2; ++gp) {
          const int c = n_tile * BN + wn * WN + j * 32 + 16 * gp + 8 * ehi;
          const bool ok = rok && c < p.N;
          float v[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) v[q] = acc[i][j][8 * gp + q];
          if (p.add) {
            float b[8];
            unpack_chunk(ok ? ld16(p.add + ro + c) : u32x4_t{0u, 0u, 0u, 0u}, b);
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] += b[q];
          }
          const u32x4_t o = pack_chunk(v);
          if (ok) st16(p.C + ro + c, o);
        }
    }
  } else if constexpr (EPI == FFN_SWIGLU_FWD) {
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int r = row_l + i * 32;
      const bool rok = r < m_valid;
      const int64_t row = m0 + (rok ? r : 0);
#pragma unroll
      for (int j = 0; j < FN / 2; ++j) {
        const f32x16_t &ga = acc[i][j];
        const f32x16_t &ua = acc[i][j + FN / 2];
        const int c0 = n_tile * (BN / 2) + wn * (WN / 2) + j * 32;
        if (p.C) {
#pragma unroll
          for (int gp = 0; gp < 2; ++gp) {
            const int c = c0 + 16 * gp + 8 * ehi;
            float gv[8], uv[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              gv[q] = ga[8 * gp + q];
              uv[q] = ua[8 * gp + q];
            }
            const u32x4_t og = pack_chunk(gv), ou = pack_chunk(uv);
            if (rok && c < p.N) {
              st16(p.C + row * p.ldc + c, og);
              st16(p.C + row * p.ldc + p.F + c, ou);
            }
          }
        }
        float a[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) a[q] = silu_f(ga[q]) * ua[q];
        if constexpr (F8) {
          // the block is this fragment's 32 columns of the row: 16 here, 16
          // in the partner lane
          uint32_t m = 0;
#pragma unroll
          for (int q = 0; q < 16; ++q) m = umax(m, abs_bits(a[q]));
          uint32_t m2 = m;
          swap32(m, m2);  // m = this half's lower lanes, m2 = the upper ones', in both halves
          m = umax(m, m2);
          const uint32_t code = mx8_scale_code(m);
          const float inv = mx8_inv_scale(code);
          uint32_t w[4];
#pragma unroll
          for (int g = 0; g < 4; ++g)
            w[g] = mx8_pack4(a[4 * g] * inv, a[4 * g + 1] * inv, a[4 * g + 2] * inv, a[4 * g + 3] * inv);
          swap32(w[0], w[2]);  // dwords 0 and 1 of the row's 8 (4 and 5 in the upper half)
          swap32(w[1], w[3]);  // dwords 2 and 3 (6 and 7)
          if (rok && c0 < p.N) {
            uint8_t *a8 = reinterpret_cast<uint8_t *>(p.C2) + row * p.F + c0 + 16 * ehi;
            st16(a8, u32x4_t{w[0], w[2], w[1], w[3]});
            if (ehi == 0) p.C2s[row * (p.F / kMx8Block) + c0 / kMx8Block] = (uint8_t)code;
          }
        } else {
#pragma unroll
          for (int gp = 0; gp < 2; ++gp) {
            const int c = c0 + 16 * gp + 8 * ehi;
            const u32x4_t o = pack_chunk(a + 8 * gp);
            if (rok && c < p.N) st16(p.C2 + row * p.F + c, o);
          }
        }
      }
    }
  } else {  // FFN_SWIGLU_BWD
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int r = row_l + i * 32;
      const bool rok = r < m_valid;
      const int64_t ro = (int64_t)(m0 + (rok ? r : 0)) * p.ldc;
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int gp = 0; gp < 2; ++gp) {
          const int c = n_tile * BN + wn * WN + j * 32 + 16 * gp + 8 * ehi;
          const bool ok = rok && c < p.N;
          const int cc = ok ? c : 0;
          float hg[8], hu[8], dg[8], du[8];
          unpack_chunk(ld16(p.H + ro + cc), hg);
          unpack_chunk(ld16(p.H + ro + p.F + cc), hu);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            // t = dA s, dH_up = t hg, dH_gate = t hu (1 + hg (1 - s))
            const float s = sigmoid_f(hg[q]);
            const float t = acc[i][j][8 * gp + q] * s;
            const float th = t * hu[q];
            du[q] = t * hg[q];
            dg[q] = fmaf(th, fmaf(-hg[q], s, hg[q]), th);
          }
          const u32x4_t og = pack_chunk(dg), ou = pack_chunk(du);
          if (ok) {
            st16(p.C + ro + c, og);
            st16(p.C + ro + p.F + c, ou);
          }
        }
    }
  }
}

template <bool F8, int BM, int BN, int WM, int WN, int KG, int STAGES, bool BKM, int EPI>
hipError_t run_ffn_tile(FfnTileParams p, hipStream_t s) {
  constexpr int NT = KG * (BM / WM) * (BN / WN) * 64;
  p.m_tiles = (p.M + BM - 1) / BM;
  p.n_tiles = EPI == FFN_SWIGLU_FWD ? (p.N + BN / 2 - 1) / (BN / 2) : (p.N + BN - 1) / BN;
  const int64_t total = (int64_t)p.m_tiles * p.n_tiles;
  const unsigned grid = (unsigned)(ceil_div(total, 8) * 8);
  ffn_tile_kernel<F8, BM, BN, WM, WN, KG, STAGES, BKM, EPI><<<dim3(grid), NT, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace moe
