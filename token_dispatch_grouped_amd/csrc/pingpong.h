// The main loop of the large products (256 x 256 tiles of C[m, n] = sum_k
// A(m, k) B(n, k)) in bf16 or fp16: two groups of four wavefronts take turns on
// the matrix cores.
//
// A SIMD holds one wavefront of each group. A group's phase is a memory part
// (DMA and LDS reads) and a compute part (16 MFMAs of 16 x 16 x 32, 256 cycles),
// each ended by the workgroup's barrier; the second group runs one barrier
// behind the first, so that one group computes while the other moves data, and
// the matrix cores change hands instead of waiting for either.
//
// A wavefront owns 128 x 64 of the tile, in four quadrants of 64 x 32; a stage of
// 64 k is four phases:
//   phase   computes   reads from LDS        issues (tile rows by DMA)
//   0       A0 B0      B0 of stage t         A1 of stage t + 1
//   1       A0 B1      B1 of stage t         A0 of stage t + 2
//   2       A1 B1      A1 of stage t         B0 of stage t + 2   (k-major: -)
//   3       A1 B0      A0 of stage t + 1     B1 of stage t + 2   (k-major: B)
// (A k-major as well, AKM: A1 is read in phase 0, A issued in phase 2.)
// A part of a ring slot is read in a phase and refilled from the second phase
// after it on: by then both groups have waited for those reads (at the start of
// their compute parts) and passed a barrier. A part is waited for (vmcnt, every
// wavefront its own) in the memory part before the one that reads it, five
// phases after its issue: 80 KB of a workgroup's loads stay in flight.
//
// Persistent: the stages of a workgroup's tiles form one stream, the first two of
// the next tile being loaded under the last two of this one. The epilogue
// leaves the ring alone; both groups meet in front of it and fall apart again
// behind it.
//
// Measured on 8192^3 bf16 (normal values): 1.55 PFLOP/s (a large library product of
// the same operands in turn 1.59), and 1.38 with MFMAs of
// 32 x 32 x 16, which read and write twice the accumulators for a product: the
// power that they draw bounds the clock (on zeros the same loop reaches 1.7).
#pragma once

#include "gemm_bf16_kernel.h"

namespace moe {

typedef __attribute__((__vector_size__(8 * sizeof(_Float16)))) _Float16 f16x8_t;

constexpr int kPpThreads = 512;
constexpr int kPpTile = 256;
constexpr int kPpLdsBytes = 4 * 32768;  // A slots, then B slots
// Rows and columns that do not exist read zeros, by the buffer's range check:
// no traffic, and matrix cores that multiply zeros draw less of the power that
// bounds the clock. A tile's own offsets stay below 2^27.
constexpr uint32_t kPpRecords = 0x40000000u, kPpOutside = 0x80000000u;

// 16 bytes per lane from rsrc + voff + soff into LDS at lds_addr + 16 lane.
MOE_DEVICE void bdma16s(rsrc_t rsrc, uint32_t voff, uint32_t soff, uint32_t lds_addr) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(lds_addr), "v"(voff), "s"(rsrc),
               "s"(soff)
               : "memory", "m0");
}

// Operands of one output tile. A, B: first row of the tile (k-contiguous) or its
// first column (k-major). AKM: k rows from k_valid on (of this tile's sum) are
// zeros, so that a sum's length need be no multiple of a stage.
struct PpTile {
  const uint16_t *A, *B;
  int m_valid, n_valid;
  int k_valid;
};

// Chunk c (16 bytes) of a k-contiguous row r of 128 bytes sits at c ^ pp_swz(r): a
// b128 read is served in four groups of 16 lanes (0-3 with 12-15 and 20-27, the
// others between them, and so for the upper half), two rows to the 64 banks, and
// with fragments of 16 rows each group finds every bank once. Counted: no
// conflict cycles, one for each active one with (r ^ r / 8) % 8.
MOE_DEVICE int pp_swz(int r) { return (r >> 1) & 7; }
// And of a k-major row r of 128 columns or more at c ^ pp_swz_km(r), so that the
// 16-lane groups of a transposing read, which are 8 rows apart, use different banks.
MOE_DEVICE int pp_swz_km(int r) { return 4 * (r & 3) ^ 2 * ((r >> 3) & 1); }

// MFMA of 16 x 16 x 32 with swapped operands: a lane holds row (lane & 15) of the
// block, 4 consecutive columns from 4 (lane >> 4) on; a fragment, 8 consecutive
// k of row (lane & 15) from 8 (lane >> 4) on.
MOE_DEVICE f32x4_t mfma16(bf16x8_t b, bf16x8_t a, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, a, c, 0, 0, 0);
}
MOE_DEVICE f32x4_t mfma16(f16x8_t b, f16x8_t a, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(b, a, c, 0, 0, 0);
}
// Accumulators of a wavefront's 128 x 64: [row block][column block].
typedef f32x4_t PpAcc[8][4];

// The kernel's one argument, to be read where it is used: an epilogue that names
// the argument itself holds dozens of scalar registers through the main loop.
template <typename P>
MOE_DEVICE const P &late_args() {
  const __attribute__((address_space(4))) void *k =
      (const __attribute__((address_space(4))) void *)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(k));
  return *(const P *)k;
}

// Rows of a wavefront's part of a tile in global memory, 32-bit byte offsets from
// its first element. Rows past the last read zeros and are not written, by the
// buffer's range check. aux 2: non-temporal.
struct TileRows {
  __amdgpu_buffer_rsrc_t r;
  // base: the part's first element; pitch: bytes of a row; rows: that exist
  MOE_DEVICE TileRows(const void *base, int64_t pitch, int rows)
      : r(__builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, rows > 0 ? (int)(rows * pitch) : 0,
                                            0x00020000)) {}
  template <int AUX = 0>
  MOE_DEVICE u32x4_t load(uint32_t off) const {
    return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, AUX));
  }
  template <int AUX = 0>
  MOE_DEVICE void store(uint32_t off, const u32x4_t &v) const {
    typedef uint32_t vec_t __attribute__((ext_vector_type(4)));
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(vec_t, v), r, (int)off, 0, AUX);
  }
};

// 32 rows of 64 16-bit values (or 32 of fp32) in a wavefront's own 4 KB of LDS,
// between whole rows as global memory is read and written (8 lanes of 16 bytes)
// and the accumulators' order.
struct RowBlock {
  static constexpr int kBytes = 4096;
  char *scr;
  int l16, l4;  // the lane's row and column group of an accumulator block
  int rr, rc;   // row (of 8) and 16-byte chunk of a row-wise access
  MOE_DEVICE RowBlock(char *s, int lane) : scr(s), l16(lane & 15), l4(lane >> 4), rr(lane >> 3), rc(lane & 7) {}
  MOE_DEVICE u32x4_t &at16(int r, int c) const {
    return *reinterpret_cast<u32x4_t *>(scr + r * 128 + ((c ^ (r & 7)) * 16));
  }
  // 4 16-bit values of accumulator block (i, j), i of 2 row blocks
  MOE_DEVICE uint2 &at8(int i, int j) const {
    const int r = i * 16 + l16;
    return *reinterpret_cast<uint2 *>(scr + r * 128 + (((j * 2 + (l4 >> 1)) ^ (r & 7)) * 16) + (l4 & 1) * 8);
  }
  // rows g[k] = row k * 8 + rr, chunk rc to f(i, j, the 4 values of block (i, j));
  // H: row blocks of 16, 2 or 1
  template <int H = 2, typename F>
  MOE_DEVICE void in_order(const u32x4_t (&g)[4], F f) const {
#pragma unroll
    for (int k = 0; k < 2 * H; ++k) at16(k * 8 + rr, rc) = g[k];
#pragma unroll
    for (int i = 0; i < H; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) f(i, j, at8(i, j));
  }
  // f(i, j) of every block to rows, put(k, chunk rc of row k * 8 + rr)
  template <int H = 2, typename F, typename Put>
  MOE_DEVICE void rows_out(F f, Put put) const {
#pragma unroll
    for (int i = 0; i < H; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) at8(i, j) = f(i, j);
#pragma unroll
    for (int k = 0; k < 2 * H; ++k) put(k, at16(k * 8 + rr, rc));
  }
};

// A place in the order of the tiles of a product: groups of kGroupM row tiles,
// column tile outer, so that the tiles an XCD works on share operands.
struct PpCursor {
  int mt, nt;      // row tile, column tile
  int base, rows;  // the group's first row tile, its row tiles

  MOE_DEVICE void start(int m_tiles, int n_tiles, int t) {
    base = __builtin_amdgcn_readfirstlane(t / (kGroupM * n_tiles) * kGroupM);
    rows = min(kGroupM, m_tiles - base);
    const int rem = t - base * n_tiles;
    nt = __builtin_amdgcn_readfirstlane(rem / rows);
    mt = base + rem - nt * rows;
  }
  // n places on; how often it began again behind the last
  MOE_DEVICE int step(int m_tiles, int n_tiles, int n) {
    int again = 0;
    mt += n;
    while (mt >= base + rows) {
      mt -= rows;
      if (++nt < n_tiles) continue;
      nt = 0;
      mt += rows;  // into the next group
      base += rows;
      if (base == m_tiles) {
        mt -= base;
        base = 0;
        ++again;
      }
      rows = min(kGroupM, m_tiles - base);
    }
    return again;
  }
};

// count: the workgroup's tiles; nk: stages of 64 k, the same for all of them.
// get(): the next tile to load, asked for once each; done(acc): the epilogue of
// the next tile, in the same order: a wavefront's acc is rows from 128 group,
// columns from 64 (wave & 3) on. AKM: row block i of either half is rows from 16
// (i ^ (wave & 3)) of it on, so that block 0 is another one in each of the four
// wavefronts that hold the same rows; stage(a0, a1), once a stage, is given the
// fragments of block 0 of both halves.
template <bool F16, bool AKM, bool BKM, typename Get, typename Done, typename Stage>
MOE_DEVICE void pp_tiles(u32x4_t *lds, int64_t lda, int64_t ldb, int nk, int count, Get get, Done done, Stage stage) {
  static_assert(!AKM || BKM, "no product has A alone k-major");
  if (count <= 0) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int grp = wave >> 2, wn = wave & 3;
  const int l16 = lane & 15, l4 = lane >> 4;
  const char *ldsc = reinterpret_cast<const char *>(lds);
  const uint32_t lds0 = (uint32_t)(uintptr_t)ldsc;

  // Fragment addresses, without slot (bit 15) and row block. k-contiguous: per k
  // step, chunk c of row r at c ^ pp_swz(r), which no row block of 16 changes.
  uint32_t la[2][2], lb[2][2];
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
    const uint32_t a = (uint32_t)(l16 * 128 + (((ks * 4 + l4) ^ pp_swz(l16)) * 16));
    la[0][ks] = a + (uint32_t)grp * 16384u;
    lb[0][ks] = a + 65536u + (uint32_t)wn * 8192u;
  }
  // k-major: of the 16 columns from `first` on
  auto km_addr = [&](int first) {
    const int col = first + 4 * (l16 & 3);
    const int k_lo = 8 * l4 + (l16 >> 2);
    const int c = (col >> 3) ^ pp_swz_km(k_lo);
    return (uint32_t)(k_lo * 512 + c * 16 + ((col >> 2) & 1) * 8);
  };
  if constexpr (BKM) {  // lb[j][x]: column block 2j + x
#pragma unroll
    for (int q = 0; q < 4; ++q) lb[q >> 1][q & 1] = 65536u + km_addr(wn * 64 + q * 16);
  }
  // AKM: la[x][y]: column block 2x + y of either half (64 columns apart: bit 3 of
  // the chunk, which the swizzle may flip: 128 bytes up or down)
  int la_half = 0;
  if constexpr (AKM) {
#pragma unroll
    for (int q = 0; q < 4; ++q) la[q >> 1][q & 1] = km_addr(grp * 128 + (q ^ wn) * 16);
    la_half = (int)(km_addr(grp * 128 + 64) - km_addr(grp * 128));
  }
  typedef typename std::conditional<F16, f16x8_t, bf16x8_t>::type frag_t;
  frag_t fa[2][4][2], fb[2][2][2];  // [half][row block][k step]
  auto read_km = [&](const char *a) {
    typedef __attribute__((__vector_size__(8 * sizeof(short)))) short i16x8_t;
    const i16x4_t lo = lds_read_tr16(a), hi = lds_read_tr16(a + 2048);
    const i16x8_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    return __builtin_bit_cast(frag_t, v);
  };
  auto read_a = [&](int h) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        if constexpr (AKM)
          fa[h][i][ks] = read_km(ldsc + (la[i >> 1][i & 1] + (uint32_t)(h ? la_half : 0)) + ks * 16384);
        else
          fa[h][i][ks] = __builtin_bit_cast(
              frag_t, *reinterpret_cast<const u32x4_t *>(ldsc + la[0][ks] + (h * 64 + i * 16) * 128));
      }
  };
  auto read_b = [&](int j) {
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        if constexpr (BKM) {
          fb[j][x][ks] = read_km(ldsc + lb[j][x] + ks * 16384);
        } else {
          fb[j][x][ks] = __builtin_bit_cast(
              frag_t, *reinterpret_cast<const u32x4_t *>(ldsc + lb[0][ks] + (j * 32 + x * 16) * 128));
        }
      }
  };

  // The loading side: stage lk of tile lt into slot ls (a byte offset), a
  // wavefront 8 rows a load.
  uint32_t va[4], vb[4];  // byte offsets: A0 of either group, A1; B0, B0, B1, B1 (k-major: one)
  rsrc_t ra, rb;
  const uint16_t *aptr = nullptr, *bptr = nullptr;
  int k_valid = 0;
  const int qb = (wave & 3) + 8 * (wave >> 2);
  // k-major: the lane's 16 bytes of k row wave * 2 + lane / 32 of a stage; row i *
  // 16 + that one has the same swizzle (bit 3 of it is wave / 4)
  auto km_off = [&](int64_t ld, int valid) {
    const int r = wave * 2 + (lane >> 5);
    const int col = ((lane & 31) ^ pp_swz_km(r)) * 8;
    return col < valid ? (uint32_t)(((int64_t)r * ld + col) * 2) : kPpOutside;
  };
  auto aim = [&](const PpTile &t) {
    const int l8 = lane >> 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (!AKM) {
        const int r = wave * 8 + l8 + (i & 1) * 128 + (i >> 1) * 64;
        va[i] = r < t.m_valid ? (uint32_t)((int64_t)r * lda * 2) + (uint32_t)(((lane & 7) ^ pp_swz(r)) * 16) : kPpOutside;
      }
      if constexpr (!BKM) {
        const int s = (qb + (i & 1) * 16 + (i >> 1) * 4) * 8 + l8;
        vb[i] = s < t.n_valid ? (uint32_t)((int64_t)s * ldb * 2) + (uint32_t)(((lane & 7) ^ pp_swz(s)) * 16) : kPpOutside;
      }
    }
    if constexpr (AKM) va[0] = km_off(lda, t.m_valid);
    if constexpr (BKM) vb[0] = km_off(ldb, t.n_valid);
    aptr = t.A;
    bptr = t.B;
    k_valid = t.k_valid;
    if constexpr (!AKM) ra = make_rsrc(t.A, kPpRecords);
    if constexpr (!BKM) rb = make_rsrc(t.B, kPpRecords);
  };
  int left = count - 1, lk = 0;  // tiles not asked for yet; the stage
  uint32_t ls = 0;
  auto issue_a = [&](int h) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      bdma16s(ra, va[h * 2 + i], (uint32_t)lk * 128u, lds0 + ls + (uint32_t)((wave * 8 + i * 128 + h * 64) * 128));
  };
  auto issue_b = [&](int j) {  // k-contiguous
#pragma unroll
    for (int i = 0; i < 2; ++i)
      bdma16s(rb, vb[j * 2 + i], (uint32_t)lk * 128u, lds0 + 65536u + ls + (uint32_t)((qb + i * 16 + j * 4) * 1024));
  };
  // a whole k-major stage, rows past the sum's end by the range check: a lane
  // offset below kPpOutside is in row floor(offset / pitch)
  auto issue_km = [&](const uint16_t *ptr, int64_t ld, uint32_t voff, uint32_t dst) {
    uint32_t records = kPpRecords;
    if constexpr (AKM) records = (uint32_t)max(0, min(64, k_valid - lk * 64)) * (uint32_t)(ld * 2);
    const rsrc_t r = make_rsrc(ptr + (int64_t)lk * 64 * ld, records);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // the row part in the lane's offset, which the range check surely sees
      const uint32_t v = AKM ? voff + (uint32_t)(i * 32 * ld) : voff;
      bdma16s(r, v, AKM ? 0u : (uint32_t)(i * 32 * ld), dst + (uint32_t)((i * 8 + wave) * 1024));
    }
  };
  auto issue_ak = [&]() { issue_km(aptr, lda, va[0], lds0 + ls); };
  auto issue_bk = [&]() { issue_km(bptr, ldb, vb[0], lds0 + 65536u + ls); };
  auto advance = [&]() {
    ls ^= 32768u;
    if (++lk < nk) return;
    if (left > 0) {
      --left;
      lk = 0;
      aim(get());
    } else {
      lk = nk - 1;  // past the last stage: any valid load keeps the counts
    }
  };

  PpAcc acc;
  auto mma = [&](int h, int j) {
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int x = 0; x < 2; ++x) acc[h * 4 + i][j * 2 + x] = mfma16(fb[j][x][ks], fa[h][i][ks], acc[h * 4 + i][j * 2 + x]);
    __builtin_amdgcn_s_setprio(0);
  };
  auto turn = [&]() {  // memory part -> compute part
    __builtin_amdgcn_sched_barrier(0);
    barrier();
    wait_lds();
    __builtin_amdgcn_sched_barrier(0);
  };
  auto end = [&]() {  // compute part -> memory part
    __builtin_amdgcn_sched_barrier(0);
    barrier();
    __builtin_amdgcn_sched_barrier(0);
  };

  aim(get());
  if constexpr (AKM) {
    issue_ak();
    issue_bk();
    advance();
    issue_ak();
    issue_bk();
    wait_vm<8>();  // the first stage
  } else {
    issue_a(0);
    if constexpr (BKM) {
      issue_bk();
    } else {
      issue_b(0);
      issue_b(1);
    }
    issue_a(1);
    advance();
    issue_a(0);
    if constexpr (BKM) {
      issue_bk();
      wait_vm<8>();  // A0 and B of the first stage
    } else {
      issue_b(0);
      issue_b(1);
      wait_vm<10>();  // A0 and B0 of the first stage
    }
  }
  barrier();

  for (int ti = 0; ti < count; ++ti) {
    // read here and not in phase 3 of the tile before, so that the epilogue has
    // those registers; waited for, as the part is refilled two barriers on
    read_a(0);
    wait_lds();
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    if (grp == 1) barrier();
    for (int kt = 0; kt < nk; ++kt) {
      read_b(0);
      if constexpr (AKM) read_a(1);
      else issue_a(1);
      if (!BKM) wait_vm<10>();  // B1 of this stage
      turn();
      mma(0, 0);
      end();

      read_b(1);
      advance();
      if constexpr (!AKM) {
        issue_a(0);
        wait_vm<10>();  // A1 of this stage
      }
      turn();
      mma(0, 1);
      if constexpr (AKM) stage(fa[0][0], fa[1][0]);
      end();

      if constexpr (AKM) {
        issue_ak();
        wait_vm<8>();  // A of the next stage: only its B and this A are younger
      } else {
        read_a(1);
        if (!BKM) issue_b(0);
        wait_vm<BKM ? 8 : 10>();  // A0 of the next stage
      }
      turn();
      mma(1, 1);
      end();

#pragma unroll
      for (int q = 0; q < (AKM ? 4 : 2); ++q) la[q >> 1][q & 1] ^= 32768u;
      if (kt + 1 < nk) read_a(0);
      if constexpr (BKM) {
        issue_bk();
        wait_vm<8>();  // B of the next stage
      } else {
        issue_b(1);
        wait_vm<10>();  // B0 of the next stage
      }
      turn();
      mma(1, 0);
#pragma unroll
      for (int q = 0; q < (BKM ? 4 : 2); ++q) lb[q >> 1][q & 1] ^= 32768u;
      end();
    }
    if (grp == 0) barrier();
    done(acc);
  }
  wait_vm<0>();  // no load may land in the next workgroup's LDS
}

template <bool F16, bool BKM, typename Get, typename Done>
MOE_DEVICE void pp_tiles(u32x4_t *lds, int64_t lda, int64_t ldb, int nk, int count, Get get, Done done) {
  pp_tiles<F16, false, BKM>(lds, lda, ldb, nk, count, get, done, 0);
}

}  // namespace moe
