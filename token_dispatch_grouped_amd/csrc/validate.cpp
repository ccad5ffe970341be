// Host-side validation of every C-ABI argument, done before anything is
// launched. Unsupported configurations are rejected explicitly and up front
// (Support combined expert and data parallelism in TrainerRank, Current
// behavior and Desired behavior), and every argument is checked before any
// is consumed (review note on Add MoE expert parallel training runtime).
#include "validate.h"

#include <algorithm>
#include <cmath>

#include <stdio.h>

namespace moe {

static moe_status fail(std::string *why, moe_status st, const char *msg) {
  if (why) *why = msg;
  return st;
}

moe_status validate_shape(const moe_shape *s, std::string *why) {
  if (!s) return fail(why, MOE_ERR_INVALID_ARGUMENT, "shape is NULL");
  if (s->T < 0) return fail(why, MOE_ERR_INVALID_ARGUMENT, "T < 0");
  if (s->d <= 0 || s->E <= 0 || s->k <= 0 || s->F <= 0)
    return fail(why, MOE_ERR_INVALID_ARGUMENT, "d, E, k and F must be positive");
  if (s->k > s->E) return fail(why, MOE_ERR_INVALID_ARGUMENT, "k > E");
  if (s->dtype != MOE_DTYPE_F32 && s->dtype != MOE_DTYPE_BF16)
    return fail(why, MOE_ERR_UNSUPPORTED, "dtype must be MOE_DTYPE_F32 or MOE_DTYPE_BF16");
  if (s->flags & ~(uint32_t)(MOE_FLAG_RENORM | MOE_FLAG_RECOMPUTE | MOE_FLAG_ACCUMULATE_DLOGITS))
    return fail(why, MOE_ERR_UNSUPPORTED, "unknown flag bits");
  if (s->E > 256) return fail(why, MOE_ERR_UNSUPPORTED, "E > 256");
  if (s->k > 16) return fail(why, MOE_ERR_UNSUPPORTED, "k > 16");
  if (s->d % 64 != 0 || s->F % 64 != 0) return fail(why, MOE_ERR_UNSUPPORTED, "d and F must be multiples of 64");
  if (s->d > 65536 || s->F > 65536) return fail(why, MOE_ERR_UNSUPPORTED, "d or F > 65536");
  const int64_t R = s->T * (int64_t)s->k;
  if (s->T > ((int64_t)1 << 31) || R >= ((int64_t)1 << 31)) return fail(why, MOE_ERR_UNSUPPORTED, "T*k >= 2^31");
  // every tile count must fit in 2^31 - 1; the bf16 bounds round like the
  // launchers: ragged-M row slots up to whole row-tile groups and the logical
  // tile count up to a multiple of 8, weight-gradient grids up to a multiple
  // of 64
  const int64_t lim = ((int64_t)1 << 31) - 1;
  const int64_t wide = s->d > 2 * (int64_t)s->F ? s->d : 2 * (int64_t)s->F;
  int64_t gemm_blocks;
  int64_t gemm_threads;  // threads of the largest grouped-GEMM launch that is not persistent
  if (s->dtype == MOE_DTYPE_BF16) {
    const int64_t slots = ceil_div(R / kGemmBM + s->E, kGemmGroupM) * kGemmGroupM;
    gemm_blocks = ceil_div(slots * ceil_div(wide, kGemmBN / 2), 8) * 8;
    const int64_t wg = ceil_div((int64_t)s->E * ceil_div(wide, kGemmBM) * ceil_div(wide, kGemmBN), 64) * 64;
    if (wg > gemm_blocks) gemm_blocks = wg;
    gemm_threads = wg * 512;  // the ragged-M products run one 512-thread workgroup per CU
  } else {
    gemm_blocks = (R / kGemmF32Tile + s->E) * ceil_div(wide, kGemmF32Tile);
    const int64_t wg = (int64_t)s->E * ceil_div(wide, kGemmF32Tile) * ceil_div(wide, kGemmF32Tile);
    if (wg > gemm_blocks) gemm_blocks = wg;
    gemm_threads = gemm_blocks * 256;
  }
  const int64_t vec = s->dtype == MOE_DTYPE_BF16 ? 8 : 4;
  const int64_t mem_blocks = ceil_div(s->T * (s->d / vec), 256);
  if (gemm_blocks > lim || mem_blocks > lim) return fail(why, MOE_ERR_UNSUPPORTED, "problem too large for one launch");
  // a grid dimension holds fewer than 2^32 threads: the per-token launches
  // (256 threads per token at most), the one-thread-per-chunk memory kernels
  // and the non-persistent grouped GEMM grids
  const int64_t items = (int64_t)1 << 32;
  if (s->T * 256 >= items || s->T * (s->d / vec) >= items || gemm_threads >= items)
    return fail(why, MOE_ERR_UNSUPPORTED, "problem too large for one launch (2^32 threads per grid dimension)");
  return MOE_OK;
}

WorkspaceLayout workspace_layout(const moe_shape &s) {
  WorkspaceLayout w{};
  const int64_t nblk = ceil_div(s.T, kRouteTokens);
  w.route_blk_cnt = align256((size_t)nblk * (size_t)s.E * 4);
  int64_t chunk_tokens = ceil_div(s.T, kRouterChunksMax);
  if (chunk_tokens < 256) chunk_tokens = 256;
  const int64_t nchunk = ceil_div(s.T, chunk_tokens);
  w.route_partial = align256((size_t)nchunk * (size_t)s.E * (size_t)s.d * 4);
  const int64_t aux_blocks = ceil_div(s.T, aux_tokens_per_block(s.T));
  w.route_aux = align256((size_t)aux_blocks * ((size_t)s.E + 3) * 4);
  w.route_total = w.route_blk_cnt + w.route_partial;
  if (w.route_aux > w.route_total) w.route_total = w.route_aux;
  const size_t es = s.dtype == MOE_DTYPE_BF16 ? 2 : 4;
  const size_t R = (size_t)s.T * (size_t)s.k;
  const bool recompute = (s.flags & MOE_FLAG_RECOMPUTE) != 0;
  w.gemm_fwd_total = recompute ? align256(R * (size_t)s.F * es) : 0;
  w.gemm_bwd_dh = align256(R * 2 * (size_t)s.F * es);
  w.gemm_bwd_order = align256((size_t)s.E * 4);
  w.gemm_bwd_a = recompute ? align256(R * (size_t)s.F * es) : 0;
  w.gemm_bwd_total = w.gemm_bwd_dh + w.gemm_bwd_order + w.gemm_bwd_a;
  return w;
}

moe_status validate_ptrs(const PtrArg *args, int n, std::string *why) {
  for (int i = 0; i < n; ++i) {
    const PtrArg &a = args[i];
    char buf[160];
    if (a.needed && !a.ptr) {
      snprintf(buf, sizeof buf, "%s is NULL", a.name);
      return fail(why, MOE_ERR_INVALID_ARGUMENT, buf);
    }
    if (a.must_be_null && a.ptr) {
      snprintf(buf, sizeof buf, "%s must be NULL in this mode", a.name);
      return fail(why, MOE_ERR_INVALID_ARGUMENT, buf);
    }
  }
  for (int i = 0; i < n; ++i) {
    const PtrArg &a = args[i];
    if (a.ptr && ((uintptr_t)a.ptr & 15u) != 0) {
      char buf[160];
      snprintf(buf, sizeof buf, "%s is not 16-byte aligned", a.name);
      return fail(why, MOE_ERR_MISALIGNED, buf);
    }
  }
  return MOE_OK;
}

moe_status validate_apart(std::initializer_list<Beside> pairs, std::string *why) {
  for (const Beside &p : pairs) {
    const uintptr_t a = (uintptr_t)p.out.ptr, b = (uintptr_t)p.other.ptr;
    if (!a || !b || a >= b + p.other.bytes || b >= a + p.out.bytes || (p.same_ok && a == b)) continue;
    char buf[160];
    snprintf(buf, sizeof buf, "%s is written and shares memory with %s%s", p.out.name, p.other.name,
             p.same_ok ? ", which it may only do from the same address on" : "");
    return fail(why, MOE_ERR_INVALID_ARGUMENT, buf);
  }
  return MOE_OK;
}

moe_status validate_workspace(const void *ws, size_t have, size_t need, std::string *why) {
  if (need == 0) return MOE_OK;
  if (!ws) return fail(why, MOE_ERR_WORKSPACE, "workspace is NULL");
  if (((uintptr_t)ws & 15u) != 0) return fail(why, MOE_ERR_MISALIGNED, "workspace is not 16-byte aligned");
  if (have < need) {
    char buf[160];
    snprintf(buf, sizeof buf, "workspace too small: %zu bytes given, %zu needed", have, need);
    return fail(why, MOE_ERR_WORKSPACE, buf);
  }
  return MOE_OK;
}

moe_status validate_adamw(const moe_adamw_config *c, int64_t n, std::string *why) {
  if (!c) return fail(why, MOE_ERR_INVALID_ARGUMENT, "adamw config is NULL");
  if (n < 0) return fail(why, MOE_ERR_INVALID_ARGUMENT, "negative element count");
  // eight elements per thread: 2^35 elements fill a grid of 2^32 threads
  if (n >= ((int64_t)1 << 35)) return fail(why, MOE_ERR_UNSUPPORTED, "element count >= 2^35");
  if (c->flags & ~(uint32_t)MOE_ADAMW_ZERO_GRAD) return fail(why, MOE_ERR_UNSUPPORTED, "unknown adamw flag bits");
  const float vals[] = {c->lr, c->beta1, c->beta2, c->eps, c->weight_decay, c->grad_scale};
  for (float v : vals)
    if (!std::isfinite(v)) return fail(why, MOE_ERR_INVALID_ARGUMENT, "non-finite adamw scalar");
  if (c->lr < 0.f) return fail(why, MOE_ERR_INVALID_ARGUMENT, "lr < 0");
  if (c->beta1 < 0.f || c->beta1 >= 1.f || c->beta2 < 0.f || c->beta2 >= 1.f)
    return fail(why, MOE_ERR_INVALID_ARGUMENT, "beta outside [0, 1)");
  if (c->eps <= 0.f) return fail(why, MOE_ERR_INVALID_ARGUMENT, "eps <= 0");
  if (c->weight_decay < 0.f) return fail(why, MOE_ERR_INVALID_ARGUMENT, "weight_decay < 0");
  if (c->step < 1) return fail(why, MOE_ERR_INVALID_ARGUMENT, "step < 1");
  return MOE_OK;
}

moe_status validate_ep(int32_t ep, int32_t e_local, int32_t d, int32_t dtype, int64_t rows_cap, std::string *why) {
  if (ep < 1 || ep > kEpMaxRanks) return fail(why, MOE_ERR_UNSUPPORTED, "ep outside [1, MOE_EP_MAX_RANKS]");
  if (e_local < 1) return fail(why, MOE_ERR_INVALID_ARGUMENT, "e_local < 1");
  if ((int64_t)ep * e_local > 256) return fail(why, MOE_ERR_UNSUPPORTED, "ep * e_local > 256");
  if (d != 0) {
    if (d < 0) return fail(why, MOE_ERR_INVALID_ARGUMENT, "d < 0");
    if (d % 64 != 0 || d > 65536) return fail(why, MOE_ERR_UNSUPPORTED, "d must be a multiple of 64, at most 65536");
    if (dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16)
      return fail(why, MOE_ERR_UNSUPPORTED, "dtype must be MOE_DTYPE_F32 or MOE_DTYPE_BF16");
  }
  if (rows_cap < 0) return fail(why, MOE_ERR_INVALID_ARGUMENT, "negative row capacity");
  // one 256-thread workgroup per row: 2^24 rows fill a grid of 2^32 threads
  if (rows_cap >= ((int64_t)1 << 24)) return fail(why, MOE_ERR_UNSUPPORTED, "row capacity >= 2^24");
  return MOE_OK;
}

moe_status validate_aux(const moe_aux_config *c, std::string *why) {
  if (!c) return fail(why, MOE_ERR_INVALID_ARGUMENT, "aux config is NULL");
  if (c->flags & ~(uint32_t)MOE_AUX_ACCUMULATE) return fail(why, MOE_ERR_UNSUPPORTED, "unknown aux flag bits");
  if (!std::isfinite(c->balance_coef) || !std::isfinite(c->z_coef))
    return fail(why, MOE_ERR_INVALID_ARGUMENT, "non-finite aux coefficient");
  return MOE_OK;
}

static moe_status validate_rows(int64_t T, int32_t d, std::string *why) {
  if (T < 0) return fail(why, MOE_ERR_INVALID_ARGUMENT, "T < 0");
  if (d <= 0) return fail(why, MOE_ERR_INVALID_ARGUMENT, "d must be positive");
  if (d % 64 != 0 || d > 65536) return fail(why, MOE_ERR_UNSUPPORTED, "d must be a multiple of 64, at most 65536");
  // a 256-thread workgroup per row: 2^24 rows fill a grid of 2^32 threads
  if (T >= ((int64_t)1 << 24)) return fail(why, MOE_ERR_UNSUPPORTED, "T >= 2^24");
  return MOE_OK;
}

moe_status validate_norm(const moe_norm_shape *s, std::string *why) {
  if (!s) return fail(why, MOE_ERR_INVALID_ARGUMENT, "norm shape is NULL");
  const moe_status st = validate_rows(s->T, s->d, why);
  if (st != MOE_OK) return st;
  if (s->dtype != MOE_DTYPE_F32 && s->dtype != MOE_DTYPE_BF16)
    return fail(why, MOE_ERR_UNSUPPORTED, "dtype must be MOE_DTYPE_F32 or MOE_DTYPE_BF16");
  if (s->flags & ~(uint32_t)MOE_NORM_OVERWRITE_DW) return fail(why, MOE_ERR_UNSUPPORTED, "unknown norm flag bits");
  if (!std::isfinite(s->eps) || s->eps <= 0.f) return fail(why, MOE_ERR_INVALID_ARGUMENT, "eps must be positive and finite");
  return MOE_OK;
}

size_t norm_workspace(const moe_norm_shape &s) { return align256((size_t)norm_bwd_blocks(s.T) * (size_t)s.d * 4); }

moe_status validate_mx8(int64_t rows, int32_t cols, int32_t dtype, std::string *why) {
  if (rows < 0) return fail(why, MOE_ERR_INVALID_ARGUMENT, "negative row count");
  if (cols <= 0) return fail(why, MOE_ERR_INVALID_ARGUMENT, "cols must be positive");
  if (cols % 64 != 0 || cols > 65536) return fail(why, MOE_ERR_UNSUPPORTED, "cols must be a multiple of 64, at most 65536");
  if (dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16)
    return fail(why, MOE_ERR_UNSUPPORTED, "dtype must be MOE_DTYPE_F32 or MOE_DTYPE_BF16");
  // one thread per 16 bytes
  if (rows >= ((int64_t)1 << 32) || rows * (cols / (dtype == MOE_DTYPE_BF16 ? 8 : 4)) >= ((int64_t)1 << 32) - 256)
    return fail(why, MOE_ERR_UNSUPPORTED, "matrix too large for one launch (2^32 threads per grid dimension)");
  return MOE_OK;
}

moe_status validate_ffn(const moe_ffn_shape *s, std::string *why) {
  if (!s) return fail(why, MOE_ERR_INVALID_ARGUMENT, "ffn shape is NULL");
  moe_status st = validate_rows(s->T, s->d, why);
  if (st != MOE_OK) return st;
  if (s->F <= 0) return fail(why, MOE_ERR_INVALID_ARGUMENT, "F must be positive");
  if (s->F % 64 != 0 || s->F > 65536) return fail(why, MOE_ERR_UNSUPPORTED, "F must be a multiple of 64, at most 65536");
  if (s->dtype != MOE_DTYPE_BF16 && s->dtype != MOE_DTYPE_MX8)
    return fail(why, MOE_ERR_UNSUPPORTED, "dtype must be MOE_DTYPE_BF16 or MOE_DTYPE_MX8");
  if (s->dtype == MOE_DTYPE_MX8 && (s->d % 128 != 0 || s->F % 128 != 0))
    return fail(why, MOE_ERR_UNSUPPORTED, "d and F must be multiples of 128 in MOE_DTYPE_MX8");
  if (s->flags & ~(uint32_t)MOE_FFN_OVERWRITE_DW) return fail(why, MOE_ERR_UNSUPPORTED, "unknown ffn flag bits");
  // the largest grid: 128 x 128 tiles of [T, 2F] or [T, d], row tiles in whole
  // groups, 256 threads each (smaller tiles are only for grids of a few CUs' worth)
  const int64_t wide = s->d > 2 * (int64_t)s->F ? s->d : 2 * (int64_t)s->F;
  const int64_t tiles = ceil_div(ceil_div(s->T, 128), kGemmGroupM) * kGemmGroupM * ceil_div(wide, 128);
  if ((tiles + 8) * 256 >= ((int64_t)1 << 32))
    return fail(why, MOE_ERR_UNSUPPORTED, "problem too large for one launch (2^32 threads per grid dimension)");
  return MOE_OK;
}

// Tiles of the two weight gradients together.
static int64_t wgrad_tiles(int tile, int d, int F) {
  return ceil_div(2 * (int64_t)F, tile) * ceil_div(d, tile) + ceil_div(d, tile) * ceil_div(F, tile);
}

// Times of the large tiles in us: of a stage with one round of workgroups and
// with more, beside the stages (the launch, the start, the end), and the most
// TFLOP/s. `tiles(tile)`: tiles of all products; elems: their elements.
struct WgradRate {
  double stage, crowded, fixed, tflops;
};
template <typename Tiles>
static FfnWgrad wgrad_plan(int64_t T, double elems, const WgradRate &large, Tiles count) {
  // Time of n slices in us: a fixed part, then rounds of workgroups, each a run
  // of stages of 64 tokens. 256 x 256 tiles run one a CU (`large`); 128 x 128
  // tiles two a CU, 0.65 us a stage alone on one, 1.05 beyond, at most 1060
  // TFLOP/s in all. A second launch writes and reads n times the gradients at 4
  // TB/s. Measured for the dense block (tile, slices: us): d = 2048, F = 1408 at 2000 tokens 256, 1: 51,
  // 256, 3: 75, 128, 1: 59; at 7001 256, 1: 145, 256, 3: 149, 128, 2: 166; at
  // 32768 256, 1: 694, 256, 3: 589; d = 512, F = 320 at 3000 256, 11: 27, 128,
  // 1: 33, 128, 4: 18.5; d = 1088, F = 576 at 700 256, 1: 23, 128, 1: 12.
  const double bytes = 4.0 * elems;
  FfnWgrad w{256, 0, 0, 1};
  double best_us = 0.0;
  int64_t best = 1;
  for (int tile = 256; tile >= 128; tile /= 2) {
    const int64_t tiles = count(tile);
    int64_t most = kWgradUnits / tiles;
    if (most > T / kWgradMinRows) most = T / kWgradMinRows;
    if (most < 1) most = 1;
    if (most > w.most) w.most = (int)most;
    for (int64_t n = 1; n <= most; ++n) {
      const int64_t rounds = ceil_div(tiles * n, tile == 256 ? 256 : 512), stages = ceil_div(ceil_div(T, n), 64);
      const double stage = tile == 256 ? (rounds > 1 ? large.crowded : large.stage) : (tiles * n > 256 ? 1.05 : 0.65);
      const double least = 2.0 * (double)T * elems / (1e6 * (tile == 256 ? large.tflops : 1060.0));
      double us = (tile == 256 ? large.fixed : 4.0) + (double)(rounds * stages) * stage;
      if (us < least) us = least;
      if (n > 1) us += 5.0 + (double)n * bytes / 4e6;
      if ((tile == 256 && n == 1) || us < best_us) {
        w.tile = tile;
        best = n;
        best_us = us;
      }
    }
  }
  w.chunk = (int)(ceil_div(ceil_div(T, best), 64) * 64);
  w.slices = T > 0 ? (int)ceil_div(T, w.chunk) : 0;
  return w;
}

// 1.35 us a stage while every workgroup has a CU from the start, 1.6 beyond.
FfnWgrad ffn_wgrad_plan(int64_t T, int d, int F) {
  return wgrad_plan(T, 3.0 * d * F, {1.35, 1.6, 4.0, 1060.0}, [&](int tile) { return wgrad_tiles(tile, d, F); });
}

FfnWorkspace ffn_workspace(const moe_ffn_shape &s) {
  FfnWorkspace w{};
  const bool mx8 = s.dtype == MOE_DTYPE_MX8;
  const size_t n = (size_t)s.T * (size_t)s.F;
  w.fwd_a = align256(mx8 ? n : 2 * n);
  w.fwd_scale = mx8 ? align256(n / 32) : 0;
  const size_t few = (size_t)(s.T < kFfnFewTokens ? s.T : kFfnFewTokens);
  w.fwd_a32 = mx8 ? align256(few * (size_t)s.F * 4) : 0;
  w.fwd_total = w.fwd_a + w.fwd_scale + w.fwd_a32;
  // gradients of so many tiles that no T is sliced are written to directly
  if (!mx8 && s.T > 0 && wgrad_tiles(256, s.d, s.F) * 2 <= kWgradUnits)
    w.wgrad_total = align256((size_t)ffn_wgrad_plan(s.T, s.d, s.F).most * 3 * (size_t)s.d * (size_t)s.F * 4);
  return w;
}

// ----- layer norm, dense product, orthogonalisation -----
size_t layernorm_workspace(const moe_norm_shape &s) {
  return align256((size_t)norm_bwd_blocks(s.T) * 2 * (size_t)s.d * 4);
}

moe_status validate_act(int32_t act, std::string *why) {
  if (act < MOE_ACT_NONE || act > MOE_ACT_SILU) return fail(why, MOE_ERR_UNSUPPORTED, "unknown activation");
  return MOE_OK;
}

moe_status validate_linear(const moe_linear_shape *s, std::string *why) {
  if (!s) return fail(why, MOE_ERR_INVALID_ARGUMENT, "linear shape is NULL");
  if (s->T < 0) return fail(why, MOE_ERR_INVALID_ARGUMENT, "T < 0");
  if (s->K <= 0 || s->N <= 0) return fail(why, MOE_ERR_INVALID_ARGUMENT, "K and N must be positive");
  if (s->K % 64 != 0 || s->K > 65536 || s->N % 64 != 0 || s->N > 65536)
    return fail(why, MOE_ERR_UNSUPPORTED, "K and N must be multiples of 64, at most 65536");
  if (s->T >= ((int64_t)1 << 24)) return fail(why, MOE_ERR_UNSUPPORTED, "T >= 2^24");
  if (s->dtype != MOE_DTYPE_BF16) return fail(why, MOE_ERR_UNSUPPORTED, "dtype must be MOE_DTYPE_BF16");
  const moe_status st = validate_act(s->act, why);
  if (st != MOE_OK) return st;
  if (s->flags & ~(uint32_t)MOE_LINEAR_OVERWRITE_DW) return fail(why, MOE_ERR_UNSUPPORTED, "unknown linear flag bits");
  // the largest grid: 128 x 128 tiles of [T, N] or [T, K], row tiles in whole
  // groups, 256 threads each; the elementwise pass has a thread for 8 values
  const int64_t wide = s->K > s->N ? s->K : s->N;
  const int64_t tiles = ceil_div(ceil_div(s->T, 128), kGemmGroupM) * kGemmGroupM * ceil_div(wide, 128);
  if ((tiles + 8) * 256 >= ((int64_t)1 << 32) || s->T * (wide / 8) >= ((int64_t)1 << 32) - 256)
    return fail(why, MOE_ERR_UNSUPPORTED, "problem too large for one launch (2^32 threads per grid dimension)");
  return MOE_OK;
}

static int64_t linear_tiles(int tile, int K, int N) { return ceil_div(N, tile) * ceil_div(K, tile); }

// The alternating main loop: a round of 256 x 256 tiles at 1.37 us a stage, further
// rounds too; 8 us of start and end; 1500 TFLOP/s at most. Low for the longest sums
// (32768 x 2048 x 1408 in 5 slices: 149 us against 186 without the joining launch),
// alike for all of them, so that the order holds: of 16 sizes the plan's choice is the
// fastest, or within 3 us of it. us, T x K x N (tile, slices; the plan's first): 32768
// x 2048 x 1408 256, 5: 195, 256, 10: 212, 256, 3: 265, 128, 2: 255; 65536 x 1024 x
// 1024 256, 16: 142, 128, 8: 189; 16384 x 4096 x 1024 256, 4: 136, 256, 3: 155, 256, 8:
// 155, 128, 2: 169; 8192 x 4096 x 4096 256, 1: 237, 256, 2: 270, 128, 1: 311; 8192 x
// 2048 x 2048 256, 4: 79, 256, 3: 86, 128, 2: 92; 9001 x 2112 x 1088 256, 5: 67, 256,
// 6: 100, 128, 3: 69; 4096 x 1024 x 1024 128, 4: 28, 128, 8: 31, 256, 16: 35; 3000 x
// 2048 x 2048 128, 1: 45, 256, 3: 47; 2048 x 8192 x 2048 256, 1: 68, 128, 1: 99; 1000 x
// 4160 x 4160 (289 tiles) 256, 1: 68, 128, 1: 66.
FfnWgrad linear_wgrad_plan(int64_t T, int K, int N) {
  return wgrad_plan(T, (double)K * N, {1.37, 1.37, 8.0, 1500.0}, [&](int tile) { return linear_tiles(tile, K, N); });
}

LinearWorkspace linear_workspace(const moe_linear_shape &s) {
  LinearWorkspace w{};
  if (s.T > 0 && linear_tiles(256, s.K, s.N) * 2 <= kWgradUnits)
    w.dw = align256((size_t)linear_wgrad_plan(s.T, s.K, s.N).most * (size_t)s.K * (size_t)s.N * 4);
  // of db: by the slices of the large tiles or of a pass of its own
  const size_t slices = (size_t)std::max(linear_db_slices(s.T), s.T > 0 ? linear_wgrad_plan(s.T, s.K, s.N).most : 0);
  w.db = align256(slices * (size_t)s.N * 4);
  w.total = w.dw + w.db;
  return w;
}

// Largest |p| of p(x) = a x + b x^3 + c x^5 on [0, m].
static double quintic_peak(double a, double b, double c, double m) {
  const auto p = [&](double x) { return std::fabs(x * (a + x * x * (b + x * x * c))); };
  double top = p(m);
  const auto at = [&](double s) {  // s = x^2 where p' may vanish
    if (s > 0.0 && s < m * m) top = std::max(top, p(std::sqrt(s)));
  };
  if (c == 0.0) {
    if (b != 0.0) at(-a / (3.0 * b));
  } else {
    const double disc = 9.0 * b * b - 20.0 * a * c;
    if (disc >= 0.0) {
      at((-3.0 * b + std::sqrt(disc)) / (10.0 * c));
      at((-3.0 * b - std::sqrt(disc)) / (10.0 * c));
    }
  }
  return top;
}

moe_status validate_orth(const moe_orth_shape *s, std::string *why) {
  if (!s) return fail(why, MOE_ERR_INVALID_ARGUMENT, "orth shape is NULL");
  if (s->batch < 0) return fail(why, MOE_ERR_INVALID_ARGUMENT, "batch < 0");
  if (s->rows <= 0 || s->cols <= 0) return fail(why, MOE_ERR_INVALID_ARGUMENT, "rows and cols must be positive");
  if (s->rows > 65536 || s->cols > 65536) return fail(why, MOE_ERR_UNSUPPORTED, "rows and cols must be at most 65536");
  if (s->dtype != MOE_DTYPE_F32 && s->dtype != MOE_DTYPE_BF16)
    return fail(why, MOE_ERR_UNSUPPORTED, "dtype must be MOE_DTYPE_F32 or MOE_DTYPE_BF16");
  if (s->steps < 1 || s->steps > 16) return fail(why, MOE_ERR_UNSUPPORTED, "steps must be between 1 and 16");
  if (!std::isfinite(s->eps) || s->eps <= 0.f) return fail(why, MOE_ERR_INVALID_ARGUMENT, "eps must be positive and finite");
  const double a = s->a, b = s->b, c = s->c;
  if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c))
    return fail(why, MOE_ERR_INVALID_ARGUMENT, "non-finite coefficient");
  // Singular values start at most 1; X, X X^T and b X X^T + c (X X^T)^2 are held
  // in fp16 times 2^12, whose largest number is below 16 times that.
  double m = 1.0;
  for (int k = 0; k < s->steps; ++k) {
    const double l = m * m;
    double poly = std::fabs(b * l + c * l * l);
    if (c != 0.0 && -b / (2.0 * c) > 0.0 && -b / (2.0 * c) < l) poly = std::max(poly, b * b / (4.0 * std::fabs(c)));
    if (l > 15.0 || poly > 15.0)
      return fail(why, MOE_ERR_UNSUPPORTED, "the coefficients let singular values grow past fp16's range");
    m = quintic_peak(a, b, c, m);
  }
  if (m > 15.0) return fail(why, MOE_ERR_UNSUPPORTED, "the coefficients let singular values grow past fp16's range");
  // the largest grids: 64 x 64 tiles of all matrices, 512 threads each, twice
  // that per tile of the smallest product shapes
  const int64_t tiles = ceil_div(s->rows, 64) * ceil_div(s->cols, 64);
  if (s->batch >= ((int64_t)1 << 22) || s->batch * tiles >= ((int64_t)1 << 22))
    return fail(why, MOE_ERR_UNSUPPORTED, "problem too large for one launch (2^32 threads per grid dimension)");
  return MOE_OK;
}

moe_status validate_muon(const moe_muon_config *c, std::string *why) {
  if (!c) return fail(why, MOE_ERR_INVALID_ARGUMENT, "muon config is NULL");
  if (c->flags & ~(uint32_t)(MOE_MUON_NESTEROV | MOE_MUON_ZERO_GRAD))
    return fail(why, MOE_ERR_UNSUPPORTED, "unknown muon flag bits");
  if (!std::isfinite(c->lr) || !std::isfinite(c->weight_decay) || !std::isfinite(c->scale) ||
      !std::isfinite(c->grad_scale) || !std::isfinite(c->momentum))
    return fail(why, MOE_ERR_INVALID_ARGUMENT, "non-finite muon scalar");
  if (c->momentum < 0.f || c->momentum >= 1.f)
    return fail(why, MOE_ERR_INVALID_ARGUMENT, "momentum must lie in [0, 1)");
  return MOE_OK;
}

OrthWorkspace orth_workspace(int64_t batch, int rows, int cols) {
  OrthWorkspace w{};
  const int small = rows < cols ? rows : cols, large = rows < cols ? cols : rows;
  w.S = (small + 63) / 64 * 64;
  w.L = (large + 63) / 64 * 64;
  // partial sums of 4096 elements or more (16 a thread), 256 of a matrix at most
  const int64_t parts = ceil_div((int64_t)rows * cols, 4096);
  w.parts = (int)(parts < 256 ? parts : 256);
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    const size_t o = at;
    at += align256(bytes);
    return o;
  };
  const size_t n = (size_t)batch;
  w.partial = take(n * (size_t)w.parts * 8);
  for (int i = 0; i < 2; ++i) {
    w.hi[i] = take(n * (size_t)w.S * (size_t)w.L * 2);
    w.lo[i] = take(n * (size_t)w.S * (size_t)w.L * 2);
  }
  w.a = take(n * (size_t)w.S * (size_t)w.S * 2);
  w.b = take(n * (size_t)w.S * (size_t)w.S * 2);
  const size_t low = orth_both_halves(w.S) ? n * (size_t)w.S * (size_t)w.S * 2 : 0;
  w.alo = take(low);
  w.blo = take(low);
  w.da = take(n * (size_t)w.S * 4);
  w.db = take(n * (size_t)w.S * 4);
  w.sums = take(batch > 0 && orth_gram_sliced(w.S, w.L) ? (size_t)kOrthSliceTiles * 128 * 128 * 4 : 0);
  w.total = at;
  return w;
}

}  // namespace moe
