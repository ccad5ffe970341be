// Host-side argument validation and workspace sizing for the C ABI. Pure
// C++ (no HIP), so it can be built and unit-tested without a GPU.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>
#include <initializer_list>
#include <string>

#include "moe.h"

namespace moe {

// Tile sizes the launchers use; validation checks that grids fit.
constexpr int kRouteTokens = 64;        // tokens per top-k workgroup (one wavefront)
constexpr int kRouterChunksMax = 32;    // router weight-gradient partial sums
constexpr int kGemmBM = 256;            // bf16 grouped GEMM rows per tile
constexpr int kGemmBN = 256;            // bf16 grouped GEMM columns per tile
constexpr int kGemmGroupM = 4;          // row tiles per group in the ragged-M tile order
constexpr int kGemmF32Tile = 16;        // fp32 grouped GEMM tile edge
constexpr int kAuxMaxBlocks = 1024;     // partial rows of the auxiliary-loss pass
// Static per-GPU scratch of moe_route_noalloc: the per-workgroup expert
// histograms of the route pass, ceil(T / kRouteTokens) * E int32.
constexpr size_t kRouteScratchBytes = (size_t)16 << 20;
constexpr int kEpMaxRanks = 8;          // expert-parallel ranks of the exchange stand-in (one node)

struct WorkspaceLayout {
  size_t route_blk_cnt;   // bytes of the per-workgroup expert histograms
  size_t route_partial;   // bytes of router weight-gradient partial sums
  size_t route_aux;       // bytes of the auxiliary-loss partial rows (shares the route workspace)
  size_t route_total;
  size_t gemm_fwd_total;  // recompute: a [R,F] at offset 0; else nothing
  size_t gemm_bwd_dh;     // bytes of dH (recompute: the recomputed h first)
  size_t gemm_bwd_order;  // bytes of the expert order (int32 [E])
  size_t gemm_bwd_a;      // recompute: bytes of the recomputed a; else 0
  size_t gemm_bwd_total;  // dh | order | a
};

inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tokens per workgroup of the auxiliary-loss pass: at least kAuxMinTokens
// (512 workgroups at 32k tokens), at most kAuxMaxBlocks workgroups.
constexpr int kAuxMinTokens = 64;
inline int aux_tokens_per_block(int64_t T) {
  int64_t tpb = ceil_div(T, kAuxMaxBlocks);
  if (tpb < kAuxMinTokens) tpb = kAuxMinTokens;
  return (int)tpb;
}

// Validates the shape alone. On failure writes a message to *why.
moe_status validate_shape(const moe_shape *s, std::string *why);

// Workspace layout of a (validated) shape.
WorkspaceLayout workspace_layout(const moe_shape &s);

// One pointer argument: `needed` tells whether the call reads or writes it.
// NULL where needed -> MOE_ERR_INVALID_ARGUMENT; non-NULL where it must be
// NULL (must_be_null) -> MOE_ERR_INVALID_ARGUMENT; not 16-byte aligned ->
// MOE_ERR_MISALIGNED.
struct PtrArg {
  const char *name;
  const void *ptr;
  bool needed;
  bool must_be_null;
};
moe_status validate_ptrs(const PtrArg *args, int n, std::string *why);

// AdamW scalars and element count (see moe_adamw_step).
moe_status validate_adamw(const moe_adamw_config *cfg, int64_t n, std::string *why);

// Auxiliary-loss coefficients and flags (see moe_aux_loss).
moe_status validate_aux(const moe_aux_config *cfg, std::string *why);

// Expert-parallel exchange sizes: 1 <= ep <= kEpMaxRanks, e_local >= 1,
// ep*e_local <= 256; d a positive multiple of 64 (<= 65536) and dtype valid
// when d > 0 is given; capacities >= 0 and below 2^31 rows.
moe_status validate_ep(int32_t ep, int32_t e_local, int32_t d, int32_t dtype, int64_t rows_cap, std::string *why);

// ----- RMS norm, 8-bit block form, dense feed-forward block -----
constexpr int kNormWaveRows = 2048;     // rows from which a norm row is one wavefront's
constexpr int kNormBwdBlocks = 512;    // workgroups (partial rows) of the norm's backward pass at most
constexpr int kNormBwdMinRows = 8;      // rows of a workgroup of the norm's backward pass at least
inline int norm_bwd_blocks(int64_t T) {
  const int64_t b = ceil_div(T, kNormBwdMinRows);
  return (int)(b < kNormBwdBlocks ? b : kNormBwdBlocks);
}

// Tokens up to which the block's forward runs the few-token kernels.
constexpr int kFfnFewTokens = 144;

// Tile and token slices of the dense block's two weight gradients (dw_gu
// [2F,d], then dw_down [d,F]): at most as many slices as make kWgradUnits
// workgroups, each at least kWgradMinRows tokens; among those the tile and
// count whose time estimate is least (ffn_wgrad_plan).
constexpr int kWgradUnits = 512;
constexpr int kWgradMinRows = 256;
struct FfnWgrad {
  int tile;           // 256 or 128: rows and columns of a tile
  int slices, chunk;  // chunk: tokens of a slice
  int most;           // slices of the workspace: never fewer for a larger T
};
FfnWgrad ffn_wgrad_plan(int64_t T, int d, int F);

// Shape of a norm call (d a multiple of 64, at most 65536; T < 2^24).
moe_status validate_norm(const moe_norm_shape *s, std::string *why);
size_t norm_workspace(const moe_norm_shape &s);

// Rows and columns of the 8-bit block form (cols a multiple of 64).
moe_status validate_mx8(int64_t rows, int32_t cols, int32_t dtype, std::string *why);

// Shape of a dense feed-forward call, and its workspaces.
moe_status validate_ffn(const moe_ffn_shape *s, std::string *why);
struct FfnWorkspace {
  size_t fwd_a, fwd_scale, fwd_a32;    // a (bf16, or e4m3, its scales, and few tokens' a in fp32)
  size_t fwd_total;
  size_t wgrad_total;                  // fp32 partial sums of the two weight gradients; 0: no T of this d and F has any
};
FfnWorkspace ffn_workspace(const moe_ffn_shape &s);

// ----- layer norm, dense product, orthogonalisation -----
size_t layernorm_workspace(const moe_norm_shape &s);

// Shape of a dense product's call, its weight gradient's tile and slices (as
// ffn_wgrad_plan, for dW [N,K] alone) and its workspace.
moe_status validate_linear(const moe_linear_shape *s, std::string *why);
moe_status validate_act(int32_t act, std::string *why);
FfnWgrad linear_wgrad_plan(int64_t T, int K, int N);
constexpr int kLinearDbSlices = 64;   // token slices of the bias gradient at most
constexpr int kLinearDbRows = 256;    // tokens of such a slice at least
inline int linear_db_slices(int64_t T) {
  const int64_t n = ceil_div(T, kLinearDbRows);
  return (int)(n < kLinearDbSlices ? n : kLinearDbSlices);
}
struct LinearWorkspace {
  size_t dw, db, total;  // fp32 partial sums of dW, then of db
};
LinearWorkspace linear_workspace(const moe_linear_shape &s);

// Shape of an orthogonalisation (its coefficients among it: every singular
// value of every iterate stays in fp16's range) and its workspace.
moe_status validate_orth(const moe_orth_shape *s, std::string *why);
moe_status validate_muon(const moe_muon_config *cfg, std::string *why);
struct OrthWorkspace {
  int S, L;                              // padded short and long side
  int parts;                             // partial sums of a matrix
  size_t partial, hi[2], lo[2], a, b, alo, blo, da, db, sums, total;  // byte offsets (alo, blo: both halves)
};
// Short sides up to which every tensor of the iteration is held and multiplied in two
// fp16 halves (three products for one), so that the result is fp32's: with X alone in
// two, the roundings that fewer terms average cost 1e-3 to 2e-3 of the norm at 8 x 8,
// 9e-4 at 40 x 40, 7e-4 at 128 x 128, 6e-4 at 300 x 300, and 4e-4 to 6e-4 at every
// longer side. Muon step in us, one half against both: 64 x 64 70, 82; 11 of 62 x 14 80, 89; 64
// of 100 x 100 88, 107; 8 of 88 x 141 86, 101; 5 of 419 x 328 110, 156; 3 of 1001 x 333
// 129, 189; 64 x 8192 200, 357; and past the border 64 of 512 x 512 571, 1002; 64 of 640
// x 640 864, 1784.
constexpr int kOrthBothSide = 384;
inline bool orth_both_halves(int S) { return S <= kOrthBothSide; }
// Slices of the sum of the product X X^T on 128 x 128 tiles, `tiles` of them, where
// they leave CUs idle, and the tiles' partial sums at most (of every batch whose
// sides are S and L): of 1365 terms at least, as many as make two workgroups a CU,
// and three or none; of more tiles than half the CUs only sums from 6144 on. The
// launch that joins them takes 8 us. Muon step in us, whole against in 3 to 6 slices,
// (matrices x) S x L: 1472 x 4096 441, 410; 1500 x 4200 467, 428; 5 x 700 x 4100 503,
// 495; 2048 x 6144 726, 715; 2048 x 8192 906, 846; 2176 x
// 8192 1167, 1127; 2 x 1408 x 8192 1035, 972; 9 x 512 x 8192 1056, 940; 1472 x 16384
// 1327, 1040; 2048 x 16384 1675, 1491. On the other side: 2176 x 4096 611, 657; 2 x 1408
// x 4096 547, 560; 2048 x 3008 485, 502; 2048 x 2048 381, 406 (2048 x 4096 568, 560, and
// 1472 x 3008 382, 367, gain a little). In 2: 2816 x 8192 1456, 1488; 2560 x 8192 1336,
// 1348; 2304 x 4096 640, 691; 2048 x 4096 568, 579 (2560 x 16384 2230, 2182).
constexpr int kOrthSliceTiles = 512;
inline bool orth_gram_sliced(int S, int L) {  // for any batch
  const int64_t m = ceil_div(S, 128);
  return (L >= 4096 && m <= 15) || (L >= 6144 && m <= 17);  // 120 and 153 tiles of a matrix
}
inline int orth_gram_slices(int S, int L, int64_t tiles) {
  if (!orth_gram_sliced(S, L) || tiles < 1 || (tiles > 128 && L < 6144)) return 1;
  const int n = (int)std::min<int64_t>(kOrthSliceTiles / tiles, L / 1365);
  return n < 3 ? 1 : n;
}
OrthWorkspace orth_workspace(int64_t batch, int rows, int cols);

// Memory a call writes (`out`) and memory it reads or writes beside it: apart, or
// where `same_ok` starting at the same address, so that every element is written
// by the thread that read it. Rows shifted against each other would be read after
// another workgroup has written them. NULL passes.
struct Span {
  const char *name;
  const void *ptr;
  size_t bytes;
};
struct Beside {
  Span out, other;
  bool same_ok;
};
moe_status validate_apart(std::initializer_list<Beside> pairs, std::string *why);

// Workspace check: NULL or short -> MOE_ERR_WORKSPACE (a zero requirement
// accepts anything).
moe_status validate_workspace(const void *ws, size_t have, size_t need, std::string *why);

}  // namespace moe
