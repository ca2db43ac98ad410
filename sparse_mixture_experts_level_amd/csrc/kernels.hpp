// Host-side launchers of the gfx950 kernels (defined in the .hip files).  Each
// launcher only enqueues work on `stream` and returns the launch status; argument
// validation happens in api.cpp before any of these is called.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>

namespace moe {

// ---- router (router.hip)
hipError_t launch_router_logits_bf16(const void *x, const void *w_router, const float *offset, float *logits,
                                     int T, int d, int E, hipStream_t s);
hipError_t launch_router_logits_f32(const float *x, const float *w_router, const float *offset, float *logits,
                                    int T, int d, int E, hipStream_t s);
// Router linear and top-k in one call for bf16 layers; with few tokens the linear is
// split over d into router_splits() parts whose partial sums (router_partials_bytes()
// of workspace) the top-k kernel adds in order.
int router_splits(int T, int d, int E);
// The router linear as a large-tile GEMM (gemm_big.hip) for many tokens and experts: its
// split count along d (0: not used for this shape) and launch (float partials [S][T][E]).
int router_gemm_splits(int T, int d, int E);
hipError_t launch_router_gemm(const void *x, const void *w_router, int T, int d, int E, float *partials,
                              hipStream_t s);
size_t router_partials_bytes(int T, int d, int E);
hipError_t launch_router_bf16(const void *x, const void *w_router, const float *offset, float *logits, int T, int d,
                              int E, int k, int32_t *ids, float *gates, int32_t *spare, float *partials,
                              hipStream_t s);
// ids / gates may be NULL (not written).  With `spare`, also writes the experts ranked
// k .. 2k-1 per token into spare [T, k] (-1 where the rank is >= E).
hipError_t launch_router_topk(const float *logits, int T, int E, int k, int32_t *ids, float *gates, hipStream_t s,
                              int32_t *spare = nullptr);

// ---- dispatch (dispatch.hip)
// Assignments are walked in fill order: token-major (position p = t * k + j) or, with
// rank_major, rank-major (p = j * T + t).  Blocks own contiguous position ranges.
struct DispatchPlan {
  int64_t per_block;  // positions per block, a multiple of 256
  int num_blocks;
};
DispatchPlan dispatch_plan(int T, int k);
// Workspace of launch_dispatch, or of launch_dispatch_reroute when reroute is set.
size_t dispatch_workspace_bytes(int T, int k, int E, bool reroute);
hipError_t launch_dispatch(const int32_t *ids, int T, int k, int E, int cap /* <0: none */, bool rank_major,
                           int32_t *counts, int32_t *offsets, int32_t *slot, int32_t *row_token, int32_t *ws,
                           hipStream_t s);
// Two-pass fill: the plain fill, then every overflowing assignment is offered to the
// token's next ranked expert (spare [T, k] from launch_router_topk: the i-th overflow of
// a token takes spare[t][i]) and kept if that expert has room left; assigned [T, k]
// receives the serving expert of each assignment.  cap >= 0.
hipError_t launch_dispatch_reroute(const int32_t *ids, const int32_t *spare, int T, int k, int E, int cap,
                                   bool rank_major, int32_t *counts, int32_t *offsets, int32_t *slot,
                                   int32_t *assigned, int32_t *row_token, int32_t *ws, hipStream_t s);
hipError_t launch_gather_rows(const void *x, const int32_t *row_token, const int32_t *offsets_end, int64_t rows_max,
                              int d, int elem_bytes, void *x_perm, hipStream_t s);

// ---- grouped expert GEMMs (gemm_stream.hip, gemm_f32.hip)
// Problem: for group g, rows [offsets[g], offsets[g+1]) of A [rows, K] times the
// group's weight W_g [N_w, K] (K contiguous).  With swiglu, N_w = 2 * n_out and
// out[r, n] = silu(A_r . W_g[n]) * (A_r . W_g[n_out + n]); otherwise N_w = n_out and
// out[r, n] = A_r . W_g[n].  `w_group_stride` is in elements.
struct GroupedGemmArgs {
  const void *A;
  // Optional row gather: with row_index set, row r of a group is A[row_index[r]] and A
  // holds a_rows rows; otherwise rows are contiguous in A.
  const int32_t *row_index;
  int64_t a_rows;
  const int32_t *offsets;
  int num_groups;
  int group_rows_max;  // tiling hint
  int64_t rows_max;    // bound on the total rows over all groups
  const void *W;
  int64_t w_group_stride;
  int n_out;
  int K;
  void *out;
  bool swiglu;
  bool out_f32 = false;  // float output instead of the element type (bf16 kernels, no SwiGLU)
  // Workspace for float partial sums when the large-tile kernel cuts few tiles along K
  // (4 * rows_max * n_out floats); NULL: no K split.
  float *split_ws = nullptr;
  // Weights stored K-major: group g's matrix is [K, n_out] (row stride n_out) instead of
  // [n_out, K] -- the layout the backward pass multiplies by (dy W_d, dGU W_gu).  No SwiGLU.
  bool w_kn = false;
  // Large-tile regime only: A in the packed tile layout (launch_pack_rows; a_rows then
  // bounds the packed buffer in bytes, row_index unused), and/or the SwiGLU output written
  // in that layout for a following large-tile GEMM over the same groups (out sized
  // packed_rows_bytes(rows_max, num_groups, n_out)).
  bool a_packed = false;
  bool out_packed = false;
  // SwiGLU backward epilogue (with swiglu, bf16, plain row layout): instead of H, the
  // kernel forms from the float G, U of each row and bwd_dhp = dH' (bf16 [rows, n_out],
  // rows in group order) out = [dG | dU] (bf16 [rows, 2 n_out]), bwd_hg = g H (bf16
  // [rows, n_out]) and, when bwd_dpart is set, the dot products dH' . H of each row over
  // each 16-column block (float [rows, n_out / 16]); g = bwd_row_gate[row], or 1 when NULL.
  const void *bwd_dhp = nullptr;
  const float *bwd_row_gate = nullptr;
  void *bwd_hg = nullptr;
  float *bwd_dpart = nullptr;
  // Tails, large-tile regime: with tail = kBigTailRows a group's last partial 256-row tile
  // of at most that many rows is left to a streaming launch over the same groups
  // (re-reading that group's weights then costs less than a nearly empty tile); 0: every
  // row in large tiles; -1: chosen by the launch (big_tails()).  With a packed A or output
  // the tail launch reads tail_A instead (row-major; rows through tail_row_index when
  // given, tail_a_rows rows) and writes tail_out (row-major, rows in group order).
  int tail = -1;
  const void *tail_A = nullptr;
  const int32_t *tail_row_index = nullptr;
  int64_t tail_a_rows = 0;
  void *tail_out = nullptr;
  // Streaming kernel: compute only each group's tail rows (set by the large-tile launch).
  bool tails_only = false;
  // The same weights in the packed tile layout (launch_pack_weights), or NULL: the
  // large-tile kernel then reads them with the packed activations or the SwiGLU backward
  // epilogue; the streaming kernel (tails included) reads W.
  const void *W_packed = nullptr;
  // Called on the host after the large-tile launch (and its K-split sum) is enqueued,
  // before the tail launch: lets the caller mark the stream between the two.
  void (*after_main)(void *ctx) = nullptr;
  void *after_main_ctx = nullptr;
};

// Large-tile row tiles and the tail rows left to the streaming kernel.
constexpr int kBigTileRows = 256, kBigTailRows = 128;
// The tail threshold for a large-tile launch over G groups with n_out output columns: the
// streaming tail launch (one workgroup per group and 64 columns) must fill the GPU.
inline int big_tails(int G, int n_out) { return (int64_t)G * ((n_out + 63) / 64) >= 512 ? kBigTailRows : 0; }

// Device-side form of the SwiGLU backward outputs (kernel argument).
struct SwigluBwdOut {
  const uint16_t *dhp;  // bf16
  const float *row_gate;
  uint16_t *hg;        // bf16
  float *dpart;
};
hipError_t launch_grouped_gemm_bf16(const GroupedGemmArgs &a, hipStream_t s);
// Packed tile layout of grouped rows for the large-tile GEMM's A operand: per 256-row tile
// of a group (numbered over all groups in order) and 32-wide K step, a 16 KB block laid out
// as the GEMM's LDS stage; rows gathered through row_index when given.
int64_t packed_rows_bytes(int64_t rows_max, int G, int K);
// Packed tile layout of G groups' row-major weights ([rows, K] each, group stride wstride
// elements) for the large-tile kernel's B operand: per group, weight tile (256 rows: with
// SwiGLU 128 gate rows and the matching up rows, n_out apart) and 32-wide K step, one 16 KB
// block laid out as the kernel's LDS stage; rows past n_out zero.  K a multiple of 32.
int64_t packed_weights_bytes(int G, int n_out, int K, bool swiglu);
hipError_t launch_pack_weights(const void *W, int G, int64_t wstride, int n_out, int K, bool swiglu, void *out,
                               hipStream_t s);
hipError_t launch_pack_rows(const void *src, const int32_t *row_index, const int32_t *offsets, int G, int64_t rows_max,
                            int K, void *out, hipStream_t s, int tail = 0);
// Whether launch_grouped_gemm_bf16 takes the large-tile kernel (many rows per group)
// rather than the streaming one; either reads weights in both layouts (w_kn).
bool grouped_gemm_big_regime(int64_t rows_max, int num_groups, int group_rows_max);
hipError_t launch_grouped_gemm_stream_bf16(const GroupedGemmArgs &a, hipStream_t s);
hipError_t launch_grouped_gemm_big_bf16(const GroupedGemmArgs &a, int64_t rows_total_max, hipStream_t s);
hipError_t launch_grouped_gemm_f32(const GroupedGemmArgs &a, hipStream_t s);

// ---- combine (combine.hip)
hipError_t launch_combine(const void *y_perm, const int32_t *ids, const float *gates, const int32_t *slot,
                          const int32_t *offsets, const void *shared, void *out, int T, int d, int k, bool bf16,
                          hipStream_t s, int e_begin = 0, int e_end = 1 << 30);

// ---- auxiliary load-balancing loss (aux_loss.hip)
size_t aux_loss_workspace_bytes(int T, int E);
hipError_t launch_aux_loss(const float *logits, const int32_t *counts, int T, int E, int k, float alpha, float *loss,
                           float *partial_ws, hipStream_t s);

// ---- balance and z losses with their gradient (balance_loss.hip)
struct BalanceCall {
  const float *logits;
  const int32_t *ids;   // unused by the backward launch
  const uint8_t *mask;  // or NULL
  const int32_t *off;   // [S + 1] or NULL: one sequence of all T tokens (S == 1)
  const float *dloss;   // [2] or NULL
  float *dlogits;       // or NULL
  int T, E, k, S;
  float alpha, beta;
};
size_t balance_workspace_bytes(int T, int E, int S);
hipError_t launch_balance_loss(const BalanceCall &c, int32_t *counts, int32_t *seq_tokens, float *mean_probs,
                               float *losses, void *ws, hipStream_t s);
hipError_t launch_balance_backward(const BalanceCall &c, const int32_t *counts, const int32_t *seq_tokens,
                                   hipStream_t s);

// ---- gradient norm and AdamW over many tensors (optimizer.hip)
constexpr int kAdamBlock = 256;  // values that share a scale in 8-bit states
struct NormTensor {
  const void *grad;
  int64_t n;
  int32_t f32;  // 1: float, 0: bf16
  int32_t pad;
};
size_t grad_norm_workspace_bytes(const NormTensor *t, int count);
// out[0] = the norm, out[1] = min(1, max_norm / (norm + 1e-6)) from the norm in 64 bits, NaN when
// that is not finite (finite gradients of 2^33 values and less never reach it).
hipError_t launch_grad_norm(const NormTensor *t, int count, float max_norm, float *out, void *ws, hipStream_t s);
struct AdamTensor {
  void *param;
  const void *grad;
  float *master;
  void *m, *v;
  float *m_scale, *v_scale;  // 8-bit states
  int64_t n;
  float decay;       // weight decay
  uint8_t param_f32, grad_f32, eight, pad;
};
struct AdamScalars {
  double lr, beta1, beta2, eps;
  int64_t step;
  const float *lr_dev;
  const int64_t *step_dev;
  const float *grad_scale;
  int64_t *skipped;  // steps left undone so far, or NULL
};
hipError_t launch_adamw(const AdamTensor *t, int count, const AdamScalars &h, hipStream_t s);
hipError_t launch_adamw_read(const AdamTensor *t, int count, float *const *m_out, float *const *v_out, hipStream_t s);

// ---- 8-bit floating point with a scale for each block of 128 (quantize.hip, gemm_fp8.hip)
// Blocks of 128 of k values; bytes of a row's codes and of its scales (layouts in fp8.hpp).
inline constexpr int kFp8Block = 128;
__host__ __device__ inline int fp8_blocks(int k) { return (k + kFp8Block - 1) / kFp8Block; }
__host__ __device__ inline int fp8_row_bytes(int k) { return fp8_blocks(k) * kFp8Block; }
__host__ __device__ inline int fp8_scale_bytes(int k) { return (fp8_blocks(k) + 3) / 4 * 4; }
hipError_t launch_quantize_rows(const void *x, bool f32, int64_t rows, int K, uint8_t *codes, uint8_t *scale,
                                hipStream_t s);
hipError_t launch_dequantize_rows(const uint8_t *codes, const uint8_t *scale, int64_t rows, int K, void *out, bool f32,
                                  hipStream_t s);
// Bytes of one group's codes and scales.
int64_t fp8_weights_bytes(int n_out, int K, bool swiglu);
int64_t fp8_weight_scales_bytes(int n_out, int K, bool swiglu);
hipError_t launch_quantize_weights(const void *w, bool f32, int G, int n_out, int K, bool swiglu, uint8_t *codes,
                                   uint8_t *scale, hipStream_t s);
// Grouped product of rows and weights in 8 bits: out bf16 [rows_max, n_out] in y, or, with h8, the
// SwiGLU of the gate and up products in 8 bits again.  Offsets outside [0, rows_max] count as its
// ends; a row index outside [0, x_rows) as a row of zeros.
struct Fp8GemmArgs {
  const uint8_t *x8, *x_scale;
  const int32_t *row_index;  // or NULL: the rows stand in order
  const int32_t *offsets;    // [num_groups + 1]
  const uint8_t *w8, *w_scale;
  uint16_t *y;
  uint8_t *h8, *h_scale;
  int num_groups, rows_max, group_rows_max, x_rows, n_out, K;
  // Products of few tiles and a long K are cut along K: float sums [parts_cap][rows_max][fp8_part_columns()] of the parts,
  // added up by a second kernel.  1 and NULL: never.
  float *parts;
  int parts_cap;
  bool rounds;  // or, of the tiles of many rows, those past the last whole 256, in [256 parts' tiles][256][256]
  int few_chunks;  // blocks of a group of up to kFp8FewRows, set by the launch; 0: one for each column tile
  int first_block;  // of this launch, where the blocks of a product are more than one takes
  // Groups of more than kFp8FewRows go in tiles of up to 256 rows (large: a group can have that many); their rows are read
  // from xp, packed tiles of fp8_packed_bytes(), or, NULL, as they are; H goes to packed tiles.
  bool large;
  const uint8_t *xp, *xp_scale;
  uint8_t *hp, *hp_scale;
};
// A group of many rows is cut into the least number of tiles of at most kFp8LargeRows, equal but for whole 32s: the
// matrix instructions of 32 rows past a tile's end are left out, so that a group of 1040 rows costs five tiles of
// 224 and less (the last has 144), not four of 256 and a nearly empty one.
// Groups of few rows are those that one pass of the weights serves (us in the kernel for few and in tiles of 256: 32 x 24
// rows x 4096 x 4096 96 and 132, 32 x 128 117 and 154, 8 x 128 x 2048 x 7168 46.7 and 48.1); calls for groups of at most
// 16 go without LDS (FFN of 32 x 2 rows x 2880 x 2880 149 and, through LDS, 163; but 32 x 16 x 7168 x 2048 275 and 242: it is for
// decoding, where most groups have fewer rows than announced, and multiplies exactly).
constexpr int kFp8LargeRows = 256, kFp8FewRows = 128, kFp8SmallRows = 16;
__host__ __device__ inline int fp8_large_tiles(int rows) {
  return rows <= kFp8FewRows ? 0 : rows / kFp8LargeRows + (rows % kFp8LargeRows != 0);
}
__host__ __device__ inline int fp8_tile_rows(int rows, int tiles) {  // (unsigned: up to 2^31 and an eighth of it)
  return (int)(((uint32_t)rows + 32u * tiles - 1u) / (32u * tiles) * 32u);
}
// A bound on the tiles of rows in all G groups: a last one each beside whole ones, and two of 257 rows are the most for
// their number.  (Workgroups past the real tiles only leave, but each holds a CU until it has read the offsets.)
inline int64_t fp8_large_tiles_max(int64_t rows, int G) {
  const int64_t a = 2 * rows / 257, b = rows / kFp8LargeRows + G;
  return a < b ? a : b;
}
// Their bytes: codes, scales.
inline int64_t fp8_packed_bytes(int64_t rows, int G, int k) {
  return fp8_large_tiles_max(rows, G) * kFp8LargeRows * fp8_row_bytes(k);
}
inline int64_t fp8_packed_scale_bytes(int64_t rows, int G, int k) {
  return fp8_large_tiles_max(rows, G) * kFp8LargeRows * fp8_scale_bytes(k);
}
// Parts of K for `blocks` workgroups (tiles of 256 x 256 or 128 x 256, tiles_n of 256 columns to a row) on 256 CUs: the
// number, of at most `most` and in one round, with the least estimated time, in 256ths of what 512 of K (a word of
// scales) takes a tile, 5 us: a part begins and ends in two of them, its sums are written and read again in 5/256 of one
// for 256 rows, the second launch costs one; an eighth has to be won.  Evaluated alike by the product and by
// the kernel that adds the parts.  It falls with growing `blocks`.  (us whole and in parts, 1 x 100 rows x 1024 x
// 7168: 59 and 27; 300 x 4096 x 14336: 118 and 50; 4096 x 1024 x 14336: 143 and 95; 8 x 400 x 1024 x 7168: 75 and 60.)
constexpr int kFp8Parts = 16;
__host__ __device__ inline int fp8_parts(int64_t blocks, int64_t rows, int tiles_n, int k, int most) {
  const int words = fp8_scale_bytes(k) / 4;
  const int64_t sums = 5 * rows * tiles_n / 256;
  int best = 1;
  int64_t least = 224 * (words + 2);
  for (int s = 2; s <= most && s <= words && blocks * s <= 256; ++s) {
    const int64_t cost = 256 * ((words + s - 1) / s + 3) + sums * s;
    if (cost < least) {
      best = s;
      least = cost;
    }
  }
  return best;
}
inline int64_t fp8_part_columns(int n_out, bool swiglu) {
  return swiglu ? ((int64_t)n_out + 127) / 128 * 256 : ((int64_t)n_out + 255) / 256 * 256;
}
// The most parts of a product of `rows` rows in groups of `group_rows` at most, which are that many tiles at
// least (with fewer rows than announced there are no more parts than this).
inline int fp8_parts_cap(int64_t rows, int64_t group_rows, int n_out, int k, bool swiglu) {
  const int64_t per = std::max<int64_t>(std::min<int64_t>(group_rows, kFp8LargeRows), 1);
  const int tiles_n = (int)(fp8_part_columns(n_out, swiglu) / 256);
  return fp8_parts((rows + per - 1) / per * tiles_n, rows, tiles_n, k, kFp8Parts);
}
// Whether the tiles of many rows past the last whole 256 are looked at for that: K past 7168; few enough rounds; and for one
// group, whose tiles are known, only if they are cut (of several only the device knows, and the second launch follows in
// any case).  us whole and cut, n_out 4096, K 4096, 7168 and 14336: 288 tiles of one group 107 and 109, 165 and 151, 304 and
// 250; of three groups 104 and 106, 163 and 150, 308 and 258; 576 of nine 176 and 184, 275 and 266, 510 and 480; 640 of
// eight 163 and 169, 258 and 263, 483 and 495; 512 of eight, none to cut, 131 and 135, 213 and 216, 397 and 399.  So up to
// 4096 it loses, by as much as 5%, past 7168 it wins up to 18% or loses 2.5%, and between it does either.
inline bool fp8_rounds(int64_t rows, int G, int n_out, int k, bool swiglu, bool large) {
  const int64_t tiles_n = fp8_part_columns(n_out, swiglu) / 256, least = (rows + kFp8LargeRows - 1) / kFp8LargeRows * tiles_n;
  if (!large || fp8_scale_bytes(k) / 4 < 15 || least > 8 * 256) return false;
  if (G == 1) return least > 256 && least % 256 && fp8_parts(least % 256, least % 256, 256, k, kFp8Parts) > 1;
  return fp8_large_tiles_max(rows, G) * tiles_n > 256;
}
inline int64_t fp8_parts_bytes(int64_t rows, int64_t group_rows, int G, int n_out, int k, bool swiglu) {
  const int cap = fp8_parts_cap(rows, group_rows, n_out, k, swiglu);
  const bool large = (rows < group_rows ? rows : group_rows) > kFp8FewRows;
  return std::max<int64_t>(cap > 1 ? 4 * cap * rows * fp8_part_columns(n_out, swiglu) : 0,
                           fp8_rounds(rows, G, n_out, k, swiglu, large) ? 256 * 4 * kFp8LargeRows * 256 : 0);
}
// Whether the rows of large tiles are packed first: a stage of 64 of K is half of each row's line, which every column tile
// then reads twice, but packing is a launch and a copy.  us as they are and packed: 4096 x 1024 x 14336 (4
// column tiles) 83 and 99, 8 x 300 x 2048 x 2048 (8) 30 and 36, 1024 x 4096 x 4096 (16) 57 and 52, 4096 x 8192 x 14336 (32)
// 384 and 375, (56) 789 and 682.  And where groups are of few rows on average, most have no such tiles: 32 x 80 rows,
// announced as up to 320 a group, spent 4.6 us on a launch that packed nothing.
constexpr int kFp8PackTiles = 8;
inline bool fp8_packs(int64_t rows, int G, int n_out, bool swiglu) {
  return rows > (int64_t)kFp8FewRows * G && fp8_part_columns(n_out, swiglu) / 256 > kFp8PackTiles;
}
// x8 (through row_index) and its scales to packed tiles.
hipError_t launch_fp8_pack_rows(const Fp8GemmArgs &a, uint8_t *xp, uint8_t *xp_scale, hipStream_t s);
hipError_t launch_fp8_gemm(const Fp8GemmArgs &a, hipStream_t s);
hipError_t launch_fp8_gemm_rows(const Fp8GemmArgs &a, hipStream_t s);  // (its part for more than kFp8SmallRows rows a group)

// ---- root-mean-square norm (norm.hip)
struct NormCall {
  const void *x, *residual, *weight;  // residual or NULL
  void *h, *y;                        // each or NULL
  uint8_t *y8, *y_scale;              // both or NULL
  float *rstd;                        // or NULL
  int T, d;
  float eps;
  bool f32;
};
hipError_t launch_rms_norm(const NormCall &c, hipStream_t s);
struct NormBwdCall {
  const void *dy, *h, *weight, *dh;  // dh or NULL
  const float *rstd;
  void *dx;
  float *dweight;
  int T, d;
  bool f32;
};
size_t rms_norm_backward_workspace_bytes(int T, int d);
hipError_t launch_rms_norm_backward(const NormBwdCall &c, void *ws, hipStream_t s);
constexpr int kNormMaxWidth = 32768;  // values of a row

// ---- small utilities (combine.hip)
hipError_t launch_fill_i32(int32_t *p, int n, int32_t v0, int32_t step, hipStream_t s);

// ---- backward (backward.hip); bf16 activations and weights
// Plain: out[b][c][p] = in[b][p][c] for p < P, zero for p >= rows (row stride out_ld).
// Grouped (group offsets off / poff, G groups): position p of group g holds row off[g] +
// (p - poff[g]) inside the group's rows (through row_index when given), zero in its
// padding, written group-major: group g's [cols, K_g] block at poff[g] * cols, row stride
// K_g = poff[g+1] - poff[g].
hipError_t launch_transpose_bf16(const void *in, int64_t in_stride_b, int64_t rows, int cols, int batch,
                                 const int32_t *row_index, const int32_t *off, const int32_t *poff, int G, int64_t P,
                                 void *out, int64_t out_ld, int64_t out_stride_b, hipStream_t s);
// poff[g] = sum over g' < g of ceil32(off[g'+1] - off[g']), poff[G] = total
hipError_t launch_pad_offsets(const int32_t *off, int G, int32_t *poff, hipStream_t s);
hipError_t launch_fill_u32(void *p, int64_t n_words, uint32_t v, hipStream_t s);
// dl (float [T, E]) and dl16 (bf16 [T, Epad]) from the gate gradients, plus extra [T, E] (a
// gradient of other losses on the logits) unless NULL: dg of each kept
// assignment is the sum of the nb block partials [rows, nb] of its row in dpart.
hipError_t launch_gates_bwd(const int32_t *ids, const float *gates, const float *dpart, int nb, const int32_t *serving,
                            const int32_t *slot, const int32_t *offsets, int T, int E, int k, int Epad,
                            const float *extra, float *dl, void *dl16, hipStream_t s);
// row_gate[offsets[serving[i]] + slot[i]] = gates[i] for every kept assignment i < n.
hipError_t launch_row_gate(const int32_t *serving, const int32_t *slot, const int32_t *offsets, const float *gates,
                           int64_t n, float *row_gate, hipStream_t s);
// dx[t] = sum over kept j of dxr[row(t, j)], then extra[t] and extra2[t] when given (float,
// in that order); dxr holds `rows` rows.
hipError_t launch_dx_gather(const void *dxr, int64_t rows, const int32_t *serving, const int32_t *slot,
                            const int32_t *offsets, int T, int d, int k, const void *extra, const void *extra2, void *dx,
                            hipStream_t s);
// out[g][m][n] = sum over rows r in [off[g], off[g+1]) of A[r][m] B[r][n] from row-major
// (K-major) A [a_rows, M] and B [b_rows, N], bf16 out; 128 x 128 tiles for short row
// ranges, no transposes.  M, N multiples of 8; operands below 2 GiB.
hipError_t launch_wgrad_kn(const void *A, int64_t a_rows, const void *B, int64_t b_rows, const int32_t *off, int G,
                           int M, int N, void *out, hipStream_t s);
// out[i] = sum over s < S of part[s * n + i], in slice order (float, n a multiple of 4).
hipError_t launch_ksplit_sum(const float *part, int S, int64_t n, float *out, hipStream_t s);
// out[m][n] = sum over k < K of AT[m][k] B[k][n] in float for one group: AT [M, K] with row
// stride K = poff[1] - poff[0] (a multiple of 32), B [b_rows, N] row-major with rows off_b[0]
// .. off_b[1] - 1; the large-tile weight-gradient form cut along K into
// wgrad_big_f32_splits(M, N, K) slices, their partials in part (that many * M * N floats)
// added in order.  N a multiple of 8.
int wgrad_big_f32_splits(int M, int N, int64_t K);
hipError_t launch_wgrad_big_kn_f32(const void *AT, int64_t lda, const int32_t *poff, const void *B, int64_t b_rows,
                                   const int32_t *off_b, int M, int N, int64_t K, float *part, float *out,
                                   hipStream_t s);
// out[g][m][n] = sum over k < K_g of AT_g[m][k] B[off_b[g] + k][n]: AT group-major transposed
// (group g's [M, K_g] block at poff[g] * M, K_g = poff[g+1] - poff[g] a multiple of 32, zero
// padding), B [b_rows, N] row-major (K-major, unpadded; k past the group's rows reads zero);
// 256 x 256 tiles.  With `transposed` each out[g] is stored as [N, M] (out[g][n][m]).
hipError_t launch_wgrad_big_kn(const void *AT, int64_t lda, const int32_t *poff, const void *B, int64_t b_rows,
                               const int32_t *off_b, int G, int M, int N, void *out, hipStream_t s,
                               bool transposed = false);
}  // namespace moe
