/*
 * moe.h — C ABI of libmoe.so, the MI355X (gfx950) forward pass of a sparse
 * Mixture-of-Experts layer.
 *
 * Sources (web pages; cited by title and section):
 *   [SMoE]   "Sparse Mixture-of-Experts", bigdataschool.ru wiki.
 *   [HF-MoE] "Что такое Mixture of Experts (MoE) в трансформерах: архитектура и
 *            параллелизм", aglamov.biz.
 *   [GW]     "Архитектура MoE в больших языковых моделях — кто такие «эксперты»?",
 *            gerwin.io.
 *
 * The layer, per token t with hidden state x_t ([SMoE] "Роутер и top-k gating",
 * "Expert capacity и capacity factor"; [HF-MoE] "Бэкенд для экспертов"):
 *   logits_t = W_r x_t                       bias-free router linear
 *   S_t      = top-k experts of softmax(logits_t); equal logits go to the lower index
 *   g_tj     = p_t[S_tj] / sum_j' p_t[S_tj']   renormalised gates
 *   capacity C = ceil(capacity_factor * T / E); assignments are filled first come,
 *   first served in token order; overflow assignments are dropped
 *   (variants, chosen in moe_desc: a rank-major fill order, and redirection of
 *   overflow to the token's next ranked expert, [GW] "Как работает MoE: принцип
 *   маршрутизации", load-balancing item 4)
 *   y_t      = [shared expert(x_t)] + sum_{kept j} g_tj * FFN_{S_tj}(x_t)
 *   FFN_e(x) = W_d[e] (silu(W_g[e] x) * (W_u[e] x))   bias-free SwiGLU
 *
 * Conventions for every call below
 *   - Tensor pointers are DEVICE pointers unless stated otherwise; row-major;
 *     allocated and owned by the caller.  The library keeps no pointer after a
 *     call returns and never writes an input.
 *   - Calls only enqueue work on `stream` (NULL = the default stream).  They never
 *     synchronise the device and never allocate or free device memory: scratch
 *     space comes from the caller's workspace `ws` of `ws_bytes` bytes.
 *   - Arguments are validated on the host before any HIP call.  On failure the
 *     call returns a non-zero moe_status, enqueues nothing, and moe_last_error()
 *     describes the problem.  Errors raised by a kernel while it runs surface at
 *     the caller's next synchronisation.
 *   - Every device pointer must be 16-byte aligned.
 *   - Stateless and thread-safe: calls on different streams may run concurrently
 *     as long as their output and workspace buffers do not overlap.
 *   - Element types: MOE_DTYPE_F32 (float) or MOE_DTYPE_BF16 (bfloat16 stored as
 *     16-bit words) for x, all weights, expert outputs and the layer output.
 *     Router logits and gates are always float.  Accumulation is float.
 *   - bf16 layers need d_model and d_ff (and d_ff_shared) to be multiples of 64
 *     (otherwise MOE_ERR_UNSUPPORTED); f32 layers accept any positive size.
 */
#ifndef MOE_MI355X_H
#define MOE_MI355X_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_NO_CAPACITY (-1)
#define MOE_MAX_EXPERTS 1024
#define MOE_MAX_SEQS 65536                         /* sequences of one balance loss */
#define MOE_MAX_TENSOR_VALUES ((int64_t)1 << 33)   /* values of one optimizer tensor */
#define MOE_FP8_BLOCK 128                          /* values (of a row) that share a scale in 8 bits */
#define MOE_NORM_MAX_WIDTH 32768                   /* values of one row of the norm */
#define MOE_ADAMW_BLOCK 256                        /* values that share a scale in 8-bit optimizer states */

typedef enum moe_status {
  MOE_OK = 0,
  MOE_ERR_INVALID = 1,     /* bad argument: NULL/misaligned pointer, size out of range */
  MOE_ERR_UNSUPPORTED = 2, /* valid but not implemented: dtype, shape granularity */
  MOE_ERR_WORKSPACE = 3,   /* ws is NULL or ws_bytes is smaller than required */
  MOE_ERR_HIP = 4          /* a HIP runtime call or kernel launch failed */
} moe_status;

typedef enum moe_dtype { MOE_DTYPE_F32 = 0, MOE_DTYPE_BF16 = 1 } moe_dtype;

/* Order in which the capacity fill visits the assignments (t, j). */
typedef enum moe_fill_order {
  MOE_FILL_TOKEN_MAJOR = 0, /* token t before token t+1, then rank j ([SMoE] "Подводные камни ...") */
  MOE_FILL_RANK_MAJOR = 1   /* every token's rank-0 choice before any rank-1 choice, ... */
} moe_fill_order;

/* What happens to an assignment that finds its expert full. */
typedef enum moe_overflow {
  MOE_OVERFLOW_DROP = 0,   /* dropped ([SMoE] "Expert capacity и capacity factor") */
  MOE_OVERFLOW_REROUTE = 1 /* offered to the token's next ranked expert ([GW] "Как работает MoE:
                              принцип маршрутизации", item 4); see moe_dispatch_reroute */
} moe_overflow;

/* Shape of one MoE layer call. */
typedef struct moe_desc {
  int32_t num_tokens;  /* T >= 0; T == 0 makes every call but moe_balance_loss a no-op returning MOE_OK */
  int32_t d_model;     /* d >= 1 */
  int32_t d_ff;        /* f >= 1: hidden width of each routed expert */
  int32_t num_experts; /* 1 <= E <= MOE_MAX_EXPERTS */
  int32_t top_k;       /* 1 <= k <= E */
  int32_t capacity;    /* C >= 0 rows per expert, or MOE_NO_CAPACITY */
  int32_t d_ff_shared; /* 0: no shared expert; else hidden width of the always-on expert */
  int32_t dtype;       /* moe_dtype */
  int32_t fill_order;  /* moe_fill_order (0 = token-major) */
  int32_t overflow;    /* moe_overflow (0 = drop) */
} moe_desc;

/* Expert weights of one layer (device pointers).  Packed layouts follow the
 * runtime layout of [HF-MoE] "Рефакторинг загрузки весов": gate_up_proj holds,
 * per expert, the gate projection rows (w1) followed by the up projection rows
 * (w3); down_proj holds w2.  Zero-initialise the struct, so that the optional
 * fields at its end are NULL unless set. */
typedef struct moe_weights {
  const void *w_router;         /* [E, d] */
  const void *w_gate_up;        /* [E, 2f, d]: rows 0..f-1 gate, f..2f-1 up */
  const void *w_down;           /* [E, d, f] */
  const void *w_shared_gate_up; /* [2 f_s, d] or NULL when d_ff_shared == 0 */
  const void *w_shared_down;    /* [d, f_s]   or NULL when d_ff_shared == 0 */
  /* Optional, bf16 only, both or neither: w_gate_up and w_down also in the tile-major
   * layout that moe_tile_expert_weights writes (NULL: not given).  The large-tile regime of
   * the routed experts' grouped GEMMs then reads these copies -- one contiguous 16 KB
   * block per weight tile and K step instead of 256 rows of 64 bytes; w_gate_up and
   * w_down stay required (the streaming kernel reads them).  The caller keeps the two
   * forms equal.  Read by moe_forward, moe_forward_expert_shard (the range's experts) and
   * moe_backward (the recomputed gate_up projection). */
  const void *w_gate_up_tiled;
  const void *w_down_tiled;
  /* Optional, bf16 only, both or neither: the shared expert's weights in the same tile-major
   * layout (moe_tile_expert_weights with a descriptor of one expert, d_ff = d_ff_shared,
   * top_k = 1).  Read by moe_forward, moe_forward_expert_shard (with add_shared) and
   * moe_backward when the shared expert takes the large-tile regime (T >= 256). */
  const void *w_shared_gate_up_tiled;
  const void *w_shared_down_tiled;
} moe_weights;

/* Optional routing outputs of moe_forward (device pointers; any may be NULL,
 * in which case the workspace holds that table instead). */
typedef struct moe_routing {
  float *logits;           /* [T, E] */
  int32_t *topk_ids;       /* [T, k] */
  float *topk_gates;       /* [T, k] */
  int32_t *expert_counts;  /* [E]   demand per expert, before capacity */
  int32_t *expert_offsets; /* [E+1] exclusive prefix sum of kept rows per expert */
  int32_t *slot;           /* [T, k] slot inside the expert's buffer, -1 = dropped */
  int32_t *row_token;      /* [R_max] token of each kept row (rows sorted by expert, then slot) */
  int32_t *assigned_ids;   /* [T, k] expert serving each assignment: topk_ids unless redirected */
} moe_routing;

/* ---------------------------------------------------------------- host helpers */

/* Expert capacity ceil(capacity_factor * T / E), evaluated in IEEE double in that
 * order ([SMoE] "Expert capacity и capacity factor").  Returns MOE_NO_CAPACITY
 * when capacity_factor <= 0 or is not finite; returns 0 for T < 0 or E < 1; values
 * above INT32_MAX are clamped to INT32_MAX.  Host only, no device access. */
int32_t moe_capacity(int32_t num_tokens, int32_t num_experts, double capacity_factor);

/* Capacity variant with a top-k factor, ceil(capacity_factor * (k * T) / E) in IEEE
 * double: the batch counted in assignments rather than tokens.  Same special cases
 * as moe_capacity; k < 1 returns 0.  Host only. */
int32_t moe_capacity_topk(int32_t num_tokens, int32_t num_experts, int32_t top_k, double capacity_factor);

/* Upper bound R_max on kept rows: min(T*k, E*C), or T*k without capacity.
 * Returns -1 for an invalid descriptor. */
int64_t moe_max_rows(const moe_desc *desc);

/* Workspace bytes needed by moe_forward for this descriptor (enough for every
 * other call with the same descriptor too).  Returns 0 for an invalid descriptor. */
size_t moe_workspace_size(const moe_desc *desc);

/* Workspace bytes needed by moe_grouped_swiglu_gemm. Returns 0 on invalid input. */
size_t moe_grouped_gemm_workspace_size(int32_t num_groups, int64_t rows_max, int32_t d_ff, int32_t dtype);

const char *moe_status_string(moe_status status);

/* Detail of the last failure in the calling thread ("" if none). */
const char *moe_last_error(void);

/* The ids precondition of moe_dispatch_permute, moe_dispatch_reroute and
 * moe_combine_unpermute, checked on a HOST copy of the ids ([SMoE] "Роутер и top-k
 * gating": each id names one of the E experts): every topk_ids_host[t][j], [T, k] int32,
 * lies in [0, E).  Returns MOE_OK, or MOE_ERR_INVALID with moe_last_error() naming the
 * first entry outside the range.  Host only, no device access.
 * Release builds do not check ids on the device: an id outside [0, E) is treated as no
 * expert (slot -1, not counted, never indexes a table).  The debug build of the library
 * (libmoe_debug.so, compiled with MOE_DEBUG_CHECKS) runs this check inside those three
 * calls on a synchronous copy of the device ids, before it enqueues any work, and returns
 * its MOE_ERR_INVALID. */
moe_status moe_check_topk_ids(const moe_desc *desc, const int32_t *topk_ids_host);

/* 1 in the debug build (MOE_DEBUG_CHECKS: host checks of device-side preconditions, which
 * synchronise the stream), 0 otherwise. */
int32_t moe_debug_checks(void);

/* ---------------------------------------------------------------- hot path */

/* Router linear ([SMoE] "Роутер и top-k gating": logits from a linear layer
 * without bias).
 *   x           [T, d] dtype
 *   w_router    [E, d] dtype
 *   logit_offset [E] float or NULL: added to every token's logits (synthetic skew)
 *   logits      [T, E] float, written.  Accumulated in float. */
moe_status moe_router_logits(const moe_desc *desc, const void *x, const void *w_router,
                             const float *logit_offset, float *logits, hipStream_t stream);

/* Softmax over experts, top-k and renormalised gates ([SMoE] "Роутер и top-k
 * gating").  Selection ranks the logits (softmax is increasing); equal logits go
 * to the lower expert index, and -0.0 equals +0.0.  Logits must be finite or -inf.
 *   logits     [T, E] float
 *   topk_ids   [T, k] int32, written in descending logit order
 *   topk_gates [T, k] float, written: exp(l_j - l_max) / sum over the k selected */
moe_status moe_router_topk(const moe_desc *desc, const float *logits, int32_t *topk_ids,
                           float *topk_gates, hipStream_t stream);

/* Capacity-limited dispatch ([SMoE] "Expert capacity и capacity factor",
 * "Подводные камни collapse экспертов и token dropping"; [HF-MoE] "Бэкенд для
 * экспертов": tokens sorted by expert id before one grouped GEMM).
 * Walking assignments (t, j) in desc->fill_order (token-major: t outer, j inner;
 * rank-major: j outer, t inner), each takes the next free slot of its expert while
 * fewer than C are taken; later ones are dropped.  desc->overflow must be
 * MOE_OVERFLOW_DROP (MOE_ERR_INVALID otherwise; redirection is moe_dispatch_reroute).
 *   topk_ids       [T, k] int32, each in [0, E) (precondition; see moe_check_topk_ids: an id
 *                  outside the range is treated as dropped, slot -1, and not counted)
 *   x              [T, d] dtype, or NULL when x_perm is NULL
 *   expert_counts  [E]   int32, written: demand per expert
 *   expert_offsets [E+1] int32, written: offsets[0] = 0, offsets[e+1] - offsets[e] =
 *                  min(counts[e], C)
 *   slot           [T, k] int32, written: slot in the expert's buffer or -1 if dropped
 *   row_token      [R_max] int32, written for rows < offsets[E]: the row's token; the rows
 *                  of an expert are in slot order (its assignments in fill order)
 *   x_perm         [R_max, d] dtype or NULL: row offsets[e] + slot(t, j) = x[t];
 *                  rows >= offsets[E] are left unspecified
 *   ws             at least moe_workspace_size(desc) bytes */
moe_status moe_dispatch_permute(const moe_desc *desc, const int32_t *topk_ids, const void *x,
                                int32_t *expert_counts, int32_t *expert_offsets, int32_t *slot,
                                int32_t *row_token, void *x_perm, void *ws, size_t ws_bytes,
                                hipStream_t stream);

/* Capacity-limited dispatch with redirection of overflow ([GW] "Как работает MoE:
 * принцип маршрутизации", load-balancing item 4: an assignment beyond an expert's
 * capacity may be sent on to the next most suitable expert instead of dropped).
 * Two passes, both in desc->fill_order:
 *   1. the plain fill of moe_dispatch_permute: kept assignments are exactly those
 *      of the drop policy;
 *   2. the i-th overflowing assignment of token t (i counted in rank order j) is
 *      offered to the expert ranked k + i in t's router order (descending logit,
 *      equal logits to the lower index); offers take the next free slot of that
 *      expert while it has room left after pass 1, otherwise (or if k + i >= E)
 *      they are dropped.  Each expert's rows: its pass-1 rows, then its offers.
 * Gates are not changed: a redirected assignment keeps its gate.  Without capacity
 * nothing overflows and the result is that of moe_dispatch_permute.
 *   logits         [T, E] float (the router's, as given to moe_router_topk)
 *   topk_ids       [T, k] int32 as written by moe_router_topk from those logits
 *   expert_counts  [E]   int32, written: the router's demand per expert (pass 1)
 *   expert_offsets [E+1] int32, written: exclusive prefix of the final kept rows
 *   slot           [T, k] int32, written: slot in the serving expert's buffer, or -1
 *   assigned_ids   [T, k] int32, written: serving expert (topk_ids[t][j] unless
 *                  redirected; for a dropped assignment, topk_ids[t][j])
 *   row_token      [R_max] int32, written for rows < offsets[E]
 *   ws             at least moe_workspace_size(desc) bytes
 * Pass assigned_ids as the ids of moe_combine_unpermute.  desc->overflow is not
 * consulted. */
moe_status moe_dispatch_reroute(const moe_desc *desc, const float *logits, const int32_t *topk_ids,
                                int32_t *expert_counts, int32_t *expert_offsets, int32_t *slot,
                                int32_t *assigned_ids, int32_t *row_token, void *ws, size_t ws_bytes,
                                hipStream_t stream);

/* Grouped SwiGLU expert FFN over rows sorted by group ([HF-MoE] "Бэкенд для
 * экспертов": one grouped GEMM over tokens sorted by expert id; [HF-MoE]
 * "Рефакторинг загрузки весов": packed gate_up / down layouts).
 * For every group g and row r in [group_offsets[g], group_offsets[g+1]):
 *   y_rows[r] = W_d[g] (silu(W_g[g] x_rows[r]) * (W_u[g] x_rows[r]))
 * The hidden activation is rounded to dtype between the two projections.
 *   num_groups      G >= 1 (<= MOE_MAX_EXPERTS)
 *   rows_max        rows available in x_rows / y_rows; group_offsets[G] <= rows_max
 *   group_rows_max  the caller's bound on any one group's rows (a tiling hint: larger
 *                   groups are still computed correctly); >= 1
 *   x_rows          [rows_max, d] dtype
 *   group_offsets   [G+1] int32 DEVICE array, non-decreasing, group_offsets[0] >= 0
 *   w_gate_up       [G, 2f, d] dtype;  w_down [G, d, f] dtype
 *   y_rows          [rows_max, d] dtype, written for rows inside a group
 *   ws              at least moe_grouped_gemm_workspace_size(G, rows_max, f, dtype) */
moe_status moe_grouped_swiglu_gemm(int32_t num_groups, int64_t rows_max, int32_t group_rows_max,
                                   int32_t d_model, int32_t d_ff, int32_t dtype, const void *x_rows,
                                   const int32_t *group_offsets, const void *w_gate_up,
                                   const void *w_down, void *y_rows, void *ws, size_t ws_bytes,
                                   hipStream_t stream);

/* The two halves of moe_grouped_swiglu_gemm as single launches (same contracts; same
 * sources; no workspace):
 *   moe_grouped_gate_up_swiglu: h_rows[r] = silu(W_g[g] a_r) * (W_u[g] a_r), h_rows
 *     [rows_max, f] dtype (rounded to dtype), where a_r = x_rows[r], or, when row_index
 *     is not NULL, a_r = x_rows[row_index[r]] with x_rows holding x_row_count rows (a
 *     row gather: the dispatch's row_token lets the projection read token rows straight
 *     from x, so x_perm need not exist; x_rows must then be < 2 GiB);
 *   moe_grouped_down: y_rows[r] = W_d[g] h_rows[r], y_rows [rows_max, d] dtype. */
moe_status moe_grouped_gate_up_swiglu(int32_t num_groups, int64_t rows_max, int32_t group_rows_max, int32_t d_model,
                                      int32_t d_ff, int32_t dtype, const void *x_rows, const int32_t *row_index,
                                      int64_t x_row_count, const int32_t *group_offsets, const void *w_gate_up,
                                      void *h_rows, hipStream_t stream);
moe_status moe_grouped_down(int32_t num_groups, int64_t rows_max, int32_t group_rows_max, int32_t d_model,
                            int32_t d_ff, int32_t dtype, const void *h_rows, const int32_t *group_offsets,
                            const void *w_down, void *y_rows, hipStream_t stream);

/* Gate-weighted combine back to token order, without atomics ([SMoE] "Роутер и
 * top-k gating": weighted sum of the selected experts' outputs; "Expert capacity и
 * capacity factor": a dropped assignment contributes nothing; [GW] drawbacks item
 * 5: shared expert added with weight 1).
 *   out[t] = shared_out[t] (or 0) + sum_{j: slot[t,j] >= 0} topk_gates[t,j] *
 *            y_perm[expert_offsets[topk_ids[t,j]] + slot[t,j]], summed in float in
 *            order j = 0..k-1, then rounded to dtype.
 *   topk_ids: the expert serving each assignment -- the router's ids, or the
 *   assigned_ids of moe_dispatch_reroute when overflow is redirected; each in [0, E)
 *   (precondition, see moe_check_topk_ids: an id outside the range adds nothing).
 *   y_perm [R_max, d] dtype; shared_out [T, d] dtype or NULL; out [T, d] dtype */
moe_status moe_combine_unpermute(const moe_desc *desc, const void *y_perm, const int32_t *topk_ids,
                                 const float *topk_gates, const int32_t *slot,
                                 const int32_t *expert_offsets, const void *shared_out, void *out,
                                 hipStream_t stream);

/* Switch-style auxiliary load-balancing loss ([SMoE] "Маршрутизация токена и auxiliary
 * loss"): loss = alpha * E * sum_i f_i * P_i, where f_i = expert_counts[i] / (T * k) is
 * the share of the batch's assignments routed to expert i (router choice, before
 * capacity) and P_i the softmax probability of expert i averaged over the T tokens.
 * For k = 1 this is the page's formula; uniform routing gives alpha.
 *   logits        [T, E] float (as written by moe_router_logits)
 *   expert_counts [E] int32 (as written by moe_dispatch_permute)
 *   loss          [1] float, written (device)
 *   ws            at least moe_workspace_size(desc) bytes
 * Float accumulation in fixed orders: bit-reproducible.  A value to report; moe_balance_loss
 * has the gradient, and counts for itself. */
moe_status moe_router_aux_loss(const moe_desc *desc, const float *logits, const int32_t *expert_counts, float alpha,
                               float *loss, void *ws, size_t ws_bytes, hipStream_t stream);

/* The whole layer: router linear, top-k, dispatch, routed grouped SwiGLU FFN, the
 * shared expert if desc->d_ff_shared > 0, and combine.  The dispatch follows
 * desc->fill_order and desc->overflow (moe_dispatch_permute or moe_dispatch_reroute).
 *   x [T, d] dtype, smaller than 2 GiB; logit_offset [E] float or NULL; out [T, d] dtype
 *   routing: NULL, or a struct whose non-NULL fields receive the routing tables
 *   ws: at least moe_workspace_size(desc) bytes
 * Only kernel launches on `stream` (no host synchronisation, allocation or memset): the
 * call can be captured into a HIP graph.  Deterministic: equal inputs give bitwise equal
 * outputs and routing tables. */
moe_status moe_forward(const moe_desc *desc, const moe_weights *weights, const void *x,
                       const float *logit_offset, void *out, moe_routing *routing, void *ws,
                       size_t ws_bytes, hipStream_t stream);

/* Bytes of the fixed scratch array behind moe_forward_noalloc (per GPU). */
#define MOE_NOALLOC_WORKSPACE_BYTES (128u << 20)

/* For callers that cannot allocate device memory -- code under HIP graph capture, tight
 * serving loops, harnesses that forbid allocation: moe_forward with its workspace taken
 * from a fixed array of MOE_NOALLOC_WORKSPACE_BYTES that the library holds on each GPU it
 * runs on (until the process ends), instead of a caller workspace.  No allocation: the
 * call neither allocates nor frees device memory.  Layers whose moe_workspace_size
 * exceeds MOE_NOALLOC_WORKSPACE_BYTES fail with MOE_ERR_WORKSPACE before any launch (e.g.
 * decode steps and Switch-style layers fit; the Mixtral- and DeepSeek-shaped layers do
 * not).  Every call on one GPU uses that GPU's one array: calls that overlap in time on
 * the same GPU (different streams or threads without ordering) race and give undefined
 * results; calls ordered on one stream are fine.  Nothing in the array has to start at
 * zero (every kernel writes what it reads back).  The first call on a device resolves
 * that device's array address with that device current.  Arguments, results and other
 * errors as for moe_forward. */
moe_status moe_forward_noalloc(const moe_desc *desc, const moe_weights *weights, const void *x,
                               const float *logit_offset, void *out, moe_routing *routing,
                               hipStream_t stream);

/* Stages of moe_forward in launch order, as moe_forward_staged marks them. */
typedef enum moe_stage {
  MOE_STAGE_ROUTER = 0,                /* router linear and top-k (the next k ranks too when redirecting) */
  MOE_STAGE_DISPATCH = 1,              /* capacity fill: counts, offsets, slots, row order */
  MOE_STAGE_PACK_ROWS = 2,             /* large-tile regime: gathered x rows copied to the packed tile layout */
  MOE_STAGE_GATE_UP = 3,               /* routed gate_up + SwiGLU grouped GEMM, main launch */
  MOE_STAGE_GATE_UP_TAILS = 4,         /* large-tile regime: the groups' tail rows, streaming launch */
  MOE_STAGE_DOWN = 5,                  /* routed down grouped GEMM, main launch (and its K-split sum) */
  MOE_STAGE_DOWN_TAILS = 6,            /* large-tile regime: tail rows of the down projection */
  MOE_STAGE_SHARED_PACK_ROWS = 7,      /* shared expert: its row offsets (large-tile regime), packed x rows */
  MOE_STAGE_SHARED_GATE_UP = 8,        /* shared expert gate_up + SwiGLU, main launch */
  MOE_STAGE_SHARED_GATE_UP_TAILS = 9,  /* shared expert: tail rows */
  MOE_STAGE_SHARED_DOWN = 10,          /* shared expert down projection, main launch */
  MOE_STAGE_SHARED_DOWN_TAILS = 11,    /* shared expert: tail rows of the down projection */
  MOE_STAGE_COMBINE = 12,              /* gate-weighted combine into out */
  MOE_NUM_STAGES = 13
} moe_stage;

/* moe_forward with HIP events recorded on `stream` between its launches, so that a caller
 * can time each stage of the very launches moe_forward makes (same kernels, arguments and
 * order; the records add only event markers to the stream).
 *   stage_events  host array of MOE_NUM_STAGES + 1 events created by the caller (hipEventCreate,
 *                 timing enabled): stage_events[0] is recorded before the first launch and
 *                 stage_events[s + 1] after the launches of stage s; a stage that launches
 *                 nothing (absent shared expert, streaming regime without tails, ...) ends where
 *                 the previous one ended.  NULL entries: MOE_ERR_INVALID.
 * Other arguments, results and errors as for moe_forward. */
moe_status moe_forward_staged(const moe_desc *desc, const moe_weights *weights, const void *x,
                              const float *logit_offset, void *out, moe_routing *routing, void *ws,
                              size_t ws_bytes, hipStream_t stream, hipEvent_t *stage_events);

/* Weight gradients of moe_backward (device pointers). */
typedef struct moe_grads {
  void *dw_router;         /* [E, d] float */
  void *dw_gate_up;        /* [E, 2f, d] dtype: gate rows then up rows, as w_gate_up */
  void *dw_down;           /* [E, d, f] dtype */
  void *dw_shared_gate_up; /* [2 f_s, d] dtype, or NULL when d_ff_shared == 0 */
  void *dw_shared_down;    /* [d, f_s]   dtype, or NULL when d_ff_shared == 0 */
} moe_grads;

/* Workspace bytes needed by moe_backward; 0 for an invalid or unsupported descriptor. */
size_t moe_backward_workspace_size(const moe_desc *desc);

/* Backward pass of the layer: gradients of L = sum(dy * out) for the out of moe_forward,
 * with the routing held fixed (top-k choice, slots and drops are piecewise constant;
 * [HF-MoE] "Обучение MoE с помощью Transformers": in training the expert projections
 * run as grouped GEMMs too).  Per kept row of expert e with gate g:
 *   dH' = dy W_d[e];  dg = dH' . H;  [dG dU] from g dH' through SwiGLU;
 *   dx += [dG dU] W_gu[e];  dW_d[e] += (g dy) (x) H;  dW_gu[e] += [dG dU] (x) x;
 * gates (softmax over the selected logits): dl_j = g_j (dg_j - sum g dg), dW_r = dl^T x,
 * dx += dl W_r; the shared expert likewise with g = 1 for every token.  Experts without
 * kept rows get zero gradients.  bf16 layers only (MOE_ERR_UNSUPPORTED otherwise).
 *   x, dy      [T, d] dtype (the forward's input; the loss gradient w.r.t. out)
 *   routing    the tables moe_forward wrote for x: topk_ids, topk_gates, expert_offsets,
 *              slot, row_token (and assigned_ids when desc->overflow redirects) are read
 *   dx         [T, d] dtype, written
 *   grads      written in full (see moe_grads)
 *   ws         at least moe_backward_workspace_size(desc) bytes
 * Accumulation in float; every sum in a fixed order (bit-reproducible).  Only kernel
 * launches on `stream` (capturable into a HIP graph). */
moe_status moe_backward(const moe_desc *desc, const moe_weights *weights, const void *x, const moe_routing *routing,
                        const void *dy, void *dx, moe_grads *grads, void *ws, size_t ws_bytes, hipStream_t stream);

/* moe_backward with a gradient on the router's logits added to the gates': the losses that
 * depend on the logits themselves (moe_balance_loss) reach dw_router and dx this way.
 *   dlogits [T, E] float (as moe_balance_loss or moe_balance_loss_backward writes it)
 * The sum dl is rounded to bf16 for the two products with it, as in moe_backward.  Other
 * arguments, results and errors as for moe_backward; dlogits of zeros gives its results. */
moe_status moe_backward_with_dlogits(const moe_desc *desc, const moe_weights *weights, const void *x,
                                     const moe_routing *routing, const void *dy, const float *dlogits, void *dx,
                                     moe_grads *grads, void *ws, size_t ws_bytes, hipStream_t stream);

/* ------------------------------------------------------------- balance loss with gradient */

/* Workspace bytes of moe_balance_loss; 0 for an invalid descriptor or num_seqs. */
size_t moe_balance_workspace_size(const moe_desc *desc, int32_t num_seqs);

/* Load-balancing loss ([SMoE] "Маршрутизация токена и auxiliary loss") sequence by sequence,
 * the router's z loss, per-expert counts and, if asked for, the gradient of their sum on the
 * logits, all in one pass over the logits.  With N_s the counted tokens of sequence s, N
 * those of all sequences and S' the sequences that count any:
 *   c_si = assignments of counted tokens to expert i (router choice, before capacity)
 *   f_si = c_si / (k N_s),  P_si = 1/N_s sum_t softmax(l_t)_i,  z_t = log sum_i exp(l_ti)
 *   losses[0] = alpha E / S' sum_s sum_i f_si P_si
 *   losses[1] = z_coeff / N sum_t z_t^2
 *   dlogits_ti = p_ti (alpha E / (S' N_s) (f_si - sum_j f_sj p_tj) + 2 z_coeff / N z_t)
 * (f held fixed: counts are piecewise constant).  One sequence of all tokens gives
 * moe_router_aux_loss's value: that call takes counts that the dispatch has written and gives
 * the value alone, to report; this one counts for itself and is the one to train with.  Of a
 * valid descriptor only num_tokens, num_experts and top_k matter.
 *   logits      [T, E] float; -inf is an expert with probability 0; a counted token with
 *               no finite logit has no probabilities: it adds nothing to P and the z loss
 *               and gets a zero gradient (its ids are counted)
 *   topk_ids    [T, k] int32; ids outside [0, E) are not counted
 *   token_mask  [T] uint8 or NULL: zero = not counted (padding); its logits may hold
 *               anything, NaN included
 *   seq_offsets [num_seqs + 1] int32 or NULL (one sequence of all T tokens, num_seqs 1):
 *               non-decreasing within [0, T] (precondition; checked by the debug build,
 *               which synchronises the stream; others read and write nothing out of range
 *               but give no meaningful result); sequence s holds tokens
 *               seq_offsets[s] .. seq_offsets[s + 1] - 1, possibly none; tokens before the
 *               first and behind the last sequence are not counted
 *   counts      [num_seqs, E] int32, written
 *   seq_tokens  [num_seqs] int32, written: N_s
 *   mean_probs  [num_seqs, E] float, written: P (zeros where N_s is 0)
 *   losses      [2] float, written; 0 when nothing is counted
 *   dlogits     [T, E] float or NULL, written in full: zero for tokens not counted; not
 *               overlapping logits (refused)
 *   ws          at least moe_balance_workspace_size(desc, num_seqs) bytes
 * An empty batch (T == 0) writes zeros to counts, seq_tokens, mean_probs and losses, and
 * looks at no other pointer.  Sums in fixed orders (bit-reproducible).  Only kernel launches on `stream`. */
moe_status moe_balance_loss(const moe_desc *desc, const float *logits, const int32_t *topk_ids,
                            const uint8_t *token_mask, const int32_t *seq_offsets, int32_t num_seqs, float alpha,
                            float z_coeff, int32_t *counts, int32_t *seq_tokens, float *mean_probs, float *losses,
                            float *dlogits, void *ws, size_t ws_bytes, hipStream_t stream);

/* The gradient alone, for upstream gradients known only after the forward pass:
 *   dlogits = dloss[0] * d losses[0] / d logits + dloss[1] * d losses[1] / d logits
 *   counts, seq_tokens  as moe_balance_loss wrote them
 *   dloss               [2] float (device) or NULL (both 1); whatever they hold, a token that
 *                       is not counted or has no finite logit gets zeros
 *   dlogits             [T, E] float, written in full; not overlapping logits (refused)
 * Other arguments as for moe_balance_loss; no workspace. */
moe_status moe_balance_loss_backward(const moe_desc *desc, const float *logits, const uint8_t *token_mask,
                                     const int32_t *seq_offsets, int32_t num_seqs, const int32_t *counts,
                                     const int32_t *seq_tokens, float alpha, float z_coeff, const float *dloss,
                                     float *dlogits, hipStream_t stream);

/* --------------------------------------------------------- gradient norm and AdamW step */

/* One gradient tensor of n values (0 <= n <= MOE_MAX_TENSOR_VALUES). */
typedef struct moe_grad_view {
  const void *grad; /* [n] dtype (device); may be NULL when n == 0 */
  int64_t n;
  int32_t dtype; /* moe_dtype */
  int32_t reserved;
} moe_grad_view;

/* Workspace bytes of moe_grad_norm for these tensors; 0 for invalid ones.  Host only. */
size_t moe_grad_norm_workspace_size(const moe_grad_view *grads, int32_t num_tensors);

/* Norm over every value of every tensor, and the factor that clips it:
 *   out[0] = sqrt(sum g^2),  out[1] = min(1, max_norm / (out[0] + 1e-6))
 * summed in 64 bits in a fixed order.  Where a gradient is not finite out[1] = NaN, which
 * moe_adamw_step takes as "leave everything as it is".  Finite gradients whose norm is past
 * the largest float have infinity in out[0] and their factor in out[1] all the same (g' is
 * finite, the step is made): out[1] alone tells.  out stays on the device:
 * moe_adamw_hparams.norm takes it as it is.
 *   grads     HOST array of num_tensors views (read during the call only)
 *   max_norm  above 0; infinity: no clipping
 *   out       [2] float, written
 *   ws        at least moe_grad_norm_workspace_size(grads, num_tensors) bytes
 * Only kernel launches on `stream`. */
moe_status moe_grad_norm(const moe_grad_view *grads, int32_t num_tensors, float max_norm, float *out, void *ws,
                         size_t ws_bytes, hipStream_t stream);

/* One parameter tensor of n values with its gradient and optimizer state (device pointers).
 * States in 8 bits: each MOE_ADAMW_BLOCK consecutive values (the last block may hold fewer)
 * share one float scale, the block's largest magnitude; a code c of m (int8) stands for
 * m_scale c |c| / 127^2, a code c of v (uint8) for v_scale (c / 255)^4.  Each takes the code
 * whose value (for v: whose value's root) is nearest, and a v above zero one at least.  m'
 * and v' are formed and compared in 64 bits, every operation of the formulas rounded by
 * itself (m_scale * (1 / 127^2) and v_scale * (1 / 255^4) first), so that codes and scales
 * are the same for any program that follows them.  A block whose largest is below the
 * smallest normal float is held as zeros; one with a value that is not finite gets a NaN
 * scale, with which all its values count as NaN from the next step on.  Zeros everywhere are
 * the initial state of both forms.
 * Take beta2 <= 0.98 with states in 8 bits.  Rounding to the nearest code undoes a step's
 * change that is below half the way to the next one: while its block's scale stays, a v of
 * code c without gradients falls only if beta2 < (1 - 1 / c + 1 / (2 c^2))^2 (0.95: c >= 39,
 * v above 5e-4 of the block's largest; 0.99: c >= 199; 0.9922 and above: never), and it rises
 * only at gradients whose square is some 1 + 2 / (c (1 - beta2)) times v.  Simulated against
 * states in 32 bits, sqrt(v') of stationary gradients is in the median the same up to beta2 =
 * 0.99; with 0.999 it is 1.5 times too high in a block of equal variances, and 4 times too
 * high 3000 steps after half of a block's gradients fell to a tenth (0.98: 1.01 times).  m
 * with beta1 = 0.9 falls from c = 10 on, 0.6% of its block's largest. */
typedef struct moe_adamw_tensor {
  void *param;      /* [n] param_dtype, updated */
  const void *grad; /* [n] grad_dtype */
  float *master;    /* [n] float copy of a bf16 parameter, updated, with param its rounding
                       (param is not read then); NULL: none -- the bf16 value itself is updated
                       and rounded to nearest, so that steps below half its last place are lost */
  void *m, *v;      /* [n] float, or int8 / uint8 codes; updated */
  float *m_scale;   /* [ceil(n / MOE_ADAMW_BLOCK)] for 8-bit states; unused otherwise */
  float *v_scale;
  int64_t n;           /* 0 <= n <= MOE_MAX_TENSOR_VALUES; 0: the tensor is passed over */
  int32_t param_dtype; /* moe_dtype; MOE_DTYPE_F32 takes no master */
  int32_t grad_dtype;  /* moe_dtype */
  int32_t state_bits;  /* 32 or 8 */
  float weight_decay;  /* finite, >= 0 */
} moe_adamw_tensor;

typedef struct moe_adamw_hparams {
  double lr, beta1, beta2, eps; /* lr >= 0; betas in [0, 1); eps a normal float above 0 */
  int64_t step;                 /* t >= 1, the number of this step */
  /* Optional device scalars, read when the step runs (a captured step then follows them on
   * every replay): lr and t in the place of the two fields above (a t below 1 counts as 1),
   * and moe_grad_norm's `out`, whose out[1] every gradient is multiplied by.  When out[1] is
   * NaN the step leaves every tensor as it is. */
  const float *lr_dev;     /* [1] or NULL */
  const int64_t *step_dev; /* [1] or NULL */
  const float *norm;       /* [2] or NULL */
  /* How many of the steps so far were left undone so (device): t is the step's number less
   * this (1 at least), so that the bias corrections count the updates that m and v have seen,
   * and a step left undone adds one to it.  NULL: t is the step's number. */
  int64_t *skipped; /* [1] or NULL */
} moe_adamw_hparams;

/* The conditions on a list of tensors that moe_adamw_step checks (pointers, alignment,
 * types, sizes), and that no buffer that the step writes overlaps another buffer of the
 * list.  Host only, no device access.  moe_adamw_step itself checks this last only among
 * the parameters (the same tensor twice), in the debug build in full. */
moe_status moe_adamw_check_tensors(const moe_adamw_tensor *tensors, int32_t num_tensors);

/* One AdamW step (decoupled weight decay) of every tensor, 64 tensors (8-bit states: 48) a
 * launch:
 *   g' = out[1] g;  m' = b1 m + (1 - b1) g';  v' = b2 v + (1 - b2) g'^2
 *   w' = w (1 - lr wd) - lr / (1 - b1^t) m' / (sqrt(v') / sqrt(1 - b2^t) + eps)
 * in float (8-bit states: m' and v' in 64 bits), w' rounded once to param_dtype.
 * A gradient that is not finite makes its value's state and parameter so.  Values past n
 * are not touched.  Tile-major weight copies are the caller's to rewrite
 * (moe_tile_expert_weights).
 *   tensors  HOST array of num_tensors descriptors (read during the call only)
 * Only kernel launches on `stream`. */
moe_status moe_adamw_step(const moe_adamw_tensor *tensors, int32_t num_tensors, const moe_adamw_hparams *hparams,
                          hipStream_t stream);

/* 8-bit states as the floats they stand for (checkpoints, inspection).
 *   tensors  as for moe_adamw_step, every one with state_bits 8; param, grad and master are
 *            not looked at
 *   m_out, v_out  HOST arrays of num_tensors device pointers to [n] float; NULL (the array or
 *            an entry): not wanted */
moe_status moe_adamw_read_states(const moe_adamw_tensor *tensors, int32_t num_tensors, float *const *m_out,
                                 float *const *v_out, hipStream_t stream);

/* ------------------------------------------------- 8-bit floating point, norm, 8-bit experts */

/* Rows in 8 bits.  Codes are e4m3 (largest 448, one NaN, no infinity), scales powers of two held
 * as a byte, exponent + 127 (255: NaN); each MOE_FP8_BLOCK consecutive values of a row share one:
 *   value[r][k] = code[r][k] * 2^(scale[r][k / 128] - 127)
 *   codes [rows, moe_fp8_row_bytes(K)] uint8, ZERO behind column K
 *   scale [rows, moe_fp8_scale_bytes(K)] uint8, a byte for each 128 columns; the bytes behind
 *         the last block pad the row to a multiple of four and are not looked at
 * The quantising calls take the least scale with which the block's largest finite magnitude is at
 * most 448 (at least 2^-126; 1 for a block of zeros), so that no finite value saturates, and for
 * each value the nearest code, ties to the even one; a value that is not finite gets the NaN
 * code and has no part in the scale.  Powers of two, because the matrix instructions of gfx950
 * apply them for nothing; against a float scale they cost no precision but that of values far
 * below their block's largest (e4m3 is a floating format).  Both helpers: host only; 0 for K < 1. */
int32_t moe_fp8_row_bytes(int32_t k);
int32_t moe_fp8_scale_bytes(int32_t k);

/* Rows to 8 bits.  x [rows, K] dtype; codes, scale as above, written in full (codes behind
 * column K zeros, padding scales ones).  0 <= rows <= INT32_MAX, 1 <= K < 2^24. */
moe_status moe_quantize_rows_fp8(int64_t rows, int32_t k, int32_t dtype, const void *x, uint8_t *codes, uint8_t *scale,
                                 hipStream_t stream);

/* The values that codes stand for.  out [rows, K] dtype, written (bf16: exact but for values
 * past its range). */
moe_status moe_dequantize_rows_fp8(int64_t rows, int32_t k, int32_t dtype, const uint8_t *codes, const uint8_t *scale,
                                   void *out, hipStream_t stream);

/* Weights of num_groups matrices in 8 bits, a scale for each 128 x 128 block, in the layout that
 * the products read (written once, when weights are loaded).  swiglu 0: w [G, n_out, K];
 * 1: w [G, 2 n_out, K], gate rows then up rows (moe_weights.w_gate_up with n_out = f), whose
 * blocks are those of the gate rows and of the up rows apart.
 *   codes  per group, blocks of 16 rows (swiglu: gate and up blocks in turn), B in all, in tiles of 16
 *          blocks (the last one of the b <= 16 left): tile t begins at byte 16 t ceil(K / 128) 2048 and holds,
 *          ordered [ceil(K / 128)][2][b], pieces of 1 KB, 16 rows by 64 of K, in which byte
 *          256 c + 16 r + i is row r, k = 16 c + i of the 64; zeros where the matrix has ended
 *   scale  per group [ceil(n_out / 128)][moe_fp8_scale_bytes(K)] (swiglu: [ceil(n_out / 128)][2][...])
 * Sizes in bytes from the two helpers (host only; 0 for invalid arguments).  Scales and codes
 * as for rows.  One group's codes must be below 2 GiB, n_out and k below 2^23
 * (MOE_ERR_UNSUPPORTED). */
size_t moe_fp8_weights_bytes(int32_t num_groups, int32_t n_out, int32_t k, int32_t swiglu);
size_t moe_fp8_weight_scales_bytes(int32_t num_groups, int32_t n_out, int32_t k, int32_t swiglu);
moe_status moe_quantize_weights_fp8(int32_t num_groups, int32_t n_out, int32_t k, int32_t swiglu, int32_t dtype,
                                    const void *w, uint8_t *codes, uint8_t *scale, hipStream_t stream);

/* Root-mean-square norm of the residual stream in front of a layer:
 *   h = x + residual, rounded to dtype (x itself without a residual)
 *   rstd = 1 / sqrt(mean of h^2 over the row + eps), the mean formed in 64 bits
 *   y = (h rstd) weight, in float; y rounded to dtype, and y8 quantised from the float
 *   x, residual  [T, d] dtype; residual may be NULL
 *   weight       [d] dtype
 *   eps          finite, >= 0 (with eps 0 a row of zeros gives NaN, and one whose root mean square is below 2^-128, so that
 *                rstd passes the floats, infinities)
 *   h            [T, d] dtype or NULL; may be x or residual
 *   y            [T, d] dtype or NULL; may be x or residual, not h
 *   y8, y_scale  y in 8 bits (layout above), both or neither NULL
 *   rstd         [T] float or NULL, what the backward takes
 * d <= MOE_NORM_MAX_WIDTH (MOE_ERR_UNSUPPORTED past it).  T == 0: no-op.  A row that holds a value
 * that is not finite gives NaN (or, where h rstd weight is one, zeros) in that row alone. */
moe_status moe_rms_norm(int32_t num_tokens, int32_t d_model, int32_t dtype, const void *x, const void *residual,
                        const void *weight, float eps, void *h, void *y, uint8_t *y8, uint8_t *y_scale, float *rstd,
                        hipStream_t stream);

/* Its gradients, with g = dy weight and xhat = h rstd (rounding to 8 bits passed through):
 *   dx = dh + rstd (g - xhat mean(g xhat)): the gradient of x and of residual
 *   dweight = sum over the tokens of dy xhat
 *   dy, h    [T, d] dtype (the gradient of y; the forward's h, or x without a residual)
 *   rstd     [T] float, the forward's
 *   dh       [T, d] dtype or NULL: the gradient that reaches h on the residual stream
 *   dx       [T, d] dtype, written; may be dy, h or dh
 *   dweight  [d] float, written (zeros when T == 0)
 *   ws       at least moe_rms_norm_backward_workspace_size(T, d) bytes (0: invalid sizes)
 * Float sums in fixed orders (bit-reproducible). */
size_t moe_rms_norm_backward_workspace_size(int32_t num_tokens, int32_t d_model);
moe_status moe_rms_norm_backward(int32_t num_tokens, int32_t d_model, int32_t dtype, const void *dy, const void *h,
                                 const void *weight, const float *rstd, const void *dh, void *dx, float *dweight,
                                 void *ws, size_t ws_bytes, hipStream_t stream);

/* Grouped products of rows and weights in 8 bits, beside moe_grouped_down and
 * moe_grouped_swiglu_gemm.  For every group g and row r in [group_offsets[g], group_offsets[g+1]):
 *   moe_grouped_linear_fp8:       y_rows[r] = W[g] a_r
 *   moe_grouped_swiglu_gemm_fp8:  y_rows[r] = W_d[g] q(silu(W_g[g] a_r) * (W_u[g] a_r))
 * in float sums, y_rows bf16 (rounded once); q is the rounding to 8 bits of
 * moe_quantize_rows_fp8, formed from the float values.  a_r = row r of x8, or, with row_index, its
 * row row_index[r] (an index outside [0, x_row_count): a row of zeros).  One group of all rows is
 * a dense product.
 *   num_groups, rows_max, group_rows_max  as for moe_grouped_swiglu_gemm; rows_max <= INT32_MAX
 *   x8, x_scale     rows in 8 bits: rows_max of them, or x_row_count, which must be below 2 GiB
 *   group_offsets   [G+1] int32 DEVICE array, non-decreasing within [0, rows_max] (entries
 *                   outside count as its ends; where they fall nothing else is touched, but the rows' results
 *                   are not defined)
 *   w8, w_scale     from moe_quantize_weights_fp8
 *   y_rows          [rows_max, n_out] bf16, written for rows inside a group, others left as they are
 *   ws              at least the bytes of the helper beside (0: invalid arguments)
 * Any n_out, d, f, K >= 1.  A NaN in a row makes that row NaN, one in a weight that output column (of the FFN: one in
 * w_down8; one in w_gate_up8 every row of its group, through H).  Calls
 * for groups of at most 16 rows (rows_max or group_rows_max) multiply in bf16, exactly wherever the scales of a row's block
 * and of a weights' block together are from 2^-121 to 2^119 (past that a result may be NaN, below it products under
 * 2^-103 lose bits); others on the 8-bit matrix
 * instruction, which drops, of 16 products at a time, what lies some 2^-14 below the largest: about 1.5e-5 of
 * a product's size.  For moe_grouped_linear_fp8 that is a hundredth of the result's bf16 rounding; in the FFN it moves one code of
 * H in two thousand over a border, by up to an eighth of its value, and the error of y_rows against 64 bits grows from
 * 1.7e-3 of its norm, the bf16 rounding's, to 1.8e-3 .. 2.1e-3 (2.5e-3 the most seen).  A caller who wants more rows
 * exact announces group_rows_max 16: the weights are then read once for each 16 rows.  Calls of few tiles are cut along K, into parts
 * whose sums are kept in ws and added in order.  Only kernel
 * launches on `stream`; every sum in a fixed order (bit-reproducible). */
size_t moe_grouped_linear_fp8_workspace_size(int32_t num_groups, int64_t rows_max, int32_t group_rows_max,
                                             int32_t n_out, int32_t k);
moe_status moe_grouped_linear_fp8(int32_t num_groups, int64_t rows_max, int32_t group_rows_max, int32_t n_out, int32_t k,
                                  const uint8_t *x8, const uint8_t *x_scale, const int32_t *row_index,
                                  int64_t x_row_count, const int32_t *group_offsets, const uint8_t *w8,
                                  const uint8_t *w_scale, void *y_rows, void *ws, size_t ws_bytes, hipStream_t stream);
size_t moe_grouped_swiglu_gemm_fp8_workspace_size(int32_t num_groups, int64_t rows_max, int32_t group_rows_max,
                                                  int32_t d_model, int32_t d_ff);
moe_status moe_grouped_swiglu_gemm_fp8(int32_t num_groups, int64_t rows_max, int32_t group_rows_max, int32_t d_model,
                                       int32_t d_ff, const uint8_t *x8, const uint8_t *x_scale,
                                       const int32_t *row_index, int64_t x_row_count, const int32_t *group_offsets,
                                       const uint8_t *w_gate_up8, const uint8_t *w_gate_up_scale,
                                       const uint8_t *w_down8, const uint8_t *w_down_scale, void *y_rows, void *ws,
                                       size_t ws_bytes, hipStream_t stream);

/* A matrix of moe_quantize_weights_fp8, and a layer's (swiglu 1 for the gate_up ones; the shared
 * expert's are one group of width d_ff_shared, NULL when that is 0). */
typedef struct moe_fp8_matrix {
  const uint8_t *codes, *scale;
} moe_fp8_matrix;
typedef struct moe_weights_fp8 {
  const void *w_router; /* [E, d] bf16 */
  moe_fp8_matrix gate_up, down, shared_gate_up, shared_down;
} moe_weights_fp8;

/* moe_forward with the experts (and the shared expert) in 8 bits: routing, dispatch and combine as
 * there, in bf16 and float, the FFNs as in moe_grouped_swiglu_gemm_fp8, announced with the most rows that an expert can
 * have: min(T, capacity), the shared expert T.  bf16 layers.
 *   x            [T, d] bf16, what the router reads
 *   x8, x_scale  x in 8 bits (moe_rms_norm writes both), or both NULL: quantised here from x
 *   ws           at least moe_forward_fp8_workspace_size(desc) bytes
 * Other arguments, results and errors as for moe_forward. */
size_t moe_forward_fp8_workspace_size(const moe_desc *desc);
moe_status moe_forward_fp8(const moe_desc *desc, const moe_weights_fp8 *weights, const void *x, const uint8_t *x8,
                           const uint8_t *x_scale, const float *logit_offset, void *out, moe_routing *routing, void *ws,
                           size_t ws_bytes, hipStream_t stream);

/* Bytes of the tile-major copy of num_experts experts' gate_up (which = 0) or down
 * (which = 1) weights for desc's shapes: per expert, ceil(f / 128) gate_up tiles (128 gate
 * rows and their 128 up rows each) or ceil(d / 256) down tiles (256 rows each), times K/32
 * steps (K = d for gate_up, f for down), times 16 KB.  0 for an invalid descriptor, a
 * dtype other than bf16, num_experts < 1 or another `which`.  Host only. */
size_t moe_tiled_weights_bytes(const moe_desc *desc, int32_t num_experts, int32_t which);

/* Writes the tile-major copies of num_experts experts' routed weights: a one-time
 * preparation of the runtime layout at weight-loading time ([HF-MoE] "Рефакторинг
 * загрузки весов": checkpoint weights are converted once, on load, into the layout the
 * runtime computes with).  Tile nt, K step kt of expert e is the 16 KB block
 * (e * tiles + nt) * K/32 + kt: the tile's 256 weight rows by 32 values, 64 bytes per row,
 * 16-byte chunk c of row r stored at chunk position c ^ ((r >> 2) & 3), rows past the
 * matrix zero.  gate_up tile nt holds gate rows 128 nt .. 128 nt + 127 followed by the
 * matching up rows (f apart); down tile nt holds rows 256 nt .. 256 nt + 255.  Inputs as in
 * moe_weights ([num_experts, 2f, d] and [num_experts, d, f]); outputs sized by
 * moe_tiled_weights_bytes, 16-byte aligned, not overlapping the inputs.  bf16 only
 * (MOE_ERR_UNSUPPORTED otherwise).  Only kernel launches on `stream`. */
moe_status moe_tile_expert_weights(const moe_desc *desc, int32_t num_experts, const void *w_gate_up,
                                   const void *w_down, void *w_gate_up_tiled, void *w_down_tiled,
                                   hipStream_t stream);

/* One rank's share of expert parallelism ([HF-MoE] "Параллелизм экспертов
 * (Expert Parallelism)": each device holds a contiguous subset of the experts,
 * computes them, and partial outputs are summed across devices with an all-reduce;
 * global expert indices map to local ones and the other experts are masked).
 * Routing, capacity and dispatch run over all E experts, so slots and drops are those
 * of the whole layer; only experts [expert_begin, expert_end) run their FFN, with
 * weights->w_gate_up / w_down holding just those experts ([expert_end - expert_begin,
 * ...], local index 0 = expert_begin); the router weights are the full [E, d].
 *   out_partial[t] = (add_shared ? shared(x_t) : 0)
 *                    + sum over kept j with expert in range of g_tj * FFN_e(x_t)
 * Summing the partials of a partition of [0, E) (shared expert added by exactly one
 * range) gives moe_forward's output up to float summation order.  Other arguments as
 * for moe_forward; 0 <= expert_begin <= expert_end <= E. */
moe_status moe_forward_expert_shard(const moe_desc *desc, const moe_weights *weights, int32_t expert_begin,
                                    int32_t expert_end, int32_t add_shared, const void *x, const float *logit_offset,
                                    void *out_partial, moe_routing *routing, void *ws, size_t ws_bytes,
                                    hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_MI355X_H */
