/*
 * moe.h -- C ABI of one GPU's share of a Mixture-of-Experts layer on MI355X (gfx950).
 *
 * The layer: a router (logits GEMM, softmax top-k, renormalised gates), dispatch into
 * expert-contiguous buffers with capacity truncation, a grouped SwiGLU expert FFN, and a
 * gate-weighted combine back to token order.  Every call below only enqueues HIP kernels on
 * the given stream and returns; none synchronises, allocates or frees.
 *
 * Pages cited:
 *   [EP-serving] aiunderstanding.org, "Expert parallelism for MoE serving" (ru / wo / id).
 *   [EP-checks]  airouter.kz blog, "Expert parallelism in MoE needs measurements before
 *                launch" ("Экспертный параллелизм MoE требует замеров до запуска").
 *
 * Conventions shared by every entry point
 *   - Shapes: T tokens, d model width, E experts, k experts per token, F expert FFN width,
 *     capacity C (see moe_shape.capacity).
 *   - Layouts: row-major.  Weights use the nn.Linear convention [out_features, in_features]
 *     stacked over experts: w_router [E, d], w_gate and w_up [E, F, d], w_down [E, d, F],
 *     so every GEMM operand is contiguous along its reduction axis.
 *   - Types: MOE_BF16 means bf16 activations and weights, fp32 logits, gates and
 *     accumulation, bf16 hidden/expert/layer outputs.  MOE_F32 means fp32 throughout.
 *     Index tables are int32.
 *   - Pointers are device pointers on the current HIP device unless marked "host".  Tensor
 *     pointers (x, weights, x_perm, y_perm, out) must be 16-byte aligned.
 *   - The caller owns every buffer; the library keeps no state between calls (but for the
 *     setting of moe_few_wait_polls), so calls with distinct workspaces and outputs may run
 *     concurrently on different streams.
 *   - Errors: arguments are validated before anything is enqueued and a negative
 *     moe_status is returned on failure (nothing is launched).  A failed launch returns
 *     MOE_ERR_HIP.  T = 0 is valid.
 *   - Limits: 1 <= E <= 1024, 1 <= k <= min(E, 64), d and F multiples of 128 and at most
 *     2^20, T * k < 2^31, and a grouped-GEMM grid (rows and columns of the shape's tiles)
 *     within 2^32 threads; moe_workspace_size() returns 0 for a shape outside them.
 */
#ifndef MOE_H
#define MOE_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = -1, /* null pointer, bad shape value, k > E, ... */
  MOE_ERR_UNSUPPORTED = -2, /* outside the limits above or unknown dtype */
  MOE_ERR_ALIGNMENT = -3,   /* a tensor pointer is not 16-byte aligned */
  MOE_ERR_WORKSPACE = -4,   /* workspace null or smaller than moe_workspace_size() */
  MOE_ERR_HIP = -5,         /* a kernel launch failed */
  MOE_ERR_SCRATCH = -6      /* the shape needs more than the static dispatch scratch */
} moe_status;

typedef enum { MOE_F32 = 0, MOE_BF16 = 1 } moe_dtype;

/* Variants of routing and dispatch, or-ed into moe_shape.flags; 0 selects the defaults
 * described at each entry point.
 *   MOE_FLAG_PAD_TO_CAPACITY  every expert owns C row slots: the kept rows of expert e are
 *       rows e*C + pos of x_perm / y_perm (expert_offsets[e] = e*C) and the slots past its
 *       kept count are zero rows, so the expert GEMMs run on E*C uniform rows.  Pages:
 *       [EP-serving] "Technical details" (fixed expert buffers keep the GEMM shapes
 *       regular) and [EP-checks] "Capacity factor changes quality, memory and tail
 *       latency" (padding spends memory and compute on empty slots).  Needs E*C < 2^31.
 *   MOE_FLAG_SLOT_MAJOR  drop priority visits assignments slot-major, (j, t): every first
 *       choice before any second choice, each slot in token order; kept rows of an expert
 *       are stored in that order.  [EP-checks] "Capacity factor changes quality, memory
 *       and tail latency" (which choices are dropped matters).
 *   MOE_FLAG_BIAS_SELECTION_ONLY  b_router shifts the selection only: logits = x w^T
 *       (no bias), the top-k uses the fp32 sums logits + b_router, and the gates use the
 *       unbiased logits of the selected experts.  [EP-checks] "Routing is a system-level
 *       decision" (balancing the load is part of routing). */
enum {
  MOE_FLAG_PAD_TO_CAPACITY = 1,
  MOE_FLAG_SLOT_MAJOR = 2,
  MOE_FLAG_BIAS_SELECTION_ONLY = 4
};

typedef struct {
  int64_t T;        /* tokens (rows of x) */
  int64_t d;        /* model width */
  int64_t E;        /* experts */
  int64_t k;        /* experts per token */
  int64_t F;        /* expert FFN width */
  int64_t capacity; /* per-expert capacity C; <= 0 means no limit (C = T) */
  int32_t dtype;    /* moe_dtype */
  int32_t flags;    /* MOE_FLAG_* bits; unknown bits are rejected */
  /* Group-limited top-k ([EP-checks] "Routing is a system-level decision": limiting how
   * many nodes a token reaches shapes the exchange).  With n_groups > 1 the experts form
   * n_groups groups of E / n_groups consecutive indices; a group's score is its best
   * selection logit; each token keeps its topk_groups best groups (ties to the lower
   * group) and picks its k experts among theirs.  n_groups 0 or 1: no limit (topk_groups
   * must then be 0).  Limits: n_groups <= 64 and divides E, 1 <= topk_groups <=
   * n_groups, k <= topk_groups * E / n_groups. */
  int32_t n_groups;
  int32_t topk_groups;
} moe_shape;

/* Drop counters written by moe_dispatch / moe_layer: drops[0] = dropped assignments,
 * drops[1 + j] = dropped assignments of slot j (j < k), drops[1 + k] = tokens whose k
 * assignments were all dropped.  Length k + 2. */

/* Regions of the workspace, for callers that want to read intermediate tables of
 * moe_layer (see moe_workspace_layout). */
typedef enum {
  MOE_WS_LOGITS = 0,  /* float [T, E] */
  MOE_WS_TOPK_IDX,    /* int32 [T, k] */
  MOE_WS_TOPK_W,      /* float [T, k] */
  MOE_WS_ROUTED,      /* int32 [E]   routed counts n_e */
  MOE_WS_KEPT,        /* int32 [E]   kept counts c_e */
  MOE_WS_OFFSETS,     /* int32 [E+1] */
  MOE_WS_SRC_TOKEN,   /* int32 [R]   R = moe_max_rows() */
  MOE_WS_DEST_ROW,    /* int32 [T, k] */
  MOE_WS_DROPS,       /* int32 [k+2] */
  MOE_WS_STATUS,      /* int32 [1] */
  MOE_WS_TILE_HIST,   /* internal */
  MOE_WS_TILE_BASE,   /* internal */
  MOE_WS_SCHED,       /* internal */
  MOE_WS_X_PERM,      /* [R, d] */
  MOE_WS_H,           /* [R, F] */
  MOE_WS_Y_PERM,      /* [R, d] */
  MOE_WS_DOWN_ACC,    /* internal: fp32 partial sums of the down GEMM's split tail tiles */
  MOE_WS_COUNT
} moe_ws_region;

/* Per-expert capacity from a capacity factor ([EP-checks], "Capacity factor changes
 * quality, memory and tail latency": mean tokens per expert times the factor; the mean is
 * T*k/E by the section "Mean expert load proves almost nothing").  Returns
 * ceil(((cf * T) * k) / E) evaluated in IEEE double; 0 (no limit) when cf <= 0; -1 when T < 0,
 * k < 1 or E < 1, cf is not finite or the result does not fit int64.  Host function. */
int64_t moe_capacity(int64_t T, int64_t k, int64_t E, double cf);

/* Row slots R of x_perm, y_perm and src_token: min(T*k, E*C) with C = T when unlimited,
 * or E*C with MOE_FLAG_PAD_TO_CAPACITY ([EP-serving] "Technical details": expert buffers
 * sized by the capacity; [EP-checks] "Capacity factor changes quality, memory and tail
 * latency": the capacity bounds what each expert's buffer must hold).  Returns -1 for an
 * invalid shape.  Host function. */
int64_t moe_max_rows(const moe_shape* shape);

/* Bytes of device workspace that any call below needs for this shape (the same size
 * serves all of them); 0 for an invalid shape.  [EP-checks] "Memory must be counted by
 * phase": the dispatch and combine buffers and the MoE temporaries are a line of their own
 * in the memory sheet, sized from the shape and capacity, not from the active parameters.
 * Host function. */
size_t moe_workspace_size(const moe_shape* shape);

/* Byte offsets (host array of MOE_WS_COUNT) of each region in the workspace; a region of
 * size 0 still gets an offset.  Regions are 256-byte aligned and laid out in the order of
 * moe_ws_region, so a region's size is bounded by the next offset (the last one by
 * moe_workspace_size).  [EP-checks] "Memory must be counted by phase" (which buffer each
 * stage holds).  Returns a moe_status.  Host function. */
int moe_workspace_layout(const moe_shape* shape, int64_t* offsets);

/* Human-readable name of a moe_status value (static string).  Host function. */
const char* moe_status_string(int status);

/* Phases of moe_layer at which [EP-checks] "Memory must be counted by phase" asks for the
 * memory held: before the MoE layer, after packing, after dispatch, after the expert
 * compute.  At expert-parallel size 1 the dispatch exchange moves nothing, so the figures
 * after packing and after dispatch are equal (a multi-GPU exchange would add its receive
 * buffers at the second). */
typedef enum {
  MOE_PHASE_BEFORE_LAYER = 0,
  MOE_PHASE_AFTER_PACK,     /* router tables, dispatch tables, x_perm when it is copied */
  MOE_PHASE_AFTER_DISPATCH, /* equal to MOE_PHASE_AFTER_PACK on one GPU */
  MOE_PHASE_AFTER_EXPERTS,  /* + the tile table, h, y_perm and any split-reduction slots */
  MOE_PHASE_COUNT
} moe_phase;

/* Bytes of the workspace that moe_layer has written by the end of each moe_phase
 * ([EP-checks] "Memory must be counted by phase"), as sums of the exact sizes of the
 * regions each stage writes (moe_ws_region; row regions at their bound R = moe_max_rows,
 * so these are upper bounds of what one call touches), assuming the optional outputs of
 * moe_layer (routed_counts, tokens_per_expert, drops, status) are NULL and so kept in the
 * workspace.  A gathered layer (see moe_layer) does not count x_perm.  The workspace itself
 * is allocated once by the caller: these figures say how much of it each phase needs.
 *   bytes  host array of MOE_PHASE_COUNT int64, out.
 * Returns a moe_status.  Host function. */
int moe_workspace_phases(const moe_shape* shape, int64_t* bytes);

/* S9: the per-layer expert statistics record of [EP-checks] "Mean expert load proves
 * almost nothing" (counts per expert after top-k, mean = sum / E, p50, p95, max, max over
 * mean, the share held by the busiest 5 % of the experts, drops).  Readings: the record is
 * over routed counts n_e (before capacity truncation, so a hot expert shows above the
 * capacity); p50 and p95 are nearest ranks, the ceil(q E)-th smallest count with q E
 * evaluated in IEEE double; the busiest 5 % are the ceil(0.05 E) largest counts. */
typedef struct {
  int64_t active_tokens;             /* T */
  int64_t top_k;                     /* k */
  int64_t experts;                   /* E */
  int64_t routed;                    /* sum of n_e */
  int64_t expert_p50;                /* nearest-rank median of n_e */
  int64_t expert_p95;                /* nearest-rank 95th percentile of n_e */
  int64_t expert_max;                /* max n_e */
  double expert_mean;                /* sum n_e / E */
  double expert_max_to_mean;         /* max / mean; NaN when nothing was routed */
  int64_t top_5_percent_experts;     /* ceil(0.05 E) */
  double top_5_percent_expert_share; /* their share of sum n_e; 0 when nothing was routed */
  int64_t kept_rows;                 /* sum c_e (sum n_e without tokens_per_expert) */
  int64_t active_experts;            /* experts with c_e > 0 */
  int64_t dropped_tokens;            /* dropped assignments, sum (n_e - c_e) */
} moe_expert_stats_t;

/* Fill *out from host copies of the counts of one layer.
 *   routed_counts      [E] int32 host, n_e >= 0
 *   tokens_per_expert  [E] int32 host, nullable: c_e with 0 <= c_e <= n_e (NULL: no drops)
 * Returns MOE_ERR_INVALID_ARG for T < 0, k < 1, E < 1, null pointers or counts outside
 * those ranges.  Host function. */
int moe_expert_stats(int64_t T, int64_t k, int64_t E, const int32_t* routed_counts,
                     const int32_t* tokens_per_expert, moe_expert_stats_t* out);

/* Per-slot record ([EP-checks] "Top-2 does not insure against hot experts": the second
 * choice can pile onto the same hot experts, and which choices get dropped matters), from
 * host copies of moe_slot_counts' tables.
 *   routed_by_slot, kept_by_slot  [k, E] int32 host (kept <= routed entry by entry)
 *   slot_max_to_mean    [k] double out: max_e routed_by_slot[j][e] / (T / E), the
 *                       imbalance of the (j+1)-th choice alone (0 when T = 0)
 *   drop_share_per_slot [k] double out: dropped assignments of slot j over all dropped
 *                       ones (0 when nothing was dropped)
 * Returns a moe_status.  Host function. */
int moe_slot_stats(int64_t T, int64_t k, int64_t E, const int32_t* routed_by_slot,
                   const int32_t* kept_by_slot, double* slot_max_to_mean,
                   double* drop_share_per_slot);

/* Load per rank and per node under a placement of the experts ([EP-checks] "Expert and GPU
 * can be balanced differently": balanced experts do not make balanced GPUs).
 *   routed_counts  [E] int32 host
 *   placement      [E] int32 host: rank holding expert e, in [0, n_ranks)
 *   ranks_per_node 0: no node figures; else ranks r * ranks_per_node ... form node r
 *   rank_load      [n_ranks] int64 out: sum of n_e over the rank's experts
 *   node_load      [ceil(n_ranks / ranks_per_node)] int64 out (nullable when
 *                  ranks_per_node is 0)
 *   max_to_mean    [2] double out: max over mean of the rank loads, then of the node loads
 *                  (0 when nothing was routed or without nodes)
 * Returns a moe_status.  Host function. */
int moe_placement_load(int64_t E, const int32_t* routed_counts, const int32_t* placement,
                       int64_t n_ranks, int64_t ranks_per_node, int64_t* rank_load,
                       int64_t* node_load, double* max_to_mean);

/*
 * moe_route -- S1 router logits and S2 top-k gating.
 * [EP-serving] "Deep dive": a router picks the top-k experts (often 1 or 2) of each token.
 * Layer specification: logits L = x w_router^T + b_router (fp32); the k largest logits
 * per token under (value descending, expert index ascending), -0.0 equal to +0.0; gates
 * w_j = exp(L_j - L_max) / sum over the k selected exp(L_i - L_max) (softmax restricted to
 * the selection and renormalised).  With MOE_FLAG_BIAS_SELECTION_ONLY the bias enters the
 * selection only; with n_groups > 1 the selection is group-limited (see moe_shape).
 *   x          [T, d] dtype          (unused when logits_given)
 *   w_router   [E, d] dtype          (unused when logits_given)
 *   b_router   [E] float, nullable
 *   logits     [T, E] float: output, or input when logits_given != 0
 *   topk_idx   [T, k] int32 out, slot 0 = best expert
 *   topk_w     [T, k] float out
 *   status     [1] int32 out, nullable: number of tokens with a non-finite logit (their
 *              selection and gates are then unspecified)
 */
int moe_route(const moe_shape* shape, const void* x, const void* w_router,
              const float* b_router, float* logits, int logits_given, int32_t* topk_idx,
              float* topk_w, int32_t* status, hipStream_t stream);

/*
 * moe_dispatch -- S3-S5: the single-GPU stand-in of the dispatch all-to-all.
 * [EP-serving] "Technical details" (tokens go to the experts they chose; experts have
 * capacity-limited buffers; overflow is dropped) and [EP-checks] "Capacity factor changes
 * quality, memory and tail latency" (overflow is dropped before the exchange).
 * Drop priority: first come, first kept in token order.  The assignment (t, j) -> e is
 * kept iff fewer than C earlier assignments (token-major order, or slot-major with
 * MOE_FLAG_SLOT_MAJOR) went to e.  Kept rows of expert e fill rows [expert_offsets[e],
 * expert_offsets[e] + tokens_per_expert[e]) of x_perm in that order; expert_offsets is
 * the exclusive scan of tokens_per_expert, or e*C with MOE_FLAG_PAD_TO_CAPACITY (then the
 * other slots of x_perm are zero rows).  Entries of topk_idx outside [0, E) are dropped.
 *   topk_idx          [T, k] int32 in
 *   x                 [T, d] dtype in
 *   workspace         moe_workspace_size() bytes; workspace_bytes its size
 *   routed_counts     [E] int32 out: n_e, assignments routed to e
 *   tokens_per_expert [E] int32 out: c_e = min(n_e, C)
 *   expert_offsets    [E+1] int32 out: exclusive scan of c_e
 *   src_token         [R] int32 out: token of each kept row, -1 for every other slot
 *   src_slot          [R] int32 out, nullable: slot j of the assignment (t, j) each kept
 *                     row holds, -1 for every other slot (dest_row inverted:
 *                     dest_row[src_token[r], src_slot[r]] = r)
 *   dest_row          [T, k] int32 out: row of each assignment in x_perm, -1 if dropped
 *   drops             [k+2] int32 out (see above)
 *   x_perm            [R, d] dtype out: x_perm[r] = x[src_token[r]] for kept rows; nullable:
 *                     NULL builds the tables only (no row is copied, x may then be NULL),
 *                     for moe_expert_gate_up_gathered
 */
int moe_dispatch(const moe_shape* shape, const int32_t* topk_idx, const void* x,
                 void* workspace, size_t workspace_bytes, int32_t* routed_counts,
                 int32_t* tokens_per_expert, int32_t* expert_offsets, int32_t* src_token,
                 int32_t* src_slot, int32_t* dest_row, int32_t* drops, void* x_perm,
                 hipStream_t stream);

/*
 * moe_dispatch_no_workspace -- moe_dispatch for callers that cannot allocate device memory
 * (code under HIP graph capture, tight serving loops, harnesses that forbid allocation):
 * the same operation, arguments and results as moe_dispatch, without the workspace.  The
 * dispatch's scratch tables (per-tile expert histogram and its per-expert scan, int32
 * [ntiles, E] each, 256-byte aligned, ntiles = ceil(T*k / (floor(512 / k) * k))) live in a
 * static array of MOE_DISPATCH_SCRATCH_BYTES that the library holds on each GPU it runs on
 * until the process ends.  Calls on one GPU share that array: calls that overlap on one
 * GPU (concurrent streams, or threads) race and must not be made.  Shapes whose two tables
 * need more than the array holds return MOE_ERR_SCRATCH before anything is enqueued.  The
 * first call on a device looks up that device's copy of the array (no allocation); a
 * failed lookup returns MOE_ERR_HIP.  Nothing here allocates or frees memory.
 */
#define MOE_DISPATCH_SCRATCH_BYTES (8u << 20)
int moe_dispatch_no_workspace(const moe_shape* shape, const int32_t* topk_idx, const void* x,
                              int32_t* routed_counts, int32_t* tokens_per_expert,
                              int32_t* expert_offsets, int32_t* src_token, int32_t* src_slot,
                              int32_t* dest_row, int32_t* drops, void* x_perm,
                              hipStream_t stream);

/*
 * moe_expert_ffn -- S6-S7: grouped SwiGLU FFN over the expert-contiguous rows.
 * [EP-serving] "Deep dive" (each expert is a small feed-forward network) and "Technical
 * details" (expert buffers keep the GEMM shapes regular); layer specification: for rows r
 * of expert e, h = silu(x_perm[r] w_gate[e]^T) * (x_perm[r] w_up[e]^T), rounded to dtype,
 * and y_perm[r] = h w_down[e]^T.  Row counts per expert are read on the device from
 * expert_offsets; rows >= expert_offsets[E] are not written.
 *   x_perm          [R, d] dtype in
 *   expert_offsets  [E+1] int32 in (non-decreasing, expert_offsets[E] <= R)
 *   w_gate, w_up    [E, F, d] dtype; w_down [E, d, F] dtype
 *   workspace       holds h [R, F] and the tile schedule
 *   y_perm          [R, d] dtype out
 */
int moe_expert_ffn(const moe_shape* shape, const void* x_perm, const int32_t* expert_offsets,
                   const void* w_gate, const void* w_up, const void* w_down, void* workspace,
                   size_t workspace_bytes, void* y_perm, hipStream_t stream);

/*
 * moe_expert_gate_up -- S6 alone: h = silu(x_perm w_gate[e]^T) * (x_perm w_up[e]^T) for
 * the rows of each expert, rounded to dtype (same sources as moe_expert_ffn).  One grouped
 * GEMM launch after a one-block tile-table launch.
 *   h  [R, F] dtype out (rows >= expert_offsets[E] not written)
 */
int moe_expert_gate_up(const moe_shape* shape, const void* x_perm,
                       const int32_t* expert_offsets, const void* w_gate, const void* w_up,
                       void* workspace, size_t workspace_bytes, void* h, hipStream_t stream);

/*
 * moe_expert_gate_up_gathered -- S6 reading the token rows straight from x: h[r] =
 * silu(x[src_token[r]] w_gate[e]^T) * (x[src_token[r]] w_up[e]^T) for the rows of each
 * expert (the pack step of [EP-checks] "All-to-all must be profiled separately from
 * compute" fused into the GEMM's loads, so x_perm is neither written nor read).
 *   x          [T, d] dtype in; src_token [R] int32 in (from moe_dispatch)
 *   h          [R, F] dtype out (rows >= expert_offsets[E], and empty padded slots, whose
 *              src_token is -1, are unspecified)
 * Needs T * d * sizeof(dtype) < 2^31 (MOE_ERR_UNSUPPORTED otherwise).
 */
int moe_expert_gate_up_gathered(const moe_shape* shape, const void* x,
                                const int32_t* src_token, const int32_t* expert_offsets,
                                const void* w_gate, const void* w_up, void* workspace,
                                size_t workspace_bytes, void* h, hipStream_t stream);

/*
 * moe_expert_down -- S7 alone: y_perm[r] = h[r] w_down[e]^T for the rows of each expert
 * (same sources as moe_expert_ffn).  One grouped GEMM launch after a one-block tile-table
 * launch.  For shapes whose down GEMM has few, long tiles (at most m-tiles x ceil(d / 256)
 * of them, fewer than two rounds of the 256 CUs), the tiles that fall into the last,
 * partial round (counted on the device) split their reduction axis into up to 8 pieces,
 * each storing its tile of fp32 partial sums into a slot of the workspace region
 * MOE_WS_DOWN_ACC; one more launch adds each tile's slots in piece order and converts the
 * sums to y_perm, so the result does not depend on which piece finished first.  Such shapes
 * get a non-empty MOE_WS_DOWN_ACC (at most 256 slots of BM x 256 floats, BM the row-tile
 * height) from moe_workspace_size.
 *   h      [R, F] dtype in
 *   y_perm [R, d] dtype out (rows >= expert_offsets[E] not written)
 */
int moe_expert_down(const moe_shape* shape, const void* h, const int32_t* expert_offsets,
                    const void* w_down, void* workspace, size_t workspace_bytes, void* y_perm,
                    hipStream_t stream);

/*
 * moe_combine -- S8: gate-weighted sum back to token order, without atomics.
 * [EP-serving] "Technical details" (the combine step returns expert outputs to their
 * tokens); layer specification: out[t] = sum over slots j = 0..k-1 in order, skipping
 * dropped ones (dest_row < 0), of topk_w[t, j] * y_perm[dest_row[t, j]], accumulated in
 * fp32.  Gates of dropped assignments are not renormalised; a token with every slot dropped
 * gets a zero row.
 *   y_perm [R, d] dtype in; dest_row [T, k] int32 in; topk_w [T, k] float in
 *   out    [T, d] dtype out
 */
int moe_combine(const moe_shape* shape, const void* y_perm, const int32_t* dest_row,
                const float* topk_w, void* out, hipStream_t stream);

/*
 * moe_slot_counts -- routing observability ([EP-checks] "Mean expert load proves almost
 * nothing": look past the mean, at the second choice and at what gets dropped).
 * routed_by_slot[j * E + e] = tokens whose slot j chose expert e; kept_by_slot likewise
 * for assignments with dest_row >= 0.  Entries of topk_idx outside [0, E) are not
 * counted.
 *   topk_idx [T, k] int32 in; dest_row [T, k] int32 in
 *   routed_by_slot, kept_by_slot [k, E] int32 out
 */
int moe_slot_counts(const moe_shape* shape, const int32_t* topk_idx, const int32_t* dest_row,
                    int32_t* routed_by_slot, int32_t* kept_by_slot, hipStream_t stream);

/*
 * moe_layer -- the whole layer: moe_route, moe_dispatch, the expert GEMMs and moe_combine on
 * one stream, with every intermediate in the workspace (regions in moe_ws_region).  This
 * is the expert-parallel-size-1 configuration of [EP-checks] "All-to-all must be profiled
 * separately from compute": every expert is local and no all-to-all runs.  With packed
 * rows (no MOE_FLAG_PAD_TO_CAPACITY) and T * d * sizeof(dtype) < 2^31 the gate/up GEMM
 * gathers the token rows itself (moe_expert_gate_up_gathered) and the x_perm region is
 * left unwritten.  The dispatch also writes the grouped GEMMs' tile table from the offsets
 * it computes, and both GEMMs read it from the workspace.
 *   out               [T, d] dtype out
 *   routed_counts, tokens_per_expert [E] int32 out, nullable (then kept in the workspace)
 *   drops             [k+2] int32 out, nullable
 *   status            [1] int32 out, nullable (non-finite logit count, as in moe_route)
 */
int moe_layer(const moe_shape* shape, const void* x, const void* w_router,
              const float* b_router, const void* w_gate, const void* w_up, const void* w_down,
              void* workspace, size_t workspace_bytes, void* out, int32_t* routed_counts,
              int32_t* tokens_per_expert, int32_t* drops, int32_t* status,
              hipStream_t stream);

/* ------------------------------------------------------------------------------------------
 * Expert weights in 8-bit floating point, and the gradients of the experts' products.
 *
 * 8-bit values are OCP e4m3 (one byte, largest 448, 0x7f / 0xff NaN, no infinities) with one
 * scale for each block of 128: an activation row [K] has K / 128 scales, a weight matrix
 * [N, K] has [N / 128, K / 128] of them, one for each 128 x 128 block.  A value stands for
 * e4m3 * scale.  Scales are contiguous row-major arrays of one of two types:
 *   MOE_SCALE_F32   float: any finite value (block scales as checkpoints store them).  A
 *                   product of two scales past fp32's largest number is carried all the same
 *                   (such tiles take two to two and a half times as long); one below 2^-126
 *                   may be rounded to a multiple of 2^-149, which changes a block's part of a
 *                   sum by at most 2^-125
 *   MOE_SCALE_E8M0  one byte v, standing for 2^(v - 127); 255 stands for NaN.  The matrix
 *                   instruction multiplies these itself.
 * [EP-checks] "Memory must be counted by phase": expert weights are the largest line of the
 * memory sheet, and a decode step reads all of them.
 *
 * Precision of the 8-bit products: sums are held in fp32, but the 8-bit matrix instruction adds
 * eight neighbouring products at a time and cuts them off 13 bits below the largest (measured
 * on MI355X; 1.3e-5 of the result's norm on normal data).  Outputs are therefore bf16, whose
 * half step is 2^-8 of a value at most, and MOE_F32 is refused.
 * ------------------------------------------------------------------------------------------ */
typedef enum { MOE_SCALE_F32 = 0, MOE_SCALE_E8M0 = 1 } moe_scale_type;

/* A tensor of e4m3 values and its scales (device pointers). */
typedef struct {
  const void* q;
  const void* scale;
} moe_fp8_tensor;

/* A product grouped by expert: rows [expert_offsets[e], expert_offsets[e + 1]) of the row
 * operands belong to expert e, whose weight is matrix e of [E, N, K].  Groups may be empty and
 * of any length.  Limits: 0 <= rows < 2^31, 1 <= E <= 1024, N and K multiples of 128 and at
 * most 2^20, and fewer than 2^23 tiles of work, which the kernels number with 32 bits: with rows
 * divided down and N and K up, (rows + 63 E) / 64 * max(N, K) / 128 + 2312 and E * (N / b) *
 * (K / b) + 8, b = 256 for MOE_BF16 and 128 for MOE_F32, are both below 2^23. */
typedef struct {
  int64_t rows;       /* row slots of the row operands */
  int64_t E;          /* experts */
  int64_t N;          /* output width of the product, x W^T */
  int64_t K;          /* input width */
  int32_t dtype;      /* moe_dtype of the operands (gradients) or of the output (8-bit) */
  int32_t scale_type; /* moe_scale_type of the 8-bit operands; the gradients ignore it */
} moe_group_shape;

/* Bytes of device workspace the three grouped entry points below need (the tile table and, for
 * products with few, long tiles, up to 256 slots of fp32 partial sums, 64 MiB); 0 for an invalid
 * shape.  The same size serves all three.  Host function. */
size_t moe_group_workspace_size(const moe_group_shape* shape);

/*
 * moe_quantize -- a matrix to e4m3 with a power-of-two scale for each block of block_rows x 128
 * values: block_rows 1 for activations, 128 for weights ([E, N, K] as E * N rows).
 * The scale is 2^e with the least e >= -126 for which the block's largest magnitude is at most
 * 448 * 2^e (1 for a block of zeros); q = x / 2^e rounded to nearest even.  The division is
 * exact, so a value is rounded once.  A block that holds an infinity or a NaN becomes all NaN:
 * q 0x7f throughout and a NaN scale (255 for MOE_SCALE_E8M0).
 *   x      [rows, K] dtype in; rows a multiple of block_rows, K of 128
 *   q      [rows, K] e4m3 out
 *   scale  [rows / block_rows, K / 128] scale_type out
 * x and q must be 16-byte aligned; rows * K < 2^37.  rows = 0 is valid.
 */
int moe_quantize(int64_t rows, int64_t K, int64_t block_rows, int dtype, int scale_type,
                 const void* x, void* q, void* scale, hipStream_t stream);

/*
 * moe_grouped_gemm_fp8 -- product of 8-bit operands grouped by expert:
 *   y[r, n] = sum over blocks b of x_scale[r, b] * w_scale[e, n / 128, b] *
 *             (sum over the 128 columns c of b of xq[r, c] * wq[e, n, c])
 * for the rows r of expert e.  Rows >= expert_offsets[E] of y are not written.
 *   xq, x_scale     [rows, K], [rows, K / 128] in
 *   expert_offsets  [E+1] int32 in (non-decreasing, expert_offsets[E] <= rows); NULL with
 *                   E = 1: the dense product, every row belongs to the one matrix
 *   wq, w_scale     [E, N, K], [E, N / 128, K / 128] in
 *   workspace       moe_group_workspace_size() bytes, 256-byte aligned
 *   y               [rows, N] bf16 out
 * shape->dtype must be MOE_BF16.
 */
int moe_grouped_gemm_fp8(const moe_group_shape* shape, const void* xq, const void* x_scale,
                         const int32_t* expert_offsets, const void* wq, const void* w_scale,
                         void* workspace, size_t workspace_bytes, void* y, hipStream_t stream);

/*
 * moe_grouped_dgrad -- gradient of y[r] = x[r] W[e]^T (moe_expert_down, and each product of
 * moe_expert_gate_up) by its input: dx[r, k] = sum over n of dy[r, n] * w[e, n, k].
 * Accumulated in fp32, rounded once to dtype.  Rows >= expert_offsets[E] of dx are not written
 * and those of dy not read.
 *   dy [rows, N] dtype in; w [E, N, K] dtype in; dx [rows, K] dtype out
 *   expert_offsets and workspace as in moe_grouped_gemm_fp8
 */
int moe_grouped_dgrad(const moe_group_shape* shape, const void* dy,
                      const int32_t* expert_offsets, const void* w, void* workspace,
                      size_t workspace_bytes, void* dx, hipStream_t stream);

/*
 * moe_grouped_wgrad -- the same product's gradient by its weight:
 *   dw[e, n, k] = sum over the rows r of expert e of dy[r, n] * x[r, k]
 * accumulated in fp32 in row order, rounded once to dtype.  The matrix of an expert without
 * rows is written as zeros.  Rows >= expert_offsets[E] of dy and x are not read.
 *   dy [rows, N] dtype in; x [rows, K] dtype in; dw [E, N, K] dtype out
 *   expert_offsets and workspace as in moe_grouped_gemm_fp8
 */
int moe_grouped_wgrad(const moe_group_shape* shape, const void* dy, const void* x,
                      const int32_t* expert_offsets, void* workspace, size_t workspace_bytes,
                      void* dw, hipStream_t stream);

/* ------------------------------------------------------------------------------------------
 * Linear layers with a bias, an activation and a residual, their backward pass up to the
 * products, and the clipping of gradients.
 * ------------------------------------------------------------------------------------------ */

/* Activations.  gelu is z P(z), P the normal distribution; gelu_tanh its form with a tanh,
 * z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2.  relu(0) and its slope there are 0. */
typedef enum {
  MOE_ACT_NONE = 0,
  MOE_ACT_RELU = 1,
  MOE_ACT_SILU = 2,
  MOE_ACT_GELU = 3,
  MOE_ACT_GELU_TANH = 4
} moe_activation;

/* Bytes of device workspace of moe_grouped_linear and moe_grouped_linear_grad (the same size
 * serves both); 0 for an invalid shape.  Host function. */
size_t moe_linear_workspace_size(const moe_group_shape* shape);

/* How moe_grouped_linear cuts a shape, for profiles and tests: tiles[0] rows by tiles[1] columns of
 * a tile, and tiles[2], the most pieces along the reduction that a tile of the last partial round
 * is cut into (1: none is cut).  A tile holds rows of one expert.  Host function. */
int moe_linear_tiles(const moe_group_shape* shape, int64_t tiles[3]);

/*
 * moe_grouped_linear -- linear layer grouped by expert, for the rows r of expert e:
 *   z[r, n] = (sum over k of x[r, k] * w[e, n, k]) + bias[e, n],   y[r, n] = act(z[r, n]) + residual[r, n]
 * summed and evaluated in fp32, y rounded once to dtype (act is applied to the unrounded z), and z,
 * where the caller keeps it for the backward pass, rounded once.  Rows outside [expert_offsets[0],
 * expert_offsets[E]) of x and residual are not used, and those of y and z not written.
 *   x         [rows, K] dtype in; w [E, N, K] dtype in
 *   bias      [E, N] float in, nullable
 *   residual  [rows, N] dtype in, nullable; may be y itself
 *   z         [rows, N] dtype out, nullable
 *   y         [rows, N] dtype out
 *   expert_offsets as in moe_grouped_gemm_fp8; workspace moe_linear_workspace_size() bytes,
 *   256-byte aligned
 */
int moe_grouped_linear(const moe_group_shape* shape, int activation, const void* x,
                       const int32_t* expert_offsets, const void* w, const float* bias,
                       const void* residual, void* workspace, size_t workspace_bytes, void* z,
                       void* y, hipStream_t stream);

/*
 * moe_grouped_linear_grad -- backward pass of moe_grouped_linear up to its product, from the
 * gradient dy of y and the z that the forward pass kept:
 *   dz[r, n] = dy[r, n] * act'(z[r, n]),   dbias[e, n] = sum of dz[r, n] over the rows r of expert e
 * in fp32, dz rounded once to dtype, dbias the sum of the unrounded values (0 for an expert without
 * rows).  moe_grouped_dgrad and moe_grouped_wgrad go on from dz; the residual's gradient is dy.
 * K of the shape is not used.  Rows outside [expert_offsets[0], expert_offsets[E]) of dy and z are
 * not read, and those of dz not written.
 *   dy     [rows, N] dtype in
 *   z      [rows, N] dtype in; may be NULL with MOE_ACT_NONE
 *   dz     [rows, N] dtype out, nullable; may be dy itself
 *   dbias  [E, N] float out, nullable
 *   expert_offsets as in moe_grouped_gemm_fp8; workspace moe_linear_workspace_size() bytes,
 *   256-byte aligned
 */
int moe_grouped_linear_grad(const moe_group_shape* shape, int activation, const void* dy,
                            const void* z, const int32_t* expert_offsets, void* workspace,
                            size_t workspace_bytes, void* dz, float* dbias, hipStream_t stream);

/* A gradient: n values of a dtype, contiguous, aligned to their type.  out is where moe_grad_clip
 * puts them, grad itself for clipping in place (moe_grad_norm ignores it). */
typedef struct {
  const void* grad;
  void* out;
  int64_t n;     /* 0 <= n < 2^36; pointers may be NULL when 0 */
  int64_t dtype; /* moe_dtype */
} moe_grad;

/* Bytes of device workspace of moe_grad_norm over `count` gradients; 0 for a count outside
 * [0, 2^20].  Host function. */
size_t moe_grad_workspace_size(int64_t count);

/*
 * moe_grad_norm -- the 2-norm over all values of all gradients, sqrt(sum of squares): squares and
 * sums in 64 bits, added in an order that depends on the lengths and types alone.  A NaN or an infinity among
 * the values makes the norm NaN or infinite.
 *   grads      host array [count], read before the call returns
 *   workspace  moe_grad_workspace_size() bytes, 256-byte aligned
 *   norm       [1] float out (0 without gradients)
 */
int moe_grad_norm(int64_t count, const moe_grad* grads, void* workspace, size_t workspace_bytes,
                  float* norm, hipStream_t stream);

/*
 * moe_grad_clip -- out = grad * (max_norm / norm) where norm > max_norm, and out = grad otherwise,
 * also where the norm is infinite or NaN.  The factor is an fp32 number, the product rounded to fp32
 * and then to the gradient's type.  The norm is read on the device: moe_grad_norm's, or one that the
 * caller made of several.
 * No out may overlap another gradient's memory, or its own grad unless it is the same.
 *   grads  host array [count], read before the call returns
 *   norm   [1] float in
 * max_norm is finite and at least 0.
 */
int moe_grad_clip(int64_t count, const moe_grad* grads, float max_norm, const float* norm,
                  hipStream_t stream);

/* Bytes of device workspace for moe_expert_ffn_fp8 and moe_layer_fp8 (the same size serves
 * both); 0 for an invalid shape or scale type, or a dtype other than MOE_BF16.  Host function. */
size_t moe_fp8_workspace_size(const moe_shape* shape, int scale_type);

/* Byte offsets of the regions in that workspace, as moe_workspace_layout; MOE_WS_X_PERM holds
 * the quantized rows of x and, 256-byte aligned behind them, their scales; MOE_WS_H likewise
 * the quantized hidden rows.  Returns a moe_status.  Host function. */
int moe_fp8_workspace_layout(const moe_shape* shape, int scale_type, int64_t* offsets);

/*
 * moe_expert_ffn_fp8 -- moe_expert_ffn with 8-bit weights.  Each row of x is quantized as by
 * moe_quantize (block_rows 1); gate and up are 8-bit products (moe_grouped_gemm_fp8, held in
 * fp32); h = silu(gate) * up is quantized by rows in the product's epilogue, without a
 * rounding before it; y_perm is the 8-bit product of h with w_down, rounded to bf16.
 * What the instruction cuts off gate and up (above) moves an h near the middle of two e4m3
 * values to the other one now and then: on normal data y_perm is 2.0e-3 of its norm away from
 * the exact network over the same quantized rows, against 1.7e-3 for one whose gate and up are
 * held in fp32 (its rounding to bf16 alone).
 * Same sources as moe_expert_ffn.
 *   x               with src_token: [T, d] bf16, row r of expert e reads x[src_token[r]] (an
 *                   entry outside [0, T), such as an empty padded slot's -1, reads a row of x
 *                   all the same: its row of y_perm is unspecified); without (NULL): x_perm
 *                   [R, d] bf16, R = moe_max_rows
 *   expert_offsets  [E+1] int32 in (non-decreasing, expert_offsets[E] <= R)
 *   w_gate, w_up    [E, F, d] with scales [E, F / 128, d / 128]; w_down [E, d, F] with scales
 *                   [E, d / 128, F / 128], all of scale_type
 *   workspace       moe_fp8_workspace_size() bytes, 256-byte aligned
 *   y_perm          [R, d] bf16 out; rows >= expert_offsets[E] are not written
 * shape->dtype must be MOE_BF16; max(T, R) * d and max(T, R) * F at most 2^37, and with
 * src_token T * d < 2^31 (MOE_ERR_UNSUPPORTED otherwise).
 */
int moe_expert_ffn_fp8(const moe_shape* shape, int scale_type, const void* x,
                       const int32_t* src_token, const int32_t* expert_offsets,
                       const moe_fp8_tensor* w_gate, const moe_fp8_tensor* w_up,
                       const moe_fp8_tensor* w_down, void* workspace, size_t workspace_bytes,
                       void* y_perm, hipStream_t stream);

/*
 * moe_layer_fp8 -- moe_layer with 8-bit expert weights: the router reads bf16 x and w_router as
 * there, the dispatch builds its tables only, and the experts run as moe_expert_ffn_fp8 over the
 * gathered rows.  Needs T * d < 2^31 (MOE_ERR_UNSUPPORTED otherwise).
 * Arguments as in moe_layer and moe_expert_ffn_fp8.
 */
int moe_layer_fp8(const moe_shape* shape, int scale_type, const void* x, const void* w_router,
                  const float* b_router, const moe_fp8_tensor* w_gate,
                  const moe_fp8_tensor* w_up, const moe_fp8_tensor* w_down, void* workspace,
                  size_t workspace_bytes, void* out, int32_t* routed_counts,
                  int32_t* tokens_per_expert, int32_t* drops, int32_t* status,
                  hipStream_t stream);

/* ------------------------------------------------------------------------------------------
 * The whole layer for a few tokens: a step of one chat, of some drafted tokens, of a small batch.
 * ------------------------------------------------------------------------------------------ */
#define MOE_FEW_MAX_TOKENS 16

/* Bytes of device workspace of moe_layer_few and moe_layer_few_fp8 (the same size serves both);
 * 0 for an invalid shape, T > MOE_FEW_MAX_TOKENS, T * k > 512 or T * k * F values of h past 2^31
 * bytes.  Host function. */
size_t moe_few_workspace_size(const moe_shape* shape);

/* The number of looks, of about a microsecond each, after which a block of moe_layer_few gives up
 * waiting for the others; 2^20 at first.  Sets it for the calls that the process makes from now on
 * (0: every wait is given up at once) and returns the number before; a negative one only returns it.
 * The one setting that the library keeps.  Host function. */
int32_t moe_few_wait_polls(int32_t polls);

/*
 * moe_layer_few -- moe_layer for at most MOE_FEW_MAX_TOKENS tokens, which is bound by reading the
 * chosen experts' weights once: no rows are packed and no row tiles filled.  The same layer as
 * moe_layer's, with these differences in its roundings: router logits are summed in 64 bits and
 * rounded once to fp32, so that the selection is the exact logits'; an expert's outputs are not
 * rounded before they are weighted and added (in fp32, by expert).  h is rounded to dtype.
 * MOE_FLAG_PAD_TO_CAPACITY changes nothing: there are no row slots.
 * The faster layer up to eight tokens, and up to sixteen but over few, large experts of which nearly
 * all are chosen (eight of 4096 / 14336, nine tokens 416 us and moe_layer 399).
 * Blocks wait for each other's part of h by counters in the workspace.  A wait that lasts longer than
 * any call does (moe_few_wait_polls) is given up: that takes calls that use one workspace at once,
 * against the rules.  What depends on it in out is then NaN, and status is negative.
 *   workspace  moe_few_workspace_size() bytes, 256-byte aligned
 *   routed_counts, tokens_per_expert [E], drops [k+2] int32 out, all nullable, as in moe_layer
 *   status     [1] int32 out, nullable, as in moe_layer; where a wait was given up its sign bit is
 *              set beside that count
 * Other arguments as in moe_layer.  MOE_ERR_UNSUPPORTED outside moe_few_workspace_size's limits.
 */
int moe_layer_few(const moe_shape* shape, const void* x, const void* w_router,
                  const float* b_router, const void* w_gate, const void* w_up,
                  const void* w_down, void* workspace, size_t workspace_bytes, void* out,
                  int32_t* routed_counts, int32_t* tokens_per_expert, int32_t* drops,
                  int32_t* status, hipStream_t stream);

/*
 * moe_layer_few_fp8 -- moe_layer_few with 8-bit expert weights.  x and h stay in bf16: a weight's
 * value e4m3 * scale is exact, its products with bf16 are summed in fp32 over each block of 128 and
 * then scaled, so the result is that of the weights as they are, without the quantization of x and h
 * that moe_layer_fp8 has.  (Those sums stay in fp32's range for values of x and h below 2^112.)
 * The faster layer up to three tokens; up to eight within a few percent of moe_layer_fp8 either way
 * (over 256 experts of 7168 / 2048 up to a quarter slower), and the slower one with more (there,
 * E8M0 scales, sixteen tokens 842 us and 739).
 * Arguments as in moe_layer_few and moe_expert_ffn_fp8; shape->dtype must be MOE_BF16.
 */
int moe_layer_few_fp8(const moe_shape* shape, int scale_type, const void* x,
                      const void* w_router, const float* b_router,
                      const moe_fp8_tensor* w_gate, const moe_fp8_tensor* w_up,
                      const moe_fp8_tensor* w_down, void* workspace, size_t workspace_bytes,
                      void* out, int32_t* routed_counts, int32_t* tokens_per_expert,
                      int32_t* drops, int32_t* status, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H */
