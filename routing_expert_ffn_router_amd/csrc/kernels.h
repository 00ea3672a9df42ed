// Internal launchers of the MoE kernels.  Each enqueues on stream `s` and returns the
// launch status; argument checking happens in the C ABI layer (moe_abi.cpp) before these
// are called.  dtype: 0 = fp32, 1 = bf16.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// Flat assignments handled by one dispatch tile: a multiple of k, at most kTileMax, so the
// k slots of a token never straddle two tiles.
constexpr int kTileMax = 512;
inline int64_t dispatch_tile_entries(int64_t k) { return (kTileMax / k) * k; }
inline int64_t dispatch_ntiles(int64_t T, int64_t k) {
  const int64_t te = dispatch_tile_entries(k);
  return (T * k + te - 1) / te;
}

hipError_t launch_zero_i32(int32_t* p, int64_t n, hipStream_t s);

// S1.  status_zero (nullable): an int32 the launch also sets to 0 before the logits are
// complete (the top-k status counter), without a launch of its own where it can.
hipError_t launch_router_logits(int dtype, const void* x, const void* w, const float* b,
                                float* logits, int64_t T, int64_t d, int64_t E,
                                int32_t* status_zero, hipStream_t s);
// S2
// sel_bias (nullable): selection-only bias.  n_groups > 1: group-limited selection keeping
// topk_groups groups (n_groups <= min(E, 64), dividing E).
hipError_t launch_topk(const float* logits, const float* sel_bias, int64_t T, int64_t E,
                       int64_t k, int n_groups, int topk_groups, int32_t* idx, float* w,
                       int32_t* status, hipStream_t s);

// S3-S5.  C is the effective capacity (1 <= C <= T when T > 0); R the row bound.
struct DispatchArgs {
  const int32_t* topk_idx;
  const void* x;
  int64_t T, d, E, k, C, R;
  int elt_bytes;
  bool slot_major;     // visit assignments slot-major instead of token-major
  bool pad;            // C slots per expert (offsets e * C, empty slots zero rows)
  int32_t* tile_hist;  // [ntiles, E]
  int32_t* tile_base;  // [ntiles, E]
  int32_t* routed;     // [E]
  int32_t* kept;       // [E]
  int32_t* offsets;    // [E+1]
  int32_t* src_token;  // [R]
  int32_t* src_slot;   // [R], nullable: slot of the assignment each kept row holds
  int32_t* dest_row;   // [T*k]
  int32_t* drops;      // [k+2]
  void* x_perm;        // [R, d]; null: tables only, no row copies
  // nullable: also write the grouped GEMMs' tile table of row height table_bm (at most
  // table_m_max entries, launch_expert_ffn's layout) from the offsets
  int32_t* table = nullptr;
  int table_bm = 0;
  int64_t table_m_max = 0;
};
hipError_t launch_dispatch(const DispatchArgs& a, hipStream_t s);
// The dispatch of T * k assignments over E experts runs in one block (no per-tile scratch
// tables) when it holds at most 2048 assignments over at most 256 experts.  (Measured per
// call: 5 us for 128 assignments, 9 us for 2048, against about 14 us for the three tiled
// kernels; 17 and 21 us for 4096 and 8192, where the tiled kernels are faster.)
constexpr int64_t kFusedDispatchEntries = 2048;
constexpr int64_t kFusedDispatchMaxE = 256;
inline bool dispatch_fused(int64_t T, int64_t k, int64_t E) {
  return T * k > 0 && T * k <= kFusedDispatchEntries && E <= kFusedDispatchMaxE;
}
// The static scratch of moe_dispatch_no_workspace on the current device: its address
// (looked up once per device) and size in bytes.
hipError_t dispatch_scratch(void** ptr, size_t* bytes);

// S6-S7.  The grouped GEMMs run over a device-side tile table (expert, first row) of
// row-tile height bm with at most m_max entries.
struct FfnPlan {
  bool small;      // decode-sized experts (weight streaming)
  int tile;        // 0 decode, 1 prefill 256 rows, 2 prefill 320 rows
  int bm;
  int64_t m_max;   // upper bound on m-tiles over all experts
  int down_split;  // 1, or the most pieces a tail tile of the down GEMM splits into
  int64_t down_pieces_max;  // bound on those pieces (slots of partial sums)
  bool stream_b;   // weight loads carry the non-temporal hint (each line read by ~1 tile)
  int group_cap;   // n-tiles per launch-order group (each XCD walks groups of m x group)
};
// pad: every expert holds exactly C rows (offsets e * C).  d, F and the element size
// decide whether the down GEMM splits its reduction.
FfnPlan ffn_plan(int64_t T, int64_t E, int64_t k, int64_t C, int64_t R, bool pad, int64_t d,
                 int64_t F, int64_t elt);
inline int64_t ffn_table_ints(const FfnPlan& p) { return 1 + 2 * p.m_max; }
// Upper bound on the blocks of one grouped-GEMM launch of plan p (512 threads each).
int64_t ffn_max_blocks(const FfnPlan& p, int64_t d, int64_t F);
// CUs the tail split of the down GEMM fills (MI355X: 256).
constexpr int kSplitCUs = 256;
// fp32 partial sums of the down GEMM's split tail tiles: down_pieces_max slots of
// bm x 256 floats (0 bytes when it does not split)
inline int64_t ffn_down_acc_bytes(const FfnPlan& p) {
  return p.down_split > 1 ? p.down_pieces_max * p.bm * 256 * 4 : 0;
}

struct FfnArgs {
  int dtype;
  const void* x_perm;
  const void* x;            // with src_rows: the gate/up GEMM reads x[src_rows[r]] for row r
  const int32_t* src_rows;  // nullable; [R] token of each row (-1: empty padded slot)
  const int32_t* offsets;  // [E+1]
  const void* w_gate;
  const void* w_up;
  const void* w_down;
  int64_t T, d, E, k, F, C, R;
  bool pad;
  void* h;               // [R, F]
  int32_t* sched;        // ffn_table_ints() ints
  void* y_perm;          // [R, d]
  float* down_acc;       // ffn_down_acc_bytes() of fp32 partial sums (tail split)
  bool table_ready;      // sched already holds this call's tile table (skip rebuilding it)
};
// S1 through the grouped-GEMM pipeline in dense mode (64 x 128 tiles, fp32 out + bias),
// for shapes with enough tiles (router_gemm_suits).
bool router_gemm_suits(int64_t T, int64_t E);
hipError_t launch_router_gemm(int dtype, const void* x, const void* w, const float* b,
                              float* logits, int64_t T, int64_t d, int64_t E, hipStream_t s);

// which: 1 = gate/up GEMM (x_perm -> h), 2 = down GEMM (h -> y_perm), 3 = both.  Each
// call first rebuilds the tile table from `offsets`, unless a.table_ready says an earlier
// call on the same stream built it from the same offsets.
hipError_t launch_expert_ffn(const FfnArgs& a, int which, hipStream_t s);

// ---------------------------------------------------------------------------------------
// 8-bit products and gradients
// ---------------------------------------------------------------------------------------
hipError_t launch_quantize(int64_t rows, int64_t K, int64_t block_rows, int dtype,
                           int scale_type, const void* x, void* q, void* scale, hipStream_t s);

// Tile table of row height bm over the experts' rows: table[0] = tiles, then (expert, first
// row) pairs, at most m_max of them.  Offsets are clamped to [0, rows].
hipError_t launch_tile_table(const int32_t* offsets, int64_t E, int64_t rows, int bm,
                             int64_t m_max, int32_t* table, hipStream_t s);

// Row tiling of a grouped product over R row slots of E experts.
struct GroupPlan {
  int bm;         // row-tile height
  int64_t m_max;  // bound on the row tiles over all experts
};
GroupPlan fp8_plan(int64_t R, int64_t E);
GroupPlan dgrad_plan(int64_t R, int64_t E, int elt);  // elt: bytes of a value
// The tail split of a product in 256-column tiles whose reduction takes `steps` steps, where those
// are at least `least` (fewer where the tail leaves most CUs idle): the most pieces a tail tile
// is cut into (1: no split), and the bytes of their partial sums.
struct GroupSplit {
  int s_max;
  int64_t bytes;
};
GroupSplit group_split(const GroupPlan& p, int64_t E, int64_t columns, int64_t steps,
                       int64_t least);
GroupSplit fp8_split(int64_t R, int64_t E, int64_t N, int64_t K);
GroupSplit dgrad_split(int64_t R, int64_t E, int64_t N, int64_t K, int elt);
inline int64_t group_table_ints(const GroupPlan& p) { return 1 + 2 * p.m_max; }
// Whether the grouped launches read a tile table: with few experts the blocks find their tiles
// from the offsets (RowTiles) and any table is passed over.  Every caller goes by this, so that
// one shape runs the same kernels and adds in the same order from all of them.
constexpr int kScanExperts = 64;
inline bool group_needs_table(int64_t E) { return E > kScanExperts; }

// One 8-bit grouped product.  With b1 (the up weights; b0 then the gate weights): the output is
// silu(gate) * up, quantized by rows into hq [R, N] and h_scale; else y [R, N] bf16.
struct Fp8Args {
  const void* xq;           // [x_rows, K]
  const void* x_scale;      // [x_rows, K / 128]
  const int32_t* src_rows;  // nullable: row r reads xq row src_rows[r], clamped to x_rows
  int64_t x_rows;
  const void* b0;
  const void* b0_scale;
  const void* b1;
  const void* b1_scale;
  int64_t R, E, N, K;
  int scale_type;
  const int32_t* offsets;  // [E+1]
  const int32_t* table;    // launch_tile_table of fp8_plan(R, E), or null (group_needs_table)
  void* y;
  void* hq;
  void* h_scale;
  void* partial;  // fp8_split().bytes of partial sums (not with b1)
};
hipError_t launch_fp8_gemm(const Fp8Args& a, hipStream_t s);

// dtype 0 fp32, 1 bf16.  partial: dgrad_split().bytes.  dgrad reads the table of dgrad_plan (or
// null: group_needs_table); wgrad needs only the offsets.
hipError_t launch_dgrad(int dtype, const void* dy, const int32_t* offsets,
                        const int32_t* table, const void* w, void* dx, void* partial, int64_t R,
                        int64_t E, int64_t N, int64_t K, hipStream_t s);
hipError_t launch_wgrad(int dtype, const void* dy, const void* x, const int32_t* offsets,
                        void* dw, int64_t R, int64_t E, int64_t N, int64_t K, hipStream_t s);
// Upper bound on the tiles and pieces that the grouped launches above number.
int64_t group_max_tiles(int64_t R, int64_t E, int64_t N, int64_t K, int elt);

// ---------------------------------------------------------------------------------------
// linear layers of the experts and clipping of gradients
// ---------------------------------------------------------------------------------------
// y = act(x W[e]^T + bias[e]) + residual, z what act takes.
struct LinearArgs {
  int dtype, act;
  const void* x;           // [R, K]
  const void* w;           // [E, N, K]
  const int32_t* offsets;  // [E+1], nullable: one expert holds all rows
  const int32_t* table;    // launch_tile_table of linear_plan, or null (group_needs_table)
  const float* bias;       // [E, N], nullable
  const void* residual;    // [R, N], nullable
  void* z;                 // [R, N], nullable
  void* y;                 // [R, N]
  void* partial;           // linear_split().bytes
  int64_t R, E, N, K;
};
GroupPlan linear_plan(int64_t R, int64_t E, int64_t N, int elt);
int64_t linear_columns(int64_t R, int64_t E, int64_t N, int elt);  // of a tile
GroupSplit linear_split(int64_t R, int64_t E, int64_t N, int64_t K, int elt);
hipError_t launch_linear(const LinearArgs& a, hipStream_t s);

// dz = dy * act'(z) and db[e] = sum of dz over the rows of expert e.  partial: rows of N sums, one
// for each of linear_grad_slots() row tiles (with db only).  dz and z may be null without an
// activation.
constexpr int kGradRows = 64;
inline int64_t linear_grad_slots(int64_t R, int64_t E) { return R / kGradRows + E; }
hipError_t launch_linear_grad(int dtype, int act, const void* dy, const void* z,
                              const int32_t* offsets, void* dz, float* db, float* partial,
                              int64_t R, int64_t E, int64_t N, hipStream_t s);

// ---------------------------------------------------------------------------------------
// the whole layer for a few tokens
// ---------------------------------------------------------------------------------------
constexpr int64_t kFewTokens = 16, kFewPairs = 512;
// counters of tickets, each in a line of its own, before those of the column tiles; the most
// chunks of the down product's reduction
constexpr int kFewCounters = 96, kFewChunks = 32;
struct FewArgs {
  int dtype, scale_type;  // scale_type < 0: weights of dtype
  const void* x;          // [T, d]
  const void* w_router;   // [E, d]
  const float* bias;      // [E], nullable: of the logits
  const float* sel_bias;  // [E], nullable: of the selection alone
  const void* w[3];       // gate, up [E, F, d], down [E, d, F]
  const void* w_scale[3];
  float* logits;          // [T, E]
  void* h;                // [T k, F]
  float* partial;         // [kFewChunks][T, d]
  int32_t* counters;      // kFewCounters + d / 16
  void* out;              // [T, d]
  int32_t* routed;        // nullable, as the three below
  int32_t* kept;
  int32_t* drops;
  int32_t* status;
  int64_t T, d, E, k, F, C;
  int n_groups, topk_groups;  // 1, 1: no limit
  bool slot_major;
};
hipError_t launch_few(const FewArgs& a, hipStream_t s);
int32_t few_wait_polls(int32_t polls);  // moe_few_wait_polls

struct GradTensor {  // moe_grad
  const void* grad;
  void* out;
  int64_t n;
  int64_t dtype;
};
// Tensors of one launch: what 4 KB of kernel arguments hold.
constexpr int kNormTensors = 192, kClipTensors = 136;
// Blocks of a launch: eight of 256 threads for each of the 256 CUs.
constexpr int kNormBlocks = 2048, kClipBlocks = 2048;
// Sums that launch_grad_norm may leave in partial: those of each launch's blocks.
inline int64_t grad_norm_sums(int64_t count) {
  return (count + kNormTensors - 1) / kNormTensors * kNormBlocks;
}
hipError_t launch_grad_norm(int64_t count, const GradTensor* g, double* partial, float* norm,
                            hipStream_t s);
hipError_t launch_grad_clip(int64_t count, const GradTensor* g, float max_norm,
                            const float* norm, hipStream_t s);

// S8
hipError_t launch_combine(int dtype, const void* y_perm, const int32_t* dest_row,
                          const float* topk_w, void* out, int64_t T, int64_t d, int64_t k,
                          hipStream_t s);

// Observability: routed_by_slot / kept_by_slot [k, E] (zeroed here first).
hipError_t launch_slot_counts(const int32_t* idx, const int32_t* dest_row, int64_t T,
                              int64_t k, int64_t E, int32_t* routed_by_slot,
                              int32_t* kept_by_slot, hipStream_t s);

}  // namespace moe
