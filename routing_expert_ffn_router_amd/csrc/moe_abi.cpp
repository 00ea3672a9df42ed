// C ABI of the MoE layer: argument validation, workspace layout and the call sequence of
// each entry point.  Every check happens before anything is enqueued; kernels only see
// arguments that passed them.  See include/moe.h for the contract of each function.
#include <math.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "../../include/moe.h"
#include "kernels.h"

namespace {

constexpr int64_t kAlign = 256;
constexpr int64_t kMaxE = 1024;
constexpr int64_t kMaxK = 64;

int64_t align_up(int64_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

int elt_bytes(int32_t dtype) { return dtype == MOE_BF16 ? 2 : 4; }

int64_t eff_capacity(const moe_shape* s) {
  return (s->capacity <= 0 || s->capacity > s->T) ? s->T : s->capacity;
}

constexpr int32_t kKnownFlags =
    MOE_FLAG_PAD_TO_CAPACITY | MOE_FLAG_SLOT_MAJOR | MOE_FLAG_BIAS_SELECTION_ONLY;
constexpr int64_t kMaxGroups = 64;

bool padded(const moe_shape* s) { return (s->flags & MOE_FLAG_PAD_TO_CAPACITY) != 0; }
bool grouped(const moe_shape* s) { return s->n_groups > 1 && s->topk_groups < s->n_groups; }

int64_t max_rows(const moe_shape* s) {
  const int64_t a = s->T * s->k, b = s->E * eff_capacity(s);
  if (padded(s)) return b;
  return a < b ? a : b;
}

int check_shape(const moe_shape* s) {
  if (!s) return MOE_ERR_INVALID_ARG;
  if (s->T < 0 || s->d <= 0 || s->E <= 0 || s->k <= 0 || s->F <= 0) return MOE_ERR_INVALID_ARG;
  if (s->flags & ~kKnownFlags) return MOE_ERR_INVALID_ARG;
  if (s->k > s->E) return MOE_ERR_INVALID_ARG;
  if (s->dtype != MOE_F32 && s->dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  if (s->E > kMaxE || s->k > kMaxK) return MOE_ERR_UNSUPPORTED;
  if (s->d % 128 != 0 || s->F % 128 != 0) return MOE_ERR_UNSUPPORTED;
  if (s->T > ((((int64_t)1 << 31) - 1) / s->k)) return MOE_ERR_UNSUPPORTED;  // T * k < 2^31
  if (s->d > ((int64_t)1 << 20) || s->F > ((int64_t)1 << 20)) return MOE_ERR_UNSUPPORTED;
  if (padded(s) && s->E * eff_capacity(s) >= ((int64_t)1 << 31)) return MOE_ERR_UNSUPPORTED;
  // group-limited selection
  if (s->n_groups < 0 || s->topk_groups < 0) return MOE_ERR_INVALID_ARG;
  if (s->n_groups <= 1) {
    if (s->topk_groups != 0) return MOE_ERR_INVALID_ARG;
  } else {
    if (s->n_groups > kMaxGroups || s->n_groups > s->E) return MOE_ERR_UNSUPPORTED;
    if (s->E % s->n_groups != 0) return MOE_ERR_INVALID_ARG;
    if (s->topk_groups < 1 || s->topk_groups > s->n_groups) return MOE_ERR_INVALID_ARG;
    if (s->k > (int64_t)s->topk_groups * (s->E / s->n_groups)) return MOE_ERR_INVALID_ARG;
  }
  // every grouped-GEMM launch within 2^32 threads (512 per block)
  const int64_t R = max_rows(s);
  const moe::FfnPlan plan = moe::ffn_plan(s->T, s->E, s->k, eff_capacity(s), R, padded(s),
                                          s->d, s->F, elt_bytes(s->dtype));
  if (moe::ffn_max_blocks(plan, s->d, s->F) >= ((int64_t)1 << 23)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

struct Layout {
  int64_t off[MOE_WS_COUNT];
  int64_t size[MOE_WS_COUNT];
  int64_t total;
};

Layout make_layout(const moe_shape* s) {
  Layout L;
  const int64_t T = s->T, E = s->E, k = s->k, R = max_rows(s), b = elt_bytes(s->dtype);
  const int64_t ntiles = moe::dispatch_ntiles(T, k);
  L.size[MOE_WS_LOGITS] = T * E * 4;
  L.size[MOE_WS_TOPK_IDX] = T * k * 4;
  L.size[MOE_WS_TOPK_W] = T * k * 4;
  L.size[MOE_WS_ROUTED] = E * 4;
  L.size[MOE_WS_KEPT] = E * 4;
  L.size[MOE_WS_OFFSETS] = (E + 1) * 4;
  L.size[MOE_WS_SRC_TOKEN] = R * 4;
  L.size[MOE_WS_DEST_ROW] = T * k * 4;
  L.size[MOE_WS_DROPS] = (k + 2) * 4;
  L.size[MOE_WS_STATUS] = 4;
  L.size[MOE_WS_TILE_HIST] = ntiles * E * 4;
  L.size[MOE_WS_TILE_BASE] = ntiles * E * 4;
  const moe::FfnPlan plan =
      moe::ffn_plan(T, E, k, eff_capacity(s), R, padded(s), s->d, s->F, b);
  L.size[MOE_WS_SCHED] = moe::ffn_table_ints(plan) * 4;
  L.size[MOE_WS_X_PERM] = R * s->d * b;
  L.size[MOE_WS_H] = R * s->F * b;
  L.size[MOE_WS_Y_PERM] = R * s->d * b;
  L.size[MOE_WS_DOWN_ACC] = moe::ffn_down_acc_bytes(plan);
  int64_t o = 0;
  for (int i = 0; i < MOE_WS_COUNT; ++i) {
    L.off[i] = o;
    o += align_up(L.size[i]);
  }
  L.total = o;
  return L;
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

template <class P>
P* region(void* ws, const Layout& L, int r) {
  return reinterpret_cast<P*>(static_cast<char*>(ws) + L.off[r]);
}

int hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// Rows of x addressed by 32-bit byte offsets in the gathered gate/up GEMM.
bool gather_fits(const moe_shape* s) {
  return s->T * s->d * elt_bytes(s->dtype) < ((int64_t)1 << 31);
}

// moe_layer lets the gate/up GEMM gather the token rows (x_perm is not written) with packed
// rows whose x fits 32-bit offsets.
bool layer_gathers(const moe_shape* s) { return !padded(s) && gather_fits(s); }

int check_workspace(const moe_shape* s, const void* ws, size_t bytes, Layout* L) {
  *L = make_layout(s);
  if (!ws || (int64_t)bytes < L->total) return MOE_ERR_WORKSPACE;
  if (((uintptr_t)ws & (kAlign - 1)) != 0) return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}

// Argument checks of the dispatch (everything but the scratch tables).
int check_dispatch_args(const moe_shape* s, const int32_t* topk_idx, const void* x,
                        const int32_t* routed_counts, const int32_t* tokens_per_expert,
                        const int32_t* expert_offsets, const int32_t* src_token,
                        const int32_t* dest_row, const int32_t* drops, const void* x_perm) {
  int rc = check_shape(s);
  if (rc != MOE_OK) return rc;
  if (!routed_counts || !tokens_per_expert || !expert_offsets || !drops)
    return MOE_ERR_INVALID_ARG;
  if (s->T > 0 && (!topk_idx || !src_token || !dest_row || (x_perm && !x)))
    return MOE_ERR_INVALID_ARG;
  if (s->T > 0 && x_perm && (!aligned16(x) || !aligned16(x_perm))) return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}

// The dispatch launches, with the scratch tables tile_hist / tile_base ([ntiles, E] int32
// each) from the workspace or from the static array.
// With table set, the dispatch also writes the grouped GEMMs' tile table there, of row height
// table_bm with at most table_m_max tiles (moe_layer, moe_layer_fp8).
int dispatch_launch(const moe_shape* s, const int32_t* topk_idx, const void* x,
                    int32_t* tile_hist, int32_t* tile_base, int32_t* routed_counts,
                    int32_t* tokens_per_expert, int32_t* expert_offsets, int32_t* src_token,
                    int32_t* src_slot, int32_t* dest_row, int32_t* drops, void* x_perm,
                    hipStream_t st, int32_t* table = nullptr, int table_bm = 0,
                    int64_t table_m_max = 0) {
  moe::DispatchArgs a;
  a.topk_idx = topk_idx;
  a.x = x;
  a.T = s->T;
  a.d = s->d;
  a.E = s->E;
  a.k = s->k;
  a.C = eff_capacity(s);
  a.R = max_rows(s);
  a.elt_bytes = elt_bytes(s->dtype);
  a.slot_major = (s->flags & MOE_FLAG_SLOT_MAJOR) != 0;
  a.pad = padded(s);
  a.tile_hist = tile_hist;
  a.tile_base = tile_base;
  a.routed = routed_counts;
  a.kept = tokens_per_expert;
  a.offsets = expert_offsets;
  a.src_token = src_token;
  a.src_slot = src_slot;
  a.dest_row = dest_row;
  a.drops = drops;
  a.x_perm = x_perm;
  a.table = table;
  a.table_bm = table_bm;
  a.table_m_max = table_m_max;
  return hip_status(moe::launch_dispatch(a, st));
}

int route_impl(const moe_shape* s, const void* x, const void* w_router, const float* b_router,
               float* logits, int logits_given, int32_t* idx, float* gates, int32_t* status,
               hipStream_t st) {
  hipError_t e;
  // the status counter starts at zero: cleared by the router launch when there is one
  if (logits_given || s->T == 0) {
    if (status && (e = moe::launch_zero_i32(status, 1, st)) != hipSuccess) return MOE_ERR_HIP;
    if (s->T == 0) return MOE_OK;
  }
  // with a selection-only bias the logits stay unbiased and the bias goes to the top-k
  const bool sel_only = (s->flags & MOE_FLAG_BIAS_SELECTION_ONLY) != 0;
  if (!logits_given) {
    e = moe::launch_router_logits(s->dtype, x, w_router, sel_only ? nullptr : b_router, logits,
                                  s->T, s->d, s->E, status, st);
    if (e != hipSuccess) return MOE_ERR_HIP;
  }
  const int ng = grouped(s) ? s->n_groups : 1, mg = grouped(s) ? s->topk_groups : 1;
  return hip_status(moe::launch_topk(logits, sel_only ? b_router : nullptr, s->T, s->E, s->k,
                                     ng, mg, idx, gates, status, st));
}

}  // namespace

extern "C" {

int64_t moe_capacity(int64_t T, int64_t k, int64_t E, double cf) {
  if (T < 0 || k < 1 || E < 1 || !isfinite(cf)) return -1;
  if (!(cf > 0)) return 0;
  const double c = ceil(((cf * (double)T) * (double)k) / (double)E);
  if (!(c < 9.2233720368547758e18)) return -1;  // does not fit int64
  return (int64_t)c;
}

int64_t moe_max_rows(const moe_shape* s) {
  if (check_shape(s) != MOE_OK) return -1;
  return max_rows(s);
}

size_t moe_workspace_size(const moe_shape* s) {
  if (check_shape(s) != MOE_OK) return 0;
  return (size_t)make_layout(s).total;
}

int moe_workspace_layout(const moe_shape* s, int64_t* offsets) {
  int rc = check_shape(s);
  if (rc != MOE_OK) return rc;
  if (!offsets) return MOE_ERR_INVALID_ARG;
  const Layout L = make_layout(s);
  for (int i = 0; i < MOE_WS_COUNT; ++i) offsets[i] = L.off[i];
  return MOE_OK;
}

int moe_workspace_phases(const moe_shape* s, int64_t* bytes) {
  int rc = check_shape(s);
  if (rc != MOE_OK) return rc;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  const Layout L = make_layout(s);
  // regions moe_layer writes in each stage (with its optional outputs kept in the workspace);
  // its dispatch also writes the grouped GEMMs' tile table, and the per-tile scratch tables
  // only where it runs tiled (not in one block)
  static const int kPack[] = {MOE_WS_LOGITS,    MOE_WS_TOPK_IDX, MOE_WS_TOPK_W,
                              MOE_WS_STATUS,    MOE_WS_ROUTED,   MOE_WS_KEPT,
                              MOE_WS_OFFSETS,   MOE_WS_SRC_TOKEN, MOE_WS_DEST_ROW,
                              MOE_WS_DROPS,     MOE_WS_SCHED};
  static const int kExperts[] = {MOE_WS_H, MOE_WS_Y_PERM, MOE_WS_DOWN_ACC};
  int64_t pack = 0;
  for (int r : kPack) pack += L.size[r];
  if (!moe::dispatch_fused(s->T, s->k, s->E))
    pack += L.size[MOE_WS_TILE_HIST] + L.size[MOE_WS_TILE_BASE];
  if (!layer_gathers(s)) pack += L.size[MOE_WS_X_PERM];  // the copy the gathering GEMM skips
  int64_t experts = pack;
  // an empty layer writes its counters and status only: the expert GEMMs do not launch
  if (s->T > 0)
    for (int r : kExperts) experts += L.size[r];
  bytes[MOE_PHASE_BEFORE_LAYER] = 0;
  bytes[MOE_PHASE_AFTER_PACK] = pack;
  bytes[MOE_PHASE_AFTER_DISPATCH] = pack;  // expert-parallel size 1: nothing is exchanged
  bytes[MOE_PHASE_AFTER_EXPERTS] = experts;
  return MOE_OK;
}

const char* moe_status_string(int st) {
  switch (st) {
    case MOE_OK: return "ok";
    case MOE_ERR_INVALID_ARG: return "invalid argument";
    case MOE_ERR_UNSUPPORTED: return "unsupported shape or dtype";
    case MOE_ERR_ALIGNMENT: return "pointer not 16-byte aligned";
    case MOE_ERR_WORKSPACE: return "workspace missing or too small";
    case MOE_ERR_HIP: return "HIP launch failed";
    case MOE_ERR_SCRATCH: return "shape needs more than the static dispatch scratch";
    default: return "unknown status";
  }
}

int moe_route(const moe_shape* s, const void* x, const void* w_router, const float* b_router,
              float* logits, int logits_given, int32_t* topk_idx, float* topk_w,
              int32_t* status, hipStream_t st) {
  int rc = check_shape(s);
  if (rc != MOE_OK) return rc;
  if (s->T > 0 && (!logits || !topk_idx || !topk_w)) return MOE_ERR_INVALID_ARG;
  if (!logits_given && s->T > 0) {
    if (!x || !w_router) return MOE_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(w_router)) return MOE_ERR_ALIGNMENT;
  }
  return route_impl(s, x, w_router, b_router, logits, logits_given, topk_idx, topk_w, status,
                    st);
}

int moe_dispatch(const moe_shape* s, const int32_t* topk_idx, const void* x, void* ws,
                 size_t ws_bytes, int32_t* routed_counts, int32_t* tokens_per_expert,
                 int32_t* expert_offsets, int32_t* src_token, int32_t* src_slot,
                 int32_t* dest_row, int32_t* drops, void* x_perm, hipStream_t st) {
  int rc = check_dispatch_args(s, topk_idx, x, routed_counts, tokens_per_expert,
                               expert_offsets, src_token, dest_row, drops, x_perm);
  if (rc != MOE_OK) return rc;
  Layout L;
  if ((rc = check_workspace(s, ws, ws_bytes, &L)) != MOE_OK) return rc;
  return dispatch_launch(s, topk_idx, x, region<int32_t>(ws, L, MOE_WS_TILE_HIST),
                         region<int32_t>(ws, L, MOE_WS_TILE_BASE), routed_counts,
                         tokens_per_expert, expert_offsets, src_token, src_slot, dest_row,
                         drops, x_perm, st);
}

int moe_dispatch_no_workspace(const moe_shape* s, const int32_t* topk_idx, const void* x,
                              int32_t* routed_counts, int32_t* tokens_per_expert,
                              int32_t* expert_offsets, int32_t* src_token, int32_t* src_slot,
                              int32_t* dest_row, int32_t* drops, void* x_perm,
                              hipStream_t st) {
  int rc = check_dispatch_args(s, topk_idx, x, routed_counts, tokens_per_expert,
                               expert_offsets, src_token, dest_row, drops, x_perm);
  if (rc != MOE_OK) return rc;
  // the two scratch tables, each 256-byte aligned, in the static array
  const int64_t table = align_up(moe::dispatch_ntiles(s->T, s->k) * s->E * 4);
  if (2 * table > (int64_t)MOE_DISPATCH_SCRATCH_BYTES) return MOE_ERR_SCRATCH;
  void* scratch = nullptr;
  size_t bytes = 0;
  if (moe::dispatch_scratch(&scratch, &bytes) != hipSuccess) return MOE_ERR_HIP;
  if ((int64_t)bytes < 2 * table) return MOE_ERR_SCRATCH;
  int32_t* hist = static_cast<int32_t*>(scratch);
  int32_t* base = reinterpret_cast<int32_t*>(static_cast<char*>(scratch) + table);
  return dispatch_launch(s, topk_idx, x, hist, base, routed_counts, tokens_per_expert,
                         expert_offsets, src_token, src_slot, dest_row, drops, x_perm, st);
}

}  // extern "C"

namespace {

// Shared body of the expert-FFN entry points; which = 1 (gate/up), 2 (down), 3 (both).  The
// gate/up activations are x_perm, or, with src_rows, the rows src_rows[r] of x.
// With table_ready the workspace already holds the tile table of these offsets (moe_layer's
// dispatch wrote it).
int expert_ffn_impl(const moe_shape* s, int which, const void* x_perm, const void* x,
                    const int32_t* src_rows, void* h, const int32_t* expert_offsets,
                    const void* w_gate, const void* w_up, const void* w_down, void* ws,
                    size_t ws_bytes, void* y_perm, hipStream_t st, bool table_ready = false) {
  int rc = check_shape(s);
  if (rc != MOE_OK) return rc;
  if (s->T == 0) return MOE_OK;
  if (!expert_offsets) return MOE_ERR_INVALID_ARG;
  const void* act = src_rows ? x : x_perm;
  if ((which & 1) && (!act || !w_gate || !w_up || !h)) return MOE_ERR_INVALID_ARG;
  if ((which & 2) && (!w_down || !y_perm || !h)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(act) || !aligned16(w_gate) || !aligned16(w_up) || !aligned16(w_down) ||
      !aligned16(y_perm) || !aligned16(h))
    return MOE_ERR_ALIGNMENT;
  if (src_rows && !gather_fits(s)) return MOE_ERR_UNSUPPORTED;
  Layout L;
  if ((rc = check_workspace(s, ws, ws_bytes, &L)) != MOE_OK) return rc;
  moe::FfnArgs a;
  a.dtype = s->dtype;
  a.x_perm = x_perm;
  a.x = x;
  a.src_rows = src_rows;
  a.offsets = expert_offsets;
  a.w_gate = w_gate;
  a.w_up = w_up;
  a.w_down = w_down;
  a.T = s->T;
  a.d = s->d;
  a.E = s->E;
  a.k = s->k;
  a.F = s->F;
  a.C = eff_capacity(s);
  a.R = max_rows(s);
  a.pad = padded(s);
  a.h = h;
  a.sched = region<int32_t>(ws, L, MOE_WS_SCHED);
  a.y_perm = y_perm;
  a.down_acc = region<float>(ws, L, MOE_WS_DOWN_ACC);
  a.table_ready = table_ready;
  return hip_status(moe::launch_expert_ffn(a, which, st));
}

}  // namespace

extern "C" {

int moe_expert_ffn(const moe_shape* s, const void* x_perm, const int32_t* expert_offsets,
                   const void* w_gate, const void* w_up, const void* w_down, void* ws,
                   size_t ws_bytes, void* y_perm, hipStream_t st) {
  int rc = check_shape(s);
  if (rc != MOE_OK) return rc;
  Layout L;
  if (s->T > 0 && (rc = check_workspace(s, ws, ws_bytes, &L)) != MOE_OK) return rc;
  void* h = s->T > 0 ? region<void>(ws, L, MOE_WS_H) : nullptr;
  return expert_ffn_impl(s, 3, x_perm, nullptr, nullptr, h, expert_offsets, w_gate, w_up,
                         w_down, ws, ws_bytes, y_perm, st);
}

int moe_expert_gate_up(const moe_shape* s, const void* x_perm, const int32_t* expert_offsets,
                       const void* w_gate, const void* w_up, void* ws, size_t ws_bytes,
                       void* h, hipStream_t st) {
  return expert_ffn_impl(s, 1, x_perm, nullptr, nullptr, h, expert_offsets, w_gate, w_up,
                         nullptr, ws, ws_bytes, nullptr, st);
}

int moe_expert_gate_up_gathered(const moe_shape* s, const void* x, const int32_t* src_token,
                                const int32_t* expert_offsets, const void* w_gate,
                                const void* w_up, void* ws, size_t ws_bytes, void* h,
                                hipStream_t st) {
  int rc = check_shape(s);
  if (rc != MOE_OK) return rc;
  if (s->T > 0 && !src_token) return MOE_ERR_INVALID_ARG;
  return expert_ffn_impl(s, 1, nullptr, x, src_token, h, expert_offsets, w_gate, w_up,
                         nullptr, ws, ws_bytes, nullptr, st);
}

int moe_expert_down(const moe_shape* s, const void* h, const int32_t* expert_offsets,
                    const void* w_down, void* ws, size_t ws_bytes, void* y_perm,
                    hipStream_t st) {
  return expert_ffn_impl(s, 2, nullptr, nullptr, nullptr, const_cast<void*>(h), expert_offsets,
                         nullptr, nullptr, w_down, ws, ws_bytes, y_perm, st);
}

int moe_combine(const moe_shape* s, const void* y_perm, const int32_t* dest_row,
                const float* topk_w, void* out, hipStream_t st) {
  int rc = check_shape(s);
  if (rc != MOE_OK) return rc;
  if (s->T == 0) return MOE_OK;
  if (!y_perm || !dest_row || !topk_w || !out) return MOE_ERR_INVALID_ARG;
  if (!aligned16(y_perm) || !aligned16(out)) return MOE_ERR_ALIGNMENT;
  return hip_status(
      moe::launch_combine(s->dtype, y_perm, dest_row, topk_w, out, s->T, s->d, s->k, st));
}

int moe_slot_counts(const moe_shape* s, const int32_t* topk_idx, const int32_t* dest_row,
                    int32_t* routed_by_slot, int32_t* kept_by_slot, hipStream_t st) {
  int rc = check_shape(s);
  if (rc != MOE_OK) return rc;
  if (!routed_by_slot || !kept_by_slot) return MOE_ERR_INVALID_ARG;
  if (s->T > 0 && (!topk_idx || !dest_row)) return MOE_ERR_INVALID_ARG;
  return hip_status(moe::launch_slot_counts(topk_idx, dest_row, s->T, s->k, s->E,
                                            routed_by_slot, kept_by_slot, st));
}

int moe_layer(const moe_shape* s, const void* x, const void* w_router, const float* b_router,
              const void* w_gate, const void* w_up, const void* w_down, void* ws,
              size_t ws_bytes, void* out, int32_t* routed_counts, int32_t* tokens_per_expert,
              int32_t* drops, int32_t* status, hipStream_t st) {
  int rc = check_shape(s);
  if (rc != MOE_OK) return rc;
  if (!w_router || !w_gate || !w_up || !w_down) return MOE_ERR_INVALID_ARG;
  if (s->T > 0 && (!x || !out)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w_router) || !aligned16(w_gate) || !aligned16(w_up) ||
      !aligned16(w_down) || !aligned16(out))
    return MOE_ERR_ALIGNMENT;
  Layout L;
  if ((rc = check_workspace(s, ws, ws_bytes, &L)) != MOE_OK) return rc;
  float* logits = region<float>(ws, L, MOE_WS_LOGITS);
  int32_t* idx = region<int32_t>(ws, L, MOE_WS_TOPK_IDX);
  float* gates = region<float>(ws, L, MOE_WS_TOPK_W);
  int32_t* routed = routed_counts ? routed_counts : region<int32_t>(ws, L, MOE_WS_ROUTED);
  int32_t* kept = tokens_per_expert ? tokens_per_expert : region<int32_t>(ws, L, MOE_WS_KEPT);
  int32_t* offsets = region<int32_t>(ws, L, MOE_WS_OFFSETS);
  int32_t* src = region<int32_t>(ws, L, MOE_WS_SRC_TOKEN);
  int32_t* dest = region<int32_t>(ws, L, MOE_WS_DEST_ROW);
  int32_t* dr = drops ? drops : region<int32_t>(ws, L, MOE_WS_DROPS);
  int32_t* stt = status ? status : region<int32_t>(ws, L, MOE_WS_STATUS);
  void* x_perm = region<void>(ws, L, MOE_WS_X_PERM);
  void* y_perm = region<void>(ws, L, MOE_WS_Y_PERM);

  rc = route_impl(s, x, w_router, b_router, logits, 0, idx, gates, stt, st);
  if (rc != MOE_OK) return rc;
  // packed rows: the gate/up GEMM gathers the token rows itself (x_perm is not written)
  const bool gathered = layer_gathers(s);
  void* x_copy = gathered ? nullptr : x_perm;
  rc = check_dispatch_args(s, idx, x, routed, kept, offsets, src, dest, dr, x_copy);
  if (rc != MOE_OK) return rc;
  // the dispatch also writes the grouped GEMMs' tile table from the offsets it computes
  const moe::FfnPlan plan = moe::ffn_plan(s->T, s->E, s->k, eff_capacity(s), max_rows(s),
                                          padded(s), s->d, s->F, elt_bytes(s->dtype));
  rc = dispatch_launch(s, idx, x, region<int32_t>(ws, L, MOE_WS_TILE_HIST),
                       region<int32_t>(ws, L, MOE_WS_TILE_BASE), routed, kept, offsets, src,
                       nullptr, dest, dr, x_copy, st, region<int32_t>(ws, L, MOE_WS_SCHED),
                       plan.bm, plan.m_max);
  if (rc != MOE_OK) return rc;
  void* h = region<void>(ws, L, MOE_WS_H);
  rc = expert_ffn_impl(s, 1, gathered ? nullptr : x_perm, gathered ? x : nullptr,
                       gathered ? src : nullptr, h, offsets, w_gate, w_up, nullptr, ws,
                       ws_bytes, nullptr, st, /*table_ready=*/true);
  if (rc != MOE_OK) return rc;
  rc = expert_ffn_impl(s, 2, nullptr, nullptr, nullptr, h, offsets, nullptr, nullptr, w_down,
                       ws, ws_bytes, y_perm, st, /*table_ready=*/true);
  if (rc != MOE_OK) return rc;
  return moe_combine(s, y_perm, dest, gates, out, st);
}

}  // extern "C"

// ------------------------------------------------------------------------------------------
// 8-bit products and the gradients of the experts' products
// ------------------------------------------------------------------------------------------
namespace {

// tiles and pieces, numbered with 32 bits on the device and a block each in the few-tiles form
constexpr int64_t kMaxTiles = (int64_t)1 << 23;

int scale_bytes(int scale_type) { return scale_type == MOE_SCALE_E8M0 ? 1 : 4; }

bool known_scale(int scale_type) {
  return scale_type == MOE_SCALE_F32 || scale_type == MOE_SCALE_E8M0;
}

// a * b <= limit for positive a, b
bool product_within(int64_t a, int64_t b, int64_t limit) { return a <= limit / b; }

int check_group(const moe_group_shape* g) {
  if (!g) return MOE_ERR_INVALID_ARG;
  if (g->rows < 0 || g->E <= 0 || g->N <= 0 || g->K <= 0) return MOE_ERR_INVALID_ARG;
  if (g->dtype != MOE_F32 && g->dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  if (!known_scale(g->scale_type)) return MOE_ERR_UNSUPPORTED;
  if (g->E > kMaxE || g->rows >= ((int64_t)1 << 31)) return MOE_ERR_UNSUPPORTED;
  if (g->N % 128 != 0 || g->K % 128 != 0) return MOE_ERR_UNSUPPORTED;
  if (g->N > ((int64_t)1 << 20) || g->K > ((int64_t)1 << 20)) return MOE_ERR_UNSUPPORTED;
  if (moe::group_max_tiles(g->rows, g->E, g->N, g->K, elt_bytes(g->dtype)) >= kMaxTiles)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int64_t group_table_bytes(int64_t R, int64_t E, int elt) {
  const int64_t a = moe::group_table_ints(moe::fp8_plan(R, E));
  const int64_t b = moe::group_table_ints(moe::dgrad_plan(R, E, elt));
  return align_up((a > b ? a : b) * 4);
}

// The tile table, then the partial sums of split tiles.
int64_t group_workspace(const moe_group_shape* g) {
  const int elt = elt_bytes(g->dtype);
  const int64_t a = moe::fp8_split(g->rows, g->E, g->N, g->K).bytes;
  const int64_t b = moe::dgrad_split(g->rows, g->E, g->N, g->K, elt).bytes;
  return group_table_bytes(g->rows, g->E, elt) + (a > b ? a : b);
}
void* group_partial(const moe_group_shape* g, void* ws) {
  return static_cast<char*>(ws) + group_table_bytes(g->rows, g->E, elt_bytes(g->dtype));
}

// Checks shared by the grouped entry points; the operands are checked by the caller.
int check_group_call(const moe_group_shape* g, const int32_t* offsets, const void* ws,
                     size_t ws_bytes) {
  const int rc = check_group(g);
  if (rc != MOE_OK) return rc;
  if (!offsets && g->E != 1) return MOE_ERR_INVALID_ARG;
  if (!ws || (int64_t)ws_bytes < group_workspace(g))
    return MOE_ERR_WORKSPACE;
  if (((uintptr_t)ws & (kAlign - 1)) != 0) return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}

// The tile table of plan p in the workspace, where the launches read one; null otherwise.
int group_table(const moe_group_shape* g, const moe::GroupPlan& p, const int32_t* offsets,
                void* ws, int32_t** table, hipStream_t st) {
  *table = moe::group_needs_table(g->E) ? static_cast<int32_t*>(ws) : nullptr;
  if (!*table) return MOE_OK;
  return hip_status(
      moe::launch_tile_table(offsets, g->E, g->rows, p.bm, p.m_max, *table, st));
}

bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

int check_fp8(const moe_fp8_tensor* w, int scale_type) {
  if (!w || !w->q || !w->scale) return MOE_ERR_INVALID_ARG;
  if (!aligned16(w->q)) return MOE_ERR_ALIGNMENT;
  if (scale_type == MOE_SCALE_F32 && !aligned4(w->scale)) return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}

// Bytes of q and, 256-byte aligned behind it, the scales of [rows, K] activations.
int64_t fp8_rows_bytes(int64_t rows, int64_t K, int scale_type) {
  return align_up(rows * K) + rows * (K / 128) * scale_bytes(scale_type);
}

int check_fp8_shape(const moe_shape* s, int scale_type) {
  const int rc = check_shape(s);
  if (rc != MOE_OK) return rc;
  if (s->dtype != MOE_BF16 || !known_scale(scale_type)) return MOE_ERR_UNSUPPORTED;
  const int64_t R = max_rows(s), x_rows = s->T > R ? s->T : R;
  if (x_rows > 0 && (!product_within(x_rows, s->d, (int64_t)1 << 37) ||
                     !product_within(x_rows, s->F, (int64_t)1 << 37)))
    return MOE_ERR_UNSUPPORTED;
  // both products' tiles (either orientation)
  if (moe::group_max_tiles(R, s->E, s->F, s->d, 2) >= kMaxTiles) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// The regions of moe_layer with the row buffers in 8 bits.
Layout fp8_layout(const moe_shape* s, int scale_type) {
  Layout L = make_layout(s);
  const int64_t R = max_rows(s);
  L.size[MOE_WS_SCHED] = moe::group_table_ints(moe::fp8_plan(R, s->E)) * 4;
  L.size[MOE_WS_X_PERM] = fp8_rows_bytes(s->T > R ? s->T : R, s->d, scale_type);
  L.size[MOE_WS_H] = fp8_rows_bytes(R, s->F, scale_type);
  L.size[MOE_WS_DOWN_ACC] = moe::fp8_split(R, s->E, s->d, s->F).bytes;
  int64_t o = 0;
  for (int i = 0; i < MOE_WS_COUNT; ++i) {
    L.off[i] = o;
    o += align_up(L.size[i]);
  }
  L.total = o;
  return L;
}

int check_fp8_workspace(const moe_shape* s, int scale_type, const void* ws, size_t bytes,
                        Layout* L) {
  *L = fp8_layout(s, scale_type);
  if (!ws || (int64_t)bytes < L->total) return MOE_ERR_WORKSPACE;
  if (((uintptr_t)ws & (kAlign - 1)) != 0) return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}

int check_fp8_weights(const moe_fp8_tensor* w_gate, const moe_fp8_tensor* w_up,
                      const moe_fp8_tensor* w_down, int scale_type) {
  int rc = check_fp8(w_gate, scale_type);
  if (rc == MOE_OK) rc = check_fp8(w_up, scale_type);
  if (rc == MOE_OK) rc = check_fp8(w_down, scale_type);
  return rc;
}

// The expert launches over checked arguments: x quantized, gate/up, down.  With table_ready the
// workspace holds the tile table of these offsets, where the launches read one.
int fp8_experts(const moe_shape* s, int scale_type, const void* x, const int32_t* src_token,
                const int32_t* offsets, const moe_fp8_tensor* w_gate,
                const moe_fp8_tensor* w_up, const moe_fp8_tensor* w_down, void* ws,
                const Layout& L, void* y_perm, hipStream_t st, bool table_ready) {
  const int64_t R = max_rows(s), x_rows = src_token ? s->T : R;
  const int64_t cap = s->T > R ? s->T : R;  // rows the x region is laid out for
  char* xq = region<char>(ws, L, MOE_WS_X_PERM);
  char* hq = region<char>(ws, L, MOE_WS_H);
  int32_t* table =
      moe::group_needs_table(s->E) ? region<int32_t>(ws, L, MOE_WS_SCHED) : nullptr;
  hipError_t e = moe::launch_quantize(x_rows, s->d, 1, s->dtype, scale_type, x, xq,
                                      xq + align_up(cap * s->d), st);
  if (e != hipSuccess) return MOE_ERR_HIP;
  if (table && !table_ready) {
    const moe::GroupPlan p = moe::fp8_plan(R, s->E);
    if ((e = moe::launch_tile_table(offsets, s->E, R, p.bm, p.m_max, table, st)) != hipSuccess)
      return MOE_ERR_HIP;
  }
  moe::Fp8Args a = {};
  a.xq = xq;
  a.x_scale = xq + align_up(cap * s->d);
  a.src_rows = src_token;
  a.x_rows = x_rows;
  a.b0 = w_gate->q;
  a.b0_scale = w_gate->scale;
  a.b1 = w_up->q;
  a.b1_scale = w_up->scale;
  a.R = R;
  a.E = s->E;
  a.N = s->F;
  a.K = s->d;
  a.scale_type = scale_type;
  a.offsets = offsets;
  a.table = table;
  a.hq = hq;
  a.h_scale = hq + align_up(R * s->F);
  if ((e = moe::launch_fp8_gemm(a, st)) != hipSuccess) return MOE_ERR_HIP;
  a.xq = hq;
  a.x_scale = hq + align_up(R * s->F);
  a.src_rows = nullptr;
  a.x_rows = R;
  a.b0 = w_down->q;
  a.b0_scale = w_down->scale;
  a.b1 = a.b1_scale = nullptr;
  a.N = s->d;
  a.K = s->F;
  a.y = y_perm;
  a.hq = a.h_scale = nullptr;
  a.partial = region<void>(ws, L, MOE_WS_DOWN_ACC);
  return hip_status(moe::launch_fp8_gemm(a, st));
}

}  // namespace

extern "C" {

size_t moe_group_workspace_size(const moe_group_shape* g) {
  if (check_group(g) != MOE_OK) return 0;
  return (size_t)group_workspace(g);
}

int moe_quantize(int64_t rows, int64_t K, int64_t block_rows, int dtype, int scale_type,
                 const void* x, void* q, void* scale, hipStream_t st) {
  if (rows < 0 || K <= 0 || (block_rows != 1 && block_rows != 128)) return MOE_ERR_INVALID_ARG;
  if (rows % block_rows != 0) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  if (!known_scale(scale_type)) return MOE_ERR_UNSUPPORTED;
  // 2^37 values: a grid within 2^32 threads
  if (K % 128 != 0 || !product_within(rows > 0 ? rows : 1, K, ((int64_t)1 << 37) - 1))
    return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!x || !q || !scale) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(q)) return MOE_ERR_ALIGNMENT;
  if (scale_type == MOE_SCALE_F32 && !aligned4(scale)) return MOE_ERR_ALIGNMENT;
  return hip_status(
      moe::launch_quantize(rows, K, block_rows, dtype, scale_type, x, q, scale, st));
}

int moe_grouped_gemm_fp8(const moe_group_shape* g, const void* xq, const void* x_scale,
                         const int32_t* expert_offsets, const void* wq, const void* w_scale,
                         void* ws, size_t ws_bytes, void* y, hipStream_t st) {
  int rc = check_group_call(g, expert_offsets, ws, ws_bytes);
  if (rc != MOE_OK) return rc;
  if (g->dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  if (g->rows == 0) return MOE_OK;
  const moe_fp8_tensor x = {xq, x_scale}, w = {wq, w_scale};
  if ((rc = check_fp8(&x, g->scale_type)) != MOE_OK) return rc;
  if ((rc = check_fp8(&w, g->scale_type)) != MOE_OK) return rc;
  if (!y) return MOE_ERR_INVALID_ARG;
  if (!aligned16(y)) return MOE_ERR_ALIGNMENT;
  int32_t* table = nullptr;
  rc = group_table(g, moe::fp8_plan(g->rows, g->E), expert_offsets, ws, &table, st);
  if (rc != MOE_OK) return rc;
  moe::Fp8Args a = {};
  a.xq = xq;
  a.x_scale = x_scale;
  a.x_rows = g->rows;
  a.b0 = wq;
  a.b0_scale = w_scale;
  a.R = g->rows;
  a.E = g->E;
  a.N = g->N;
  a.K = g->K;
  a.scale_type = g->scale_type;
  a.offsets = expert_offsets;
  a.table = table;
  a.y = y;
  a.partial = group_partial(g, ws);
  return hip_status(moe::launch_fp8_gemm(a, st));
}

int moe_grouped_dgrad(const moe_group_shape* g, const void* dy, const int32_t* expert_offsets,
                      const void* w, void* ws, size_t ws_bytes, void* dx, hipStream_t st) {
  int rc = check_group_call(g, expert_offsets, ws, ws_bytes);
  if (rc != MOE_OK) return rc;
  if (g->rows == 0) return MOE_OK;
  if (!dy || !w || !dx) return MOE_ERR_INVALID_ARG;
  if (!aligned16(dy) || !aligned16(w) || !aligned16(dx)) return MOE_ERR_ALIGNMENT;
  int32_t* table = nullptr;
  rc = group_table(g, moe::dgrad_plan(g->rows, g->E, elt_bytes(g->dtype)), expert_offsets, ws,
                   &table, st);
  if (rc != MOE_OK) return rc;
  return hip_status(moe::launch_dgrad(g->dtype, dy, expert_offsets, table, w, dx,
                                      group_partial(g, ws), g->rows, g->E, g->N, g->K, st));
}

int moe_grouped_wgrad(const moe_group_shape* g, const void* dy, const void* x,
                      const int32_t* expert_offsets, void* ws, size_t ws_bytes, void* dw,
                      hipStream_t st) {
  const int rc = check_group_call(g, expert_offsets, ws, ws_bytes);
  if (rc != MOE_OK) return rc;
  // without rows every matrix is zeros: dy and x may be null
  if (!dw || (g->rows > 0 && (!dy || !x))) return MOE_ERR_INVALID_ARG;
  if (!aligned16(dy) || !aligned16(x) || !aligned16(dw)) return MOE_ERR_ALIGNMENT;
  return hip_status(moe::launch_wgrad(g->dtype, dy, x, expert_offsets, dw, g->rows, g->E, g->N,
                                      g->K, st));
}

size_t moe_fp8_workspace_size(const moe_shape* s, int scale_type) {
  if (check_fp8_shape(s, scale_type) != MOE_OK) return 0;
  return (size_t)fp8_layout(s, scale_type).total;
}

int moe_fp8_workspace_layout(const moe_shape* s, int scale_type, int64_t* offsets) {
  const int rc = check_fp8_shape(s, scale_type);
  if (rc != MOE_OK) return rc;
  if (!offsets) return MOE_ERR_INVALID_ARG;
  const Layout L = fp8_layout(s, scale_type);
  for (int i = 0; i < MOE_WS_COUNT; ++i) offsets[i] = L.off[i];
  return MOE_OK;
}

int moe_expert_ffn_fp8(const moe_shape* s, int scale_type, const void* x,
                       const int32_t* src_token, const int32_t* expert_offsets,
                       const moe_fp8_tensor* w_gate, const moe_fp8_tensor* w_up,
                       const moe_fp8_tensor* w_down, void* ws, size_t ws_bytes, void* y_perm,
                       hipStream_t st) {
  int rc = check_fp8_shape(s, scale_type);
  if (rc != MOE_OK) return rc;
  if (s->T == 0) return MOE_OK;
  if (!x || !expert_offsets || !y_perm) return MOE_ERR_INVALID_ARG;
  if ((rc = check_fp8_weights(w_gate, w_up, w_down, scale_type)) != MOE_OK) return rc;
  if (!aligned16(x) || !aligned16(y_perm)) return MOE_ERR_ALIGNMENT;
  if (src_token && s->T * s->d >= ((int64_t)1 << 31)) return MOE_ERR_UNSUPPORTED;
  Layout L;
  if ((rc = check_fp8_workspace(s, scale_type, ws, ws_bytes, &L)) != MOE_OK) return rc;
  return fp8_experts(s, scale_type, x, src_token, expert_offsets, w_gate, w_up, w_down, ws, L,
                     y_perm, st, /*table_ready=*/false);
}

int moe_layer_fp8(const moe_shape* s, int scale_type, const void* x, const void* w_router,
                  const float* b_router, const moe_fp8_tensor* w_gate,
                  const moe_fp8_tensor* w_up, const moe_fp8_tensor* w_down, void* ws,
                  size_t ws_bytes, void* out, int32_t* routed_counts,
                  int32_t* tokens_per_expert, int32_t* drops, int32_t* status, hipStream_t st) {
  int rc = check_fp8_shape(s, scale_type);
  if (rc != MOE_OK) return rc;
  if (!w_router) return MOE_ERR_INVALID_ARG;
  if ((rc = check_fp8_weights(w_gate, w_up, w_down, scale_type)) != MOE_OK) return rc;
  if (s->T > 0 && (!x || !out)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w_router) || !aligned16(out)) return MOE_ERR_ALIGNMENT;
  if (s->T * s->d >= ((int64_t)1 << 31)) return MOE_ERR_UNSUPPORTED;
  Layout L;
  if ((rc = check_fp8_workspace(s, scale_type, ws, ws_bytes, &L)) != MOE_OK) return rc;
  float* logits = region<float>(ws, L, MOE_WS_LOGITS);
  int32_t* idx = region<int32_t>(ws, L, MOE_WS_TOPK_IDX);
  float* gates = region<float>(ws, L, MOE_WS_TOPK_W);
  int32_t* routed = routed_counts ? routed_counts : region<int32_t>(ws, L, MOE_WS_ROUTED);
  int32_t* kept = tokens_per_expert ? tokens_per_expert : region<int32_t>(ws, L, MOE_WS_KEPT);
  int32_t* offsets = region<int32_t>(ws, L, MOE_WS_OFFSETS);
  int32_t* src = region<int32_t>(ws, L, MOE_WS_SRC_TOKEN);
  int32_t* dest = region<int32_t>(ws, L, MOE_WS_DEST_ROW);
  int32_t* dr = drops ? drops : region<int32_t>(ws, L, MOE_WS_DROPS);
  int32_t* stt = status ? status : region<int32_t>(ws, L, MOE_WS_STATUS);
  void* y_perm = region<void>(ws, L, MOE_WS_Y_PERM);
  rc = route_impl(s, x, w_router, b_router, logits, 0, idx, gates, stt, st);
  if (rc != MOE_OK) return rc;
  // tables only, the experts' tile table among them where the products read one: the gate/up
  // product gathers the rows
  const moe::GroupPlan p = moe::fp8_plan(max_rows(s), s->E);
  int32_t* table =
      moe::group_needs_table(s->E) ? region<int32_t>(ws, L, MOE_WS_SCHED) : nullptr;
  rc = dispatch_launch(s, idx, nullptr, region<int32_t>(ws, L, MOE_WS_TILE_HIST),
                       region<int32_t>(ws, L, MOE_WS_TILE_BASE), routed, kept, offsets, src,
                       nullptr, dest, dr, nullptr, st, table, p.bm, p.m_max);
  if (rc != MOE_OK || s->T == 0) return rc;
  rc = fp8_experts(s, scale_type, x, src, offsets, w_gate, w_up, w_down, ws, L, y_perm, st,
                   /*table_ready=*/true);
  if (rc != MOE_OK) return rc;
  return moe_combine(s, y_perm, dest, gates, out, st);
}

}  // extern "C"

// ------------------------------------------------------------------------------------------
// linear layers and clipping
// ------------------------------------------------------------------------------------------
namespace {

constexpr int64_t kMaxGrads = (int64_t)1 << 20;
static_assert(sizeof(moe_grad) == sizeof(moe::GradTensor), "one layout");

bool known_activation(int act) { return act >= MOE_ACT_NONE && act <= MOE_ACT_GELU_TANH; }

int64_t linear_table_bytes(const moe_group_shape* g) {
  return align_up(moe::group_table_ints(
                      moe::linear_plan(g->rows, g->E, g->N, elt_bytes(g->dtype))) *
                  4);
}
// Forward: the tile table, then the partial sums of split tiles; backward: the sums of dz by row
// tiles.
int64_t linear_workspace(const moe_group_shape* g) {
  const int64_t a = linear_table_bytes(g) +
                    moe::linear_split(g->rows, g->E, g->N, g->K, elt_bytes(g->dtype)).bytes;
  const int64_t b = align_up(moe::linear_grad_slots(g->rows, g->E) * g->N * 4);
  return a > b ? a : b;
}

int check_linear_call(const moe_group_shape* g, int act, const int32_t* offsets, const void* ws,
                      size_t ws_bytes) {
  const int rc = check_group(g);
  if (rc != MOE_OK) return rc;
  if (!known_activation(act)) return MOE_ERR_UNSUPPORTED;
  if (!offsets && g->E != 1) return MOE_ERR_INVALID_ARG;
  if (!ws || (int64_t)ws_bytes < linear_workspace(g)) return MOE_ERR_WORKSPACE;
  if (((uintptr_t)ws & (kAlign - 1)) != 0) return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}

int check_grads(int64_t count, const moe_grad* g, bool out) {
  if (count < 0 || (count > 0 && !g)) return MOE_ERR_INVALID_ARG;
  if (count > kMaxGrads) return MOE_ERR_UNSUPPORTED;
  for (int64_t i = 0; i < count; ++i) {
    if (g[i].n < 0) return MOE_ERR_INVALID_ARG;
    if (g[i].dtype != MOE_F32 && g[i].dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
    if (g[i].n >= ((int64_t)1 << 36)) return MOE_ERR_UNSUPPORTED;
    if (g[i].n == 0) continue;
    if (!g[i].grad || (out && !g[i].out)) return MOE_ERR_INVALID_ARG;
    const uintptr_t mask = (uintptr_t)elt_bytes((int32_t)g[i].dtype) - 1;
    if (((uintptr_t)g[i].grad & mask) != 0 || (out && ((uintptr_t)g[i].out & mask) != 0))
      return MOE_ERR_ALIGNMENT;
  }
  return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_linear_workspace_size(const moe_group_shape* g) {
  if (check_group(g) != MOE_OK) return 0;
  return (size_t)linear_workspace(g);
}

int moe_linear_tiles(const moe_group_shape* g, int64_t* tiles) {
  const int rc = check_group(g);
  if (rc != MOE_OK) return rc;
  if (!tiles) return MOE_ERR_INVALID_ARG;
  const int elt = elt_bytes(g->dtype);
  tiles[0] = moe::linear_plan(g->rows, g->E, g->N, elt).bm;
  tiles[1] = moe::linear_columns(g->rows, g->E, g->N, elt);
  tiles[2] = moe::linear_split(g->rows, g->E, g->N, g->K, elt).s_max;
  return MOE_OK;
}

int moe_grouped_linear(const moe_group_shape* g, int act, const void* x,
                       const int32_t* expert_offsets, const void* w, const float* bias,
                       const void* residual, void* ws, size_t ws_bytes, void* z, void* y,
                       hipStream_t st) {
  int rc = check_linear_call(g, act, expert_offsets, ws, ws_bytes);
  if (rc != MOE_OK) return rc;
  if (g->rows == 0) return MOE_OK;
  if (!x || !w || !y) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w) || !aligned16(bias) || !aligned16(residual) ||
      !aligned16(z) || !aligned16(y))
    return MOE_ERR_ALIGNMENT;
  moe::LinearArgs a = {};
  int32_t* table = nullptr;
  rc = group_table(g, moe::linear_plan(g->rows, g->E, g->N, elt_bytes(g->dtype)), expert_offsets,
                   ws, &table, st);
  if (rc != MOE_OK) return rc;
  a.dtype = g->dtype;
  a.act = act;
  a.x = x;
  a.w = w;
  a.offsets = expert_offsets;
  a.table = table;
  a.bias = bias;
  a.residual = residual;
  a.z = z;
  a.y = y;
  a.partial = static_cast<char*>(ws) + linear_table_bytes(g);
  a.R = g->rows;
  a.E = g->E;
  a.N = g->N;
  a.K = g->K;
  return hip_status(moe::launch_linear(a, st));
}

int moe_grouped_linear_grad(const moe_group_shape* g, int act, const void* dy, const void* z,
                            const int32_t* expert_offsets, void* ws, size_t ws_bytes, void* dz,
                            float* dbias, hipStream_t st) {
  const int rc = check_linear_call(g, act, expert_offsets, ws, ws_bytes);
  if (rc != MOE_OK) return rc;
  // without rows every sum is zero: dy and z may be null
  if (g->rows > 0 && (!dy || (!z && act != MOE_ACT_NONE))) return MOE_ERR_INVALID_ARG;
  if (!aligned16(dy) || !aligned16(z) || !aligned16(dz) || !aligned16(dbias))
    return MOE_ERR_ALIGNMENT;
  return hip_status(moe::launch_linear_grad(g->dtype, act, dy, z, expert_offsets, dz, dbias,
                                            static_cast<float*>(ws), g->rows, g->E, g->N, st));
}

size_t moe_grad_workspace_size(int64_t count) {
  if (count < 0 || count > kMaxGrads) return 0;
  return (size_t)align_up((moe::grad_norm_sums(count) + 1) * 8);
}

int moe_grad_norm(int64_t count, const moe_grad* grads, void* ws, size_t ws_bytes, float* norm,
                  hipStream_t st) {
  const int rc = check_grads(count, grads, false);
  if (rc != MOE_OK) return rc;
  if (!norm) return MOE_ERR_INVALID_ARG;
  if (!aligned4(norm)) return MOE_ERR_ALIGNMENT;
  if (!ws || ws_bytes < moe_grad_workspace_size(count)) return MOE_ERR_WORKSPACE;
  if (((uintptr_t)ws & (kAlign - 1)) != 0) return MOE_ERR_ALIGNMENT;
  return hip_status(moe::launch_grad_norm(count, reinterpret_cast<const moe::GradTensor*>(grads),
                                          static_cast<double*>(ws), norm, st));
}

int moe_grad_clip(int64_t count, const moe_grad* grads, float max_norm, const float* norm,
                  hipStream_t st) {
  const int rc = check_grads(count, grads, true);
  if (rc != MOE_OK) return rc;
  if (!norm || !(max_norm >= 0) || !isfinite(max_norm)) return MOE_ERR_INVALID_ARG;
  if (!aligned4(norm)) return MOE_ERR_ALIGNMENT;
  return hip_status(moe::launch_grad_clip(
      count, reinterpret_cast<const moe::GradTensor*>(grads), max_norm, norm, st));
}

}  // extern "C"

// ------------------------------------------------------------------------------------------
// the whole layer for a few tokens
// ------------------------------------------------------------------------------------------
namespace {

int check_few_shape(const moe_shape* s) {
  const int rc = check_shape(s);
  if (rc != MOE_OK) return rc;
  if (s->T > MOE_FEW_MAX_TOKENS || s->T * s->k > moe::kFewPairs) return MOE_ERR_UNSUPPORTED;
  // h is read with 32-bit offsets
  if (s->T * s->k * s->F * elt_bytes(s->dtype) >= ((int64_t)1 << 31) - 4096)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

struct FewLayout {
  int64_t counters, h, partial, total;  // the logits come first
};
FewLayout few_layout(const moe_shape* s) {
  FewLayout L;
  L.counters = align_up(s->T * s->E * 4);
  L.h = L.counters + align_up((moe::kFewCounters + s->d / 16) * 4);
  L.partial = L.h + align_up(s->T * s->k * s->F * elt_bytes(s->dtype));
  L.total = L.partial + align_up(moe::kFewChunks * s->T * s->d * 4);
  return L;
}

// The launches over checked weights.
int few_layer(const moe_shape* s, int scale_type, const void* x, const void* w_router,
              const float* b_router, const void* const (&w)[3], const void* const (&w_scale)[3],
              void* ws, size_t ws_bytes, void* out, int32_t* routed_counts,
              int32_t* tokens_per_expert, int32_t* drops, int32_t* status, hipStream_t st) {
  if (!w_router) return MOE_ERR_INVALID_ARG;
  if (s->T > 0 && (!x || !out)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w_router) || !aligned16(out)) return MOE_ERR_ALIGNMENT;
  const FewLayout L = few_layout(s);
  if (!ws || (int64_t)ws_bytes < L.total) return MOE_ERR_WORKSPACE;
  if (((uintptr_t)ws & (kAlign - 1)) != 0) return MOE_ERR_ALIGNMENT;
  const bool sel_only = (s->flags & MOE_FLAG_BIAS_SELECTION_ONLY) != 0;
  moe::FewArgs a = {};
  a.dtype = s->dtype;
  a.scale_type = scale_type;
  a.x = x;
  a.w_router = w_router;
  a.bias = sel_only ? nullptr : b_router;
  a.sel_bias = sel_only ? b_router : nullptr;
  for (int i = 0; i < 3; ++i) {
    a.w[i] = w[i];
    a.w_scale[i] = w_scale[i];
  }
  a.logits = static_cast<float*>(ws);
  a.h = static_cast<char*>(ws) + L.h;
  a.partial = reinterpret_cast<float*>(static_cast<char*>(ws) + L.partial);
  a.counters = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + L.counters);
  a.out = out;
  a.routed = routed_counts;
  a.kept = tokens_per_expert;
  a.drops = drops;
  a.status = status;
  a.T = s->T;
  a.d = s->d;
  a.E = s->E;
  a.k = s->k;
  a.F = s->F;
  a.C = eff_capacity(s);
  a.n_groups = grouped(s) ? s->n_groups : 1;
  a.topk_groups = grouped(s) ? s->topk_groups : 1;
  a.slot_major = (s->flags & MOE_FLAG_SLOT_MAJOR) != 0;
  return hip_status(moe::launch_few(a, st));
}

}  // namespace

extern "C" {

int32_t moe_few_wait_polls(int32_t polls) { return moe::few_wait_polls(polls); }

size_t moe_few_workspace_size(const moe_shape* s) {
  if (check_few_shape(s) != MOE_OK) return 0;
  return (size_t)few_layout(s).total;
}

int moe_layer_few(const moe_shape* s, const void* x, const void* w_router, const float* b_router,
                  const void* w_gate, const void* w_up, const void* w_down, void* ws,
                  size_t ws_bytes, void* out, int32_t* routed_counts, int32_t* tokens_per_expert,
                  int32_t* drops, int32_t* status, hipStream_t st) {
  const int rc = check_few_shape(s);
  if (rc != MOE_OK) return rc;
  if (!w_gate || !w_up || !w_down) return MOE_ERR_INVALID_ARG;
  if (!aligned16(w_gate) || !aligned16(w_up) || !aligned16(w_down)) return MOE_ERR_ALIGNMENT;
  const void* const w[3] = {w_gate, w_up, w_down};
  const void* const none[3] = {nullptr, nullptr, nullptr};
  return few_layer(s, -1, x, w_router, b_router, w, none, ws, ws_bytes, out, routed_counts,
                   tokens_per_expert, drops, status, st);
}

int moe_layer_few_fp8(const moe_shape* s, int scale_type, const void* x, const void* w_router,
                      const float* b_router, const moe_fp8_tensor* w_gate,
                      const moe_fp8_tensor* w_up, const moe_fp8_tensor* w_down, void* ws,
                      size_t ws_bytes, void* out, int32_t* routed_counts,
                      int32_t* tokens_per_expert, int32_t* drops, int32_t* status,
                      hipStream_t st) {
  int rc = check_few_shape(s);
  if (rc != MOE_OK) return rc;
  if (s->dtype != MOE_BF16 || !known_scale(scale_type)) return MOE_ERR_UNSUPPORTED;
  if ((rc = check_fp8_weights(w_gate, w_up, w_down, scale_type)) != MOE_OK) return rc;
  const void* const w[3] = {w_gate->q, w_up->q, w_down->q};
  const void* const scale[3] = {w_gate->scale, w_up->scale, w_down->scale};
  return few_layer(s, scale_type, x, w_router, b_router, w, scale, ws, ws_bytes, out,
                   routed_counts, tokens_per_expert, drops, status, st);
}

}  // extern "C"
