// The whole layer for at most 16 tokens: router, selection, the chosen experts' SwiGLU networks and
// the gate-weighted sum.
//
//   logits = x w_router^T + b (64-bit sums, rounded once);  top-k, gates;
//   h = silu(x Wg^T) * (x Wu^T), rounded to x's type;  out = sum over experts of gate (h Wd^T)
//
// Bound by HBM: a chosen expert's weights are read once, whatever the number of its tokens, and
// everything else is small.  No rows are packed: the matrix instruction's sixteen columns are the
// tokens themselves, each expert is multiplied with all of them, and what a token did not choose is
// not stored (h) or not added (out).  Every block finds the routing for itself from the logits,
// since its cost is less than another launch's.
//
// A block is eight waves on one CU that take items in turn: gate/up, 8 or 16 columns of an expert's
// hidden layer; down, 16 or 32 output columns over all chosen experts.  The eight waves split an
// item's reduction, counted in units of 128 bytes of a weight row.  Weights and the rows they meet
// come in whole lines, eight rows of 128 bytes a load, into registers, one group of units ahead of
// the one that is multiplied, across the items' borders; a wave turns them into the matrix
// instruction's layout through its own part of the LDS, without a barrier.  At an item's end the
// waves' sums meet in LDS, where one wave, a different one each time, adds them in wave order and
// finishes the item, while the others go on.
#include <algorithm>

#include "fp8_common.h"
#include "gemm_common.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kWaves = 8, kThreads = kWaves * kWave, kTokens = 16;

typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) f32x4 lds_f32x4;

// Weights' kinds.
struct W16 {  // bf16
  typedef bf16 X;
  static constexpr int kElt = 2, kScale = 0, kXBytes = 128;
};
struct W32 {
  typedef float X;
  static constexpr int kElt = 4, kScale = 0, kXBytes = 128;
};
template <int SCALE_BYTES>
struct W8 {  // e4m3 with fp32 or E8M0 scales, bf16 rows: 128 values a unit
  typedef bf16 X;
  static constexpr int kElt = 1, kScale = SCALE_BYTES, kXBytes = 256;
};

struct Weight {
  const char* q;
  const char* scale;
};

struct FewKern {
  const void* x;  // [T, d]
  const float* logits;
  const float* sel_bias;  // nullable
  Weight gate, up, down;
  void* h;  // [T k, F]
  void* out;
  int32_t* routed;
  int32_t* kept;
  int32_t* drops;
  int32_t* status;
  int T, d, E, k, F, C, n_groups, topk_groups, slot_major;
};

// ---------------------------------------------------------------------------------------
// router logits
// ---------------------------------------------------------------------------------------
// One block for each expert; a product of two bf16 (fp32) values is exact in 64 bits and so are,
// for a logit, the sums: the selection is that of the exact logits rounded to fp32.
template <class T, int TT>
__global__ void __launch_bounds__(256)
few_logits_kernel(const T* __restrict__ x, const T* __restrict__ w, const float* __restrict__ b,
                  float* __restrict__ logits, int tokens, int d, int E) {
  constexpr int V = 16 / sizeof(T);
  typedef T tx __attribute__((ext_vector_type(V)));
  __shared__ double part[4][TT];
  const int e = blockIdx.x, tid = threadIdx.x;
  double sum[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) sum[t] = 0.0;
  for (int i = tid * V; i < d; i += 256 * V) {
    const tx wv = *reinterpret_cast<const tx*>(w + (int64_t)e * d + i);
    tx xv[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t)
      if (t < tokens) xv[t] = *reinterpret_cast<const tx*>(x + (int64_t)t * d + i);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const double wd = (double)Elt<T>::to_f32(wv[j]);
#pragma unroll
      for (int t = 0; t < TT; ++t)
        if (t < tokens) sum[t] = fma(wd, (double)Elt<T>::to_f32(xv[t][j]), sum[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < TT; ++t) {
#pragma unroll
    for (int m = 1; m < kWave; m <<= 1)
      sum[t] += __longlong_as_double(
          (long long)shfl_xor_u64((uint64_t)__double_as_longlong(sum[t]), m));
    if (lane_id() == 0) part[tid / kWave][t] = sum[t];
  }
  __syncthreads();
  if (tid < TT && tid < tokens) {
    const double v = part[0][tid] + part[1][tid] + part[2][tid] + part[3][tid];
    logits[(int64_t)tid * E + e] = (float)(b ? v + (double)b[e] : v);
  }
}

// ---------------------------------------------------------------------------------------
// routing, in every block
// ---------------------------------------------------------------------------------------
// The block's tables, in LDS.
struct Routing {
  uint8_t* slot;     // [E][16]: 1 + the slot in which a token chose an expert and was kept, or 0
  float* gate_of;    // [T k]
  float* gates;      // [active][16]: a token's gate, -1 where it did not choose the expert
  uint16_t* active;  // experts with tokens, in order
  int count;
};

__host__ __device__ inline int few_active_max(int T, int k, int E) { return min(E, T * k); }
// slot, gate_of, gates, active and what their making needs (selected experts, group keys, scans)
__host__ __device__ inline int few_routing_bytes(int T, int k, int E) {
  const int a = few_active_max(T, k, E);
  const int bytes = E * 16 + T * k * 4 + a * 64 + (a * 2 + 15) / 16 * 16 + (T * k * 2 + 15) / 16 * 16;
  return (bytes + 15) / 16 * 16;
}

__device__ inline uint32_t ordered_key(float v) {
  if (v == 0.0f) v = 0.0f;  // -0.0 == +0.0
  const uint32_t u = __float_as_uint(v);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Largest of a wave, to all lanes.
__device__ inline uint32_t wave_max_u32(uint32_t v) {
  auto step = [&](auto ctrl, auto rows) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value,
                                                             decltype(rows)::value, 0xF, false);
    v = o > v ? o : v;
  };
  step(IntC<0x111>{}, IntC<0xF>{});  // row_shr:1, 2, 4, 8
  step(IntC<0x112>{}, IntC<0xF>{});
  step(IntC<0x114>{}, IntC<0xF>{});
  step(IntC<0x118>{}, IntC<0xF>{});
  step(IntC<0x142>{}, IntC<0xA>{});  // row_bcast:15, 31
  step(IntC<0x143>{}, IntC<0xC>{});
  return (uint32_t)__builtin_amdgcn_readlane((int)v, kWave - 1);
}

// A token's k experts, slot j on lane j: value descending, index ascending, as moe_route selects.
// Returns whether a logit is not finite (such a logit is not selected).
__device__ inline bool few_select(const float* __restrict__ row, const float* __restrict__ sel_bias,
                                  int E, int k, int n_groups, int topk_groups, uint32_t* group_key,
                                  int* slot_e) {
  constexpr int V = 1024 / kWave;
  const int lane = lane_id();
  uint32_t key[V];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    key[i] = 0;
    if (i * kWave >= E) continue;
    const int e = i * kWave + lane;
    if (e < E) {
      const float v = row[e], s = sel_bias ? v + sel_bias[e] : v;
      if (__builtin_isfinite(v) && __builtin_isfinite(s))
        key[i] = ordered_key(s);
      else
        bad = true;
    }
  }
  if (n_groups > 1) {  // topk_groups groups of consecutive experts by their best logit
    const int size = E / n_groups;
    group_key[lane] = 0;
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (i * kWave >= E) continue;
      const int e = i * kWave + lane;
      if (e < E) atomicMax(&group_key[e / size], key[i]);
    }
    __builtin_amdgcn_wave_barrier();
    uint32_t mine = *(volatile uint32_t*)&group_key[lane];
    uint64_t chosen = 0;
    for (int r = 0; r < topk_groups; ++r) {
      const uint32_t best = wave_max_u32(mine);
      if (best == 0) break;  // only tokens with non-finite logits get here
      const int g = __builtin_ctzll(__ballot(mine == best));
      chosen |= 1ull << g;
      if (lane == g) mine = 0;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (i * kWave >= E) continue;
      const int e = i * kWave + lane;
      if (e < E && !((chosen >> (e / size)) & 1ull)) key[i] = 0;
    }
  }
  int picked = 0;
  for (int j = 0; j < k; ++j) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i * kWave < E) best = max(best, key[i]);
    best = wave_max_u32(best);
    int e = 0;
    if (best != 0) {
      bool found = false;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (i * kWave >= E || found) continue;
        const uint64_t m = __ballot(key[i] == best);
        if (m) {
          const int l = __builtin_ctzll(m);
          e = i * kWave + l;
          if (lane == l) key[i] = 0;
          found = true;
        }
      }
    }
    if (lane == j) picked = e;
  }
  *slot_e = picked;
  return __ballot(bad) != 0;
}

// Every thread of the block calls this.  `smem`: few_routing_bytes(); report: this block writes the
// counts.
__device__ inline Routing few_routing(const FewKern& a, char* smem, bool report) {
  __shared__ uint32_t group_key[kWaves][kWave];
  __shared__ int scan[17];
  __shared__ int tally[66 + 1];  // drops, then status
  const int tid = threadIdx.x, lane = lane_id(), wave = tid / kWave;
  const int T = a.T, E = a.E, k = a.k, pairs = T * k, most = few_active_max(T, k, E);
  Routing r;
  r.slot = reinterpret_cast<uint8_t*>(smem);
  r.gate_of = reinterpret_cast<float*>(smem + E * 16);
  r.gates = r.gate_of + pairs;
  r.active = reinterpret_cast<uint16_t*>(r.gates + most * 16);
  uint16_t* sel = r.active + (most * 2 + 15) / 16 * 8;
  u32x4* slot4 = reinterpret_cast<u32x4*>(smem);
  for (int e = tid; e < E; e += kThreads) slot4[e] = u32x4{0, 0, 0, 0};
  if (tid < 67) tally[tid] = 0;
  __syncthreads();
  for (int t = wave; t < T; t += kWaves) {
    int e;
    const float* row = a.logits + (int64_t)t * E;
    const bool bad = few_select(row, a.sel_bias, E, k, a.n_groups, a.topk_groups,
                                group_key[wave], &e);
    // gates: softmax over the selection
    const float l = lane < k ? row[e] : -__builtin_huge_valf();
    float m = l;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) m = fmaxf(m, __shfl_xor(m, o, kWave));
    const float ex = lane < k ? expf(l - m) : 0.f;
    float sum = ex;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) sum += __shfl_xor(sum, o, kWave);
    if (lane < k) {
      sel[t * k + lane] = (uint16_t)e;
      r.gate_of[t * k + lane] = ex / sum;
      r.slot[e * 16 + t] = (uint8_t)(lane + 1);
    }
    if (bad && lane == 0) atomicAdd(&tally[66], 1);
  }
  __syncthreads();
  if (report && a.routed) {
    for (int e = tid; e < E; e += kThreads) {
      int n = 0;
      for (int t = 0; t < T; ++t) n += r.slot[e * 16 + t] != 0;
      a.routed[e] = n;
    }
  }
  if (a.C < T) {  // some may be dropped: count the earlier assignments to the same expert
    int drop = 0;  // this thread's pairs (at most 512 of them in all)
    const int t = tid / k, j = tid - t * k;
    if (tid < pairs) {
      int before = 0;
      const int e = sel[tid];
      for (int o = 0; o < T; ++o) {
        const int s = r.slot[e * 16 + o];
        if (s && (a.slot_major ? s - 1 < j || (s - 1 == j && o < t) : o < t)) ++before;
      }
      drop = before >= a.C;
    }
    __syncthreads();
    if (drop) {
      r.slot[sel[tid] * 16 + t] = 0;
      atomicAdd(&tally[0], 1);
      atomicAdd(&tally[1 + j], 1);
      sel[tid] = 0xffff;
    }
    __syncthreads();
    if (report && tid < T) {
      bool none = true;
      for (int i = 0; i < k; ++i) none = none && sel[tid * k + i] == 0xffff;
      if (none) atomicAdd(&tally[k + 1], 1);
    }
    __syncthreads();
  }
  if (report) {
    if (a.kept)
      for (int e = tid; e < E; e += kThreads) {
        int n = 0;
        for (int t = 0; t < T; ++t) n += r.slot[e * 16 + t] != 0;
        a.kept[e] = n;
      }
    if (a.drops && tid < k + 2) a.drops[tid] = tally[tid];
    if (a.status && tid == 0) *a.status = tally[66];
  }
  // experts with tokens, in order
  int count = 0;
  for (int e0 = 0; e0 < E; e0 += kThreads) {
    const int e = e0 + tid;
    bool any = false;
    if (e < E) {
      const u32x4 v = slot4[e];
      any = (v[0] | v[1] | v[2] | v[3]) != 0;
    }
    int total;
    const int at = count + block_exclusive_scan(any ? 1 : 0, scan, &total);
    if (any) r.active[at] = (uint16_t)e;
    count += total;
  }
  __syncthreads();
  for (int i = tid; i < count * kTokens; i += kThreads) {
    const int t = i & 15, s = r.slot[r.active[i >> 4] * 16 + t];
    r.gates[i] = s ? r.gate_of[t * k + s - 1] : -1.f;
  }
  __syncthreads();
  r.count = __builtin_amdgcn_readfirstlane(count);
  return r;
}

// ---------------------------------------------------------------------------------------
// the experts
// ---------------------------------------------------------------------------------------
typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Eight e4m3 values as bf16 (exact).
__device__ inline u32x4 e4m3_to_bf16(uint32_t lo, uint32_t hi) {
  u32x4 r;
  r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true));
  r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false));
  r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true));
  return r;
}

// 2^(v - 127), 255 NaN
__device__ inline float e8m0_value(uint32_t v) {
  return __uint_as_float(v == 0 ? 0x00400000u : v == 255 ? 0x7fc00000u : v << 23);
}

// TP: tokens' rows that are loaded (8 or 16); RT: MFMA tiles of 16 weight rows an item has; G: units
// of a group.
template <class W, int TP_, int RT_, int G_>
struct FewTile {
  static constexpr int TP = TP_, RT = RT_, G = G_;
  static constexpr int kWLoads = 2 * RT;                     // of 1024 bytes, per unit
  static constexpr int kXLoads = TP * W::kXBytes / 1024;
  static constexpr int kSlot = RT * 2048 + TP * W::kXBytes;  // a wave's LDS
  static constexpr int kSums = 2 * kWaves * RT * 1024;       // two items' sums
  static constexpr int kLds = kWaves * kSlot + kSums;
};

template <class W, class P, bool DOWN>
__global__ void __launch_bounds__(kThreads) few_kernel(const FewKern a) {
  extern __shared__ __attribute__((aligned(1024))) char smem_dyn[];
  typedef typename W::X X;
  constexpr int RT = P::RT, G = P::G, NW = P::kWLoads, NX = P::kXLoads, ES = W::kScale;
  constexpr int kScales = !W::kScale ? 0 : DOWN || RT == 1 ? 1 : 2;
  const Routing r = few_routing(a, smem_dyn + P::kLds, !DOWN && blockIdx.x == 0);
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int c = lane & 15, g = lane >> 4;
  lds_char* slot = (lds_char*)smem_dyn + wave * P::kSlot;
  lds_char* sums = (lds_char*)smem_dyn + kWaves * P::kSlot;

  // Items and, of each, this wave's units [u0, u1): the reduction's units (down: of every chosen
  // expert, one behind the other).
  const int K = DOWN ? a.F : a.d, N = DOWN ? a.d : a.F;
  constexpr int kCols = DOWN ? 16 * RT : 8 * RT;  // columns of an item
  const int per_k = K * W::kElt / 128, tiles = N / kCols;
  const int items = DOWN ? tiles : r.count * tiles;
  const int units = DOWN ? r.count * per_k : per_k;
  const int u0 = (int)((int64_t)wave * units / kWaves), u1 = (int)((int64_t)(wave + 1) * units / kWaves);
  const uint32_t pitch = (uint32_t)K * W::kElt;
  const uint32_t vw = (uint32_t)(lane >> 3) * pitch + (uint32_t)(lane & 7) * 16;
  const uint32_t x_pitch = (uint32_t)K * (uint32_t)sizeof(X);
  const auto rx = bounded_rsrc(uniform_u64(DOWN ? a.h : a.x),
                               (int64_t)(DOWN ? a.T * a.k : a.T) * x_pitch);
  constexpr uint32_t kNone = 0x7fffff00u;  // past the resource's end: loads as zeros
  // x load i: 128-byte part i * 8 / TP of the unit's row, tokens (i * 8) % TP + L / 8
  auto x_token = [&](int i) { return (i * 8) % P::TP + (lane >> 3); };
  const int64_t matrix = (int64_t)N * pitch;

  struct Group {
    u32x4 w[G][NW], x[G][NX];
    uint32_t s[G][kScales ? kScales : 1];
  };
  // unit u of item q: where its expert stands in the list, and the unit of the row
  struct Unit {
    int at, k;
  };
  auto unit_of = [&](int q, int u) {
    if constexpr (DOWN) return Unit{u / per_k, u % per_k};
    return Unit{q / tiles, u};
  };
  auto load = [&](Group& o, int q, int u) {
    const int col0 = (DOWN ? q : q % tiles) * kCols;
#pragma unroll
    for (int i = 0; i < G; ++i) {
      if (u + i >= u1) break;
      const Unit v = unit_of(q, u + i);
      const int e = __builtin_amdgcn_readfirstlane((int)r.active[v.at]);
      const int64_t first = (int64_t)e * matrix + (int64_t)col0 * pitch;
      const auto r0 = buffer_rsrc(uniform_u64((DOWN ? a.down.q : a.gate.q) + first));
      const auto r1 = buffer_rsrc(uniform_u64((DOWN ? a.down.q : a.up.q) + first));
#pragma unroll
      for (int n = 0; n < NW; ++n) {
        const bool second = !DOWN && n >= RT;  // the up rows
        const uint32_t row = (uint32_t)(second ? n - RT : n) * 8u * pitch;
        o.w[i][n] = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(second ? r1 : r0, vw,
                                                         row + (uint32_t)v.k * 128u, 2));
      }
#pragma unroll
      for (int n = 0; n < NX; ++n) {
        const int t = x_token(n);
        uint32_t off = kNone;
        if constexpr (DOWN) {
          const int s = r.slot[e * 16 + t];
          if (s) off = (uint32_t)(t * a.k + s - 1) * x_pitch;
        } else {
          if (t < a.T) off = (uint32_t)t * x_pitch;
        }
        if (off != kNone) off += (uint32_t)(lane & 7) * 16 + (uint32_t)(n * 8 / P::TP) * 128u;
        o.x[i][n] = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, off, (uint32_t)v.k * W::kXBytes, 0));
      }
      if constexpr (kScales > 0) {
        const int kb = K / 128, row = (int)((int64_t)col0 / 128);
        const int64_t at = ((int64_t)e * (N / 128) + row) * kb + v.k;
        auto scale = [&](const char* p) -> uint32_t {
          if constexpr (ES == 4) return *reinterpret_cast<const uint32_t*>(p + at * 4);
          return *reinterpret_cast<const uint8_t*>(p + at);
        };
        if constexpr (DOWN) {
          o.s[i][0] = scale(a.down.scale);
        } else if constexpr (RT == 1) {
          o.s[i][0] = scale(g < 2 ? a.gate.scale : a.up.scale);
        } else {
          o.s[i][0] = scale(a.gate.scale);
          o.s[i][1] = scale(a.up.scale);
        }
      }
    }
  };

  f32x4 acc[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto lds_at = [&](int row, int piece) { return row * 128 + ((piece ^ ((row >> 1) & 7)) << 4); };
  lds_char* xs = slot + RT * 2048;
  auto multiply = [&](const Group& o, int q, int u) {
#pragma unroll
    for (int i = 0; i < G; ++i) {
      if (u + i >= u1) break;
#pragma unroll
      for (int n = 0; n < NW; ++n)
        *reinterpret_cast<lds_u32x4*>(slot + lds_at(n * 8 + (lane >> 3), lane & 7)) = o.w[i][n];
#pragma unroll
      for (int n = 0; n < NX; ++n)  // parts of TP rows of 128 bytes
        *reinterpret_cast<lds_u32x4*>(xs + (n * 8 / P::TP) * (P::TP * 128) +
                                      lds_at(x_token(n), lane & 7)) = o.x[i][n];
      __builtin_amdgcn_wave_barrier();
      f32x4 p[RT];
#pragma unroll
      for (int t = 0; t < RT; ++t) p[t] = f32x4{0.f, 0.f, 0.f, 0.f};
      const int xr = c & (P::TP - 1);
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        u32x4 w[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t)
          w[t] = *reinterpret_cast<const lds_u32x4*>(slot + lds_at(t * 16 + c, ks * 4 + g));
        if constexpr (W::kElt == 1) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const u32x4 x = *reinterpret_cast<const lds_u32x4*>(xs + ks * (P::TP * 128) +
                                                                lds_at(xr, 2 * g + h));
#pragma unroll
            for (int t = 0; t < RT; ++t)
              mma_chunk(p[t], e4m3_to_bf16(w[t][2 * h], w[t][2 * h + 1]), x, bf16());
          }
        } else {
          const u32x4 x = *reinterpret_cast<const lds_u32x4*>(xs + lds_at(xr, ks * 4 + g));
#pragma unroll
          for (int t = 0; t < RT; ++t) mma_chunk(p[t], w[t], x, X());
        }
      }
      __builtin_amdgcn_wave_barrier();
      float f[RT];
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        f[t] = 1.f;
        if constexpr (kScales > 0) {
          const uint32_t s = o.s[i][kScales == 2 ? t : 0];
          f[t] = ES == 4 ? __uint_as_float(s) : e8m0_value(s);
        }
      }
      if constexpr (DOWN) {
        const float gate = r.gates[unit_of(q, u + i).at * kTokens + c];
        // a token that did not choose the expert takes nothing of it, be it infinite or NaN
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          const float v = f[t] * gate;
#pragma unroll
          for (int b = 0; b < 4; ++b) acc[t][b] = gate < 0.f ? acc[t][b] : fmaf(p[t][b], v, acc[t][b]);
        }
      } else {
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
          for (int b = 0; b < 4; ++b) acc[t][b] = fmaf(p[t][b], f[t], acc[t][b]);
      }
    }
  };

  // The item's end: this wave's sums to LDS, and one wave adds and finishes.
  auto finish = [&](int q, int nth) {
    lds_char* buf = sums + (nth & 1) * (kWaves * RT * 1024);
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      *reinterpret_cast<lds_f32x4*>(buf + (wave * RT + t) * 1024 + lane * 16) = acc[t];
      acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    // (the loads under way stay under way)
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (wave != (nth & (kWaves - 1))) return;
    f32x4 v[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      v[t] = *reinterpret_cast<const lds_f32x4*>(buf + t * 1024 + lane * 16);
#pragma unroll
      for (int w = 1; w < kWaves; ++w) {
        const f32x4 o = *reinterpret_cast<const lds_f32x4*>(buf + (w * RT + t) * 1024 + lane * 16);
#pragma unroll
        for (int b = 0; b < 4; ++b) v[t][b] += o[b];
      }
    }
    // lane (c, g): token c, weight rows 4 g .. 4 g + 3 of each tile
    typedef X x4 __attribute__((ext_vector_type(4)));
    if constexpr (DOWN) {
      if (c < a.T) {
#pragma unroll
        for (int t = 0; t < RT; ++t)
          *reinterpret_cast<x4*>(static_cast<X*>(a.out) + (int64_t)c * N + q * kCols + t * 16 +
                                 4 * g) =
              x4{Elt<X>::from_f32(v[t][0]), Elt<X>::from_f32(v[t][1]), Elt<X>::from_f32(v[t][2]),
                 Elt<X>::from_f32(v[t][3])};
      }
    } else {
      const int e = r.active[q / tiles], s = c < a.T ? r.slot[e * 16 + c] : 0;
      x4 o;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        // one tile: gate rows 0..7, up rows 8..15, on the lane 32 further
        const float up = RT == 1 ? __shfl_xor(v[0][b], 32, kWave) : v[RT - 1][b];
        o[b] = Elt<X>::from_f32(silu_f32(v[0][b]) * up);
      }
      if (s && (RT == 2 || g < 2))
        *reinterpret_cast<x4*>(static_cast<X*>(a.h) + (int64_t)(c * a.k + s - 1) * N +
                               (q % tiles) * kCols + 4 * g) = o;
    }
  };

  Group ga, gb;
  int q = blockIdx.x, u = u0, nth = 0;
  if (q >= items) return;
  load(ga, q, u);
  for (;;) {
    // (both halves alike: the group that is multiplied, and the next one under way)
    auto half = [&](Group& now, Group& next) -> bool {
      const bool last = u + G >= u1;
      const int nq = last ? q + (int)gridDim.x : q, nu = last ? u0 : u + G;
      if (nq < items) load(next, nq, nu);
      __builtin_amdgcn_sched_barrier(0);
      multiply(now, q, u);
      if (last) finish(q, nth++);
      q = nq;
      u = nu;
      return nq < items;
    };
    if (!half(ga, gb)) break;
    if (!half(gb, ga)) break;
  }
}

}  // namespace

// ---------------------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------------------
template <class T>
static hipError_t run_logits(const FewArgs& a, hipStream_t s) {
  const T* x = (const T*)a.x;
  const T* w = (const T*)a.w_router;
  const int n = (int)a.T, d = (int)a.d, E = (int)a.E;
  const unsigned grid = (unsigned)a.E;
  if (n <= 1)
    few_logits_kernel<T, 1><<<grid, 256, 0, s>>>(x, w, a.bias, a.logits, n, d, E);
  else if (n <= 4)
    few_logits_kernel<T, 4><<<grid, 256, 0, s>>>(x, w, a.bias, a.logits, n, d, E);
  else
    few_logits_kernel<T, 16><<<grid, 256, 0, s>>>(x, w, a.bias, a.logits, n, d, E);
  return hipGetLastError();
}

template <class W, class P, bool DOWN>
static hipError_t run_half(const FewKern& k, hipStream_t s) {
  const int lds = P::kLds + few_routing_bytes(k.T, k.k, k.E);
  hipError_t e = hipFuncSetAttribute((const void*)few_kernel<W, P, DOWN>,
                                     hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return e;
  constexpr int cols = DOWN ? 16 * P::RT : 8 * P::RT;
  const int64_t items = DOWN ? k.d / cols
                             : (int64_t)few_active_max(k.T, k.k, k.E) * (k.F / cols);
  const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>(items, kSplitCUs));
  few_kernel<W, P, DOWN><<<grid, kThreads, lds, s>>>(k);
  return hipGetLastError();
}

template <class W, class P>
static hipError_t run_few(const FewKern& k, hipStream_t s) {
  const hipError_t e = run_half<W, P, false>(k, s);
  return e != hipSuccess || k.T == 0 ? e : run_half<W, P, true>(k, s);
}

template <class W, int G8, int G16>
static hipError_t run_few_tokens(const FewKern& k, hipStream_t s) {
  // more than eight tokens: two weight tiles share the rows they are multiplied with
  if (k.T <= 8) return run_few<W, FewTile<W, 8, 1, G8>>(k, s);
  return run_few<W, FewTile<W, 16, 2, G16>>(k, s);
}

hipError_t launch_few(const FewArgs& a, hipStream_t s) {
  if (a.T > 0) {
    const hipError_t e = a.dtype == 1 ? run_logits<bf16>(a, s) : run_logits<float>(a, s);
    if (e != hipSuccess) return e;
  }
  FewKern k = {};
  k.x = a.x;
  k.logits = a.logits;
  k.sel_bias = a.sel_bias;
  k.gate = {(const char*)a.w[0], (const char*)a.w_scale[0]};
  k.up = {(const char*)a.w[1], (const char*)a.w_scale[1]};
  k.down = {(const char*)a.w[2], (const char*)a.w_scale[2]};
  k.h = a.h;
  k.out = a.out;
  k.routed = a.routed;
  k.kept = a.kept;
  k.drops = a.drops;
  k.status = a.status;
  k.T = (int)a.T;
  k.d = (int)a.d;
  k.E = (int)a.E;
  k.k = (int)a.k;
  k.F = (int)a.F;
  k.C = (int)a.C;
  k.n_groups = a.n_groups;
  k.topk_groups = a.topk_groups;
  k.slot_major = a.slot_major;
  if (a.scale_type == kScaleF32) return run_few_tokens<W8<4>, 4, 3>(k, s);
  if (a.scale_type == kScaleE8M0) return run_few_tokens<W8<1>, 4, 3>(k, s);
  if (a.dtype == 1) return run_few_tokens<W16, 8, 4>(k, s);
  return run_few_tokens<W32, 8, 4>(k, s);
}

}  // namespace moe
