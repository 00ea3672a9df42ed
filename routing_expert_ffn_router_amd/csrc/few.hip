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
// since its cost is less than another launch's.  So there are two launches: the logits, and the
// experts' network, whose gate/up and down parts follow each other by tickets and a counter, without a
// barrier over the grid.
//
// A block is eight waves on one CU that take items in turn.  An item is sixteen weight rows (eight of
// gate with the eight of up of the same columns, or sixteen of down over all chosen experts), or
// eight times that for the block.  Weights and the token rows that they meet are copied straight to
// LDS, whole 128-byte lines, into a ring of stages that runs on across the items' borders; nothing
// of it passes through registers but a fragment before its matrix instruction.  Up to eight tokens,
// the waves divide the reduction, each with a ring of its own and no barrier before the item's end, where
// their sums meet in LDS and one wave, a different one each time, adds them in wave order and finishes
// the item while the others go on.  With more tokens their rows would be half of all that is copied:
// there the waves divide the columns and share the rows, with a barrier for each stage.
//
// Sums are fp32; h is rounded to x's type (the down product takes 16-bit operands, as in the layer for
// many tokens), the output once more; the selection is by logits summed in 64 bits.
//
// A block that waits in vain (two calls in one workspace) makes its gates NaN and goes on, so that the
// kernel ends and what it could not compute shows.
//
// Measured on one card (the number of experts read, TB/s of their weights, and the layer for many
// tokens): bf16, two of eight experts of 4096 / 14336, one token 118 us (2, 6.0 TB/s; 195), four 318 (6,
// 6.6; 350), eight 374 (7, 6.6; 399), nine 416 (7; 399) and sixteen 475 (8; 464: that layer's
// 64-row tiles read few, large experts slightly better); eight of 256 of 7168 / 2048, one token
// 122 (8, 5.8; 177), sixteen 1391 (106, 6.7; 1832); eight of 128 of 2048 / 768, one token 33 (8, 2.3; 59),
// of which the logits take 5 and the routing 4 (sixteen tokens and 256 experts: 7 and 11).
// e4m3 with E8M0 scales, eight of 256 of 7168 / 2048: one token 86 (8, 4.1; 118), three 191 (22; 210), four
// 267 (30; 247), sixteen 842 (105; 739: the rows, in 16 bits, are two lines of LDS for each line of
// weights, and an LDS instruction meets 1.9 cycles of bank conflicts).
#include <algorithm>
#include <atomic>

#include "few_walk.h"
#include "fp8_common.h"
#include "gemm_common.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kThreads = kWaves * kWave, kTokens = 16;

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
  float* partial;     // [chunks][T, d]
  int32_t* counters;  // tickets and what is done, zero
  int32_t* tile_done; // [column tiles], zero
  int T, d, E, k, F, C, n_groups, topk_groups, slot_major, chunks, tickets, tp, lds, polls;
};

// ---------------------------------------------------------------------------------------
// router logits
// ---------------------------------------------------------------------------------------
// One block for each expert and four tokens.  A product of two bf16 (fp32) values is exact in 64 bits and
// the sums lose 2^-53 of their largest term or so: the selection is that of the exact logits rounded
// to fp32.  3 to 7 us.
template <class T, int TT>
__global__ void __launch_bounds__(256)
few_logits_kernel(const T* __restrict__ x, const T* __restrict__ w, const float* __restrict__ b,
                  float* __restrict__ logits, int tokens, int d, int E, int32_t* __restrict__ zero,
                  int zeros, int32_t* __restrict__ status) {
  if (blockIdx.x == 0 && blockIdx.y == 0) {  // the experts' counters
    for (int i = threadIdx.x; i < zeros; i += 256) zero[i] = 0;
    if (status && threadIdx.x == 0) *status = 0;
  }
  x += (int64_t)blockIdx.y * TT * d;
  logits += (int64_t)blockIdx.y * TT * E;
  tokens -= blockIdx.y * TT;
  constexpr int V = 16 / sizeof(T);
  typedef T tx __attribute__((ext_vector_type(V)));
  __shared__ double part[4][TT];
  const int e = blockIdx.x, tid = threadIdx.x;
  double sum[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) sum[t] = 0.0;
  constexpr int U = TT == 1 ? 4 : 2;  // pieces under way
  for (int i0 = tid * V; i0 < d; i0 += U * 256 * V) {
    tx wv[U], xv[U][TT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * 256 * V;
      if (i < d) {
        wv[u] = *reinterpret_cast<const tx*>(w + (int64_t)e * d + i);
#pragma unroll
        for (int t = 0; t < TT; ++t)
          if (t < tokens) xv[u][t] = *reinterpret_cast<const tx*>(x + (int64_t)t * d + i);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u * 256 * V >= d) break;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const double wd = (double)Elt<T>::to_f32(wv[u][j]);
#pragma unroll
        for (int t = 0; t < TT; ++t)
          if (t < tokens) sum[t] = fma(wd, (double)Elt<T>::to_f32(xv[u][t][j]), sum[t]);
      }
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
  uint16_t* active;  // experts with tokens, in order
  int count;
};

__host__ __device__ inline int few_active_max(int T, int k, int E) { return min(E, T * k); }
// slot, gate_of, active and the selected experts
__host__ __device__ inline int few_routing_bytes(int T, int k, int E) {
  const int bytes = E * 16 + T * k * 4 + few_active_max(T, k, E) * 2 + T * k * 2;
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
// V: logits a lane holds.
template <int V>
__device__ inline bool few_select(const float* __restrict__ row, const float* __restrict__ sel_bias,
                                  int E, int k, int n_groups, int topk_groups, uint32_t* group_key,
                                  int* slot_e) {
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
#pragma unroll 1
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
#pragma unroll 1
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
  __shared__ uint64_t masks[1024 / kWave];
  __shared__ int tally[66 + 2];  // drops, then status, then tokens that took expert 0 more than once
  const int tid = threadIdx.x, lane = lane_id(), wave = tid / kWave;
  const int T = a.T, E = a.E, k = a.k, pairs = T * k, most = few_active_max(T, k, E);
  Routing r;
  r.slot = reinterpret_cast<uint8_t*>(smem);
  r.gate_of = reinterpret_cast<float*>(smem + E * 16);
  r.active = reinterpret_cast<uint16_t*>(r.gate_of + pairs);
  uint16_t* sel = r.active + most;
  u32x4* slot4 = reinterpret_cast<u32x4*>(smem);
  for (int e = tid; e < E; e += kThreads) slot4[e] = u32x4{0, 0, 0, 0};
  if (tid < 68) tally[tid] = 0;
  __syncthreads();
#pragma unroll 1
  for (int t = wave; t < T; t += kWaves) {
    int e;
    const float* row = a.logits + (int64_t)t * E;
    const bool bad =
        E <= 256 ? few_select<4>(row, a.sel_bias, E, k, a.n_groups, a.topk_groups,
                                 group_key[wave], &e)
                 : few_select<16>(row, a.sel_bias, E, k, a.n_groups, a.topk_groups,
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
    // slots without a finite logit take expert 0: the first of its slots stands in the table
    const uint64_t zero = __ballot(lane < k && e == 0);
    if (lane < k) {
      sel[t * k + lane] = (uint16_t)e;
      r.gate_of[t * k + lane] = ex / sum;
      if (e != 0 || lane == __builtin_ctzll(zero)) r.slot[e * 16 + t] = (uint8_t)(lane + 1);
    }
    if (bad && lane == 0) atomicAdd(&tally[66], 1);
    if ((zero & (zero - 1)) != 0 && lane == 0) atomicAdd(&tally[67], 1);
  }
  __syncthreads();
  const bool again = tally[67] != 0;
  auto count_to = [&](int32_t* counts) {  // each expert's slots, without those that were dropped
    for (int e = tid; e < E; e += kThreads) {
      int n = 0;
      if (again && e == 0) {
#pragma unroll 1
        for (int i = 0; i < pairs; ++i) n += sel[i] == 0;
      } else {
#pragma unroll 1
        for (int t = 0; t < T; ++t) n += r.slot[e * 16 + t] != 0;
      }
      counts[e] = n;
    }
  };
  if (report && a.routed) count_to(a.routed);
  // some may be dropped (of expert 0's that stand in, beyond T, without a limit too): count the earlier
  // assignments to the same expert
  if (a.C < T || again) {
    int drop = 0;  // this thread's pairs (at most 512 of them in all)
    const int t = tid / k, j = tid - t * k;
    if (tid < pairs) {
      int before = 0;
      const int e = sel[tid];
      if (again && e == 0) {
#pragma unroll 1
        for (int o = 0; o < T; ++o)
#pragma unroll 1
          for (int i = 0; i < k; ++i)
            if (sel[o * k + i] == 0 &&
                (a.slot_major ? i < j || (i == j && o < t) : o < t || (o == t && i < j)))
              ++before;
      } else {
#pragma unroll 1
        for (int o = 0; o < T; ++o) {
          const int s = r.slot[e * 16 + o];
          if (s && (a.slot_major ? s - 1 < j || (s - 1 == j && o < t) : o < t)) ++before;
        }
      }
      drop = before >= a.C;
    }
    __syncthreads();
    if (drop) {
      // (of several slots the first is dropped last, in either order)
      if (r.slot[sel[tid] * 16 + t] == j + 1) r.slot[sel[tid] * 16 + t] = 0;
      atomicAdd(&tally[0], 1);
      atomicAdd(&tally[1 + j], 1);
      sel[tid] = 0xffff;
    }
    __syncthreads();
    if (report && tid < T) {
      bool none = true;
#pragma unroll 1
      for (int i = 0; i < k; ++i) none = none && sel[tid * k + i] == 0xffff;
      if (none) atomicAdd(&tally[k + 1], 1);
    }
    __syncthreads();
  }
  if (report) {
    if (a.kept) count_to(a.kept);
    if (a.drops && tid < k + 2) a.drops[tid] = tally[tid];
    // (a block that gave up waiting may have marked it already)
    if (a.status && tid == 0 && tally[66]) atomicOr(a.status, tally[66]);
  }
  if (again && tid < T && r.slot[tid] != 0) {  // expert 0's slots of a token count with the first
    float* gates = r.gate_of + tid * k;
    float sum = 0.f;
#pragma unroll 1
    for (int i = 0; i < k; ++i)
      if (sel[tid * k + i] == 0) sum += gates[i];
    gates[r.slot[tid] - 1] = sum;
  }
  // experts with tokens, in order: a mask of each 64 experts
  constexpr int kMasks = 1024 / kWave;
#pragma unroll
  for (int m = wave; m < kMasks; m += kWaves) {
    const int e = m * kWave + lane;
    bool any = false;
    if (e < E) {
      const u32x4 v = slot4[e];
      any = (v[0] | v[1] | v[2] | v[3]) != 0;
    }
    const uint64_t mask = __ballot(any);
    if (lane == 0) masks[m] = mask;
  }
  __syncthreads();
  int count = 0;
#pragma unroll 1
  for (int m = 0; m * kWave < E; ++m) {
    const uint64_t mask = masks[m];
    if (m % kWaves == wave && ((mask >> lane) & 1))
      r.active[count + __builtin_popcountll(mask & ((1ull << lane) - 1))] =
          (uint16_t)(m * kWave + lane);
    count += __builtin_popcountll(mask);
  }
  __syncthreads();
  r.count = __builtin_amdgcn_readfirstlane(count);
  return r;
}

// ---------------------------------------------------------------------------------------
// the experts
// ---------------------------------------------------------------------------------------
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

// Waits until `count` tickets are done; false: it looked `polls` times in vain, something must be
// wrong with the workspace (another call's, say), and the kernel ends all the same.
__device__ inline bool wait_for(const int32_t* done, int count, int polls) {
#pragma unroll 1
  for (int i = 0; i < polls; ++i) {
    if (__hip_atomic_load(done, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) >= count) return true;
    __builtin_amdgcn_s_sleep(2);
  }
  return false;
}

// What one block writes for another (h, sums of chunks) goes through all caches to where every XCD sees
// it, and is read from there; a wave waits for its own stores before the counter that tells of them is
// raised.  (A release and an acquire instead write back and drop an XCD's whole L2, 3 us of every
// block one after the other, and with it the weights that were fetched ahead.)
template <class V>
__device__ inline void store_shared(V* p, const V& v) {
  static_assert(sizeof(V) == 8 || sizeof(V) == 16, "whole words of 64 bits");
  typedef uint64_t words __attribute__((ext_vector_type(2)));
  if constexpr (sizeof(V) == 8) {
    __hip_atomic_store(reinterpret_cast<uint64_t*>(p), __builtin_bit_cast(uint64_t, v),
                       __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  } else {
    const words w = __builtin_bit_cast(words, v);
    for (int i = 0; i < 2; ++i)
      __hip_atomic_store(reinterpret_cast<uint64_t*>(p) + i, w[i], __ATOMIC_RELAXED,
                         __HIP_MEMORY_SCOPE_AGENT);
  }
}
__device__ inline f32x4 load_shared(const f32x4* p) {
  typedef uint64_t words __attribute__((ext_vector_type(2)));
  words w;
  for (int i = 0; i < 2; ++i)
    w[i] = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p) + i, __ATOMIC_RELAXED,
                             __HIP_MEMORY_SCOPE_AGENT);
  return __builtin_bit_cast(f32x4, w);
}
__device__ inline void wait_stores() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
constexpr int kSharedLoad = 16;  // a buffer load's flag for it

// LDS accesses that the compiler does not order behind the direct loads under way: it would wait for
// all of those before each.  Each waits for itself.
__device__ inline uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}
__device__ inline uint32_t lds_u8(uint32_t at) {
  uint32_t v;
  asm volatile("ds_read_u8 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=&v"(v) : "v"(at) : "memory");
  return v;
}
__device__ inline uint32_t lds_u16(uint32_t at) {
  uint32_t v;
  asm volatile("ds_read_u16 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=&v"(v) : "v"(at) : "memory");
  return v;
}
__device__ inline uint32_t lds_u32(uint32_t at) {
  uint32_t v;
  asm volatile("ds_read_b32 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=&v"(v) : "v"(at) : "memory");
  return v;
}
__device__ inline float lds_f32(uint32_t at) { return __uint_as_float(lds_u32(at)); }
__device__ inline void lds_set(uint32_t at, uint32_t v) {
  asm volatile("ds_write_b32 %0, %1\n\ts_waitcnt lgkmcnt(0)" ::"v"(at), "v"(v) : "memory");
}
__device__ inline void lds_write(uint32_t at, const f32x4& v) {
  asm volatile("ds_write_b128 %0, %1" ::"v"(at), "v"(v) : "memory");
}
// N pieces
template <int N>
__device__ inline void lds_read(u32x4 (&v)[N], const uint32_t (&at)[N]) {
  static_assert(N == 4 || N == 6, "pieces");
  if constexpr (N == 4)
    asm volatile(
        "ds_read_b128 %0, %4\n\tds_read_b128 %1, %5\n\tds_read_b128 %2, %6\n\t"
        "ds_read_b128 %3, %7\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3])
        : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3])
        : "memory");
  if constexpr (N == 6)
    asm volatile(
        "ds_read_b128 %0, %6\n\tds_read_b128 %1, %7\n\tds_read_b128 %2, %8\n\t"
        "ds_read_b128 %3, %9\n\tds_read_b128 %4, %10\n\tds_read_b128 %5, %11\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5])
        : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "v"(at[4]), "v"(at[5])
        : "memory");
}
template <int N>
__device__ inline void wait_loads() {
  static_assert(N >= 0 && N < 64, "vmcnt immediate");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// How a block divides an item.  ALONG the reduction: every wave takes its part of the units of 16
// weight rows, with a ring of its own for weights and rows; ACROSS the columns (more than eight
// tokens, whose rows would be half of all loads): every wave takes 16 weight rows of its own through
// all units, and the block shares the rows.
constexpr bool kAlong = false, kAcross = true;

// A unit is U * 128 bytes of each of 16 weight rows.  LDS of one stage of the ring, of one wave (along)
// or of the block (across): weight rows of one unit, tp = T tokens' rows, scales (a word for each 128
// bytes of gate or down, and of up).
template <class W, int U, bool ACROSS>
__host__ __device__ constexpr int stage_bytes(int tp) {
  return (ACROSS ? kWaves : 1) * (U * 2048 + (W::kScale ? 16 : 0)) + U * tp * W::kXBytes;
}
template <class W, int U, bool ACROSS>
__host__ __device__ constexpr int ring_bytes(int tp, int stages) {
  return (ACROSS ? 1 : kWaves) * stages * stage_bytes<W, U, ACROSS>(tp);
}
constexpr int kSumBytes = 2 * kWaves * 1024;  // along: two items' sums
// columns of an item: gate and up rows of the same columns make up the sixteen
__host__ __device__ constexpr int few_columns(bool down, bool across) {
  return (down ? 16 : 8) * (across ? kWaves : 1);
}

// Items first, first + stride, ... of gate/up or of down.  ready(): called once, when the first
// weights are under way and before h and the gates are read.
template <class W, int U, int S, bool ACROSS, bool DOWN, class Ready>
__device__ __attribute__((always_inline)) inline void few_items(const FewKern& a, const Routing& r,
                                                                char* smem, int items, int first,
                                                                int stride, Ready&& ready) {
  typedef typename W::X X;
  typedef X x4 __attribute__((ext_vector_type(4)));
  constexpr int ES = W::kScale, NX = W::kXBytes / 128;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int c = lane & 15, g = lane >> 4;
  const uint32_t slot_tab = lds_address(r.slot), gate_tab = lds_address(r.gate_of),
                 active_tab = lds_address(r.active);

  const int K = DOWN ? a.F : a.d, N = DOWN ? a.d : a.F, tp = a.tp, chunks = DOWN ? a.chunks : 1;
  constexpr int kCols = few_columns(DOWN, ACROSS);
  const int per_k = (int)((uint32_t)K * W::kElt / (128u * U)), tiles = (int)((uint32_t)N / kCols);
  const int units = DOWN ? r.count * per_k : per_k;
  const uint32_t pitch = (uint32_t)K * W::kElt, x_pitch = (uint32_t)K * (uint32_t)sizeof(X);
  const int64_t matrix = (int64_t)N * pitch;
  constexpr uint32_t kNone = 0x80000000u;  // past a resource's end: loads as zeros

  // A stage: this wave's weight rows, then (along: its, across: the block's) tokens' rows and scales.
  // A weight load brings eight rows of 128 bytes; the 16-byte piece p of row n lies in slot
  // p ^ ((n >> 1) & 7), which keeps a fragment's reads free of bank conflicts.
  const int stage = stage_bytes<W, U, ACROSS>(tp);
  lds_char* const ring = (lds_char*)smem + (ACROSS ? 0 : wave * S * stage);
  const int w_at = ACROSS ? wave * (U * 2048) : 0, x_at = (ACROSS ? kWaves : 1) * (U * 2048);
  const int s_at = x_at + U * tp * W::kXBytes + (ACROSS ? wave * 16 : 0);
  const uint32_t ring_lds = lds_address(smem) + (ACROSS ? 0 : wave * S * stage);
  uint32_t vw[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    vw[i] = (uint32_t)(lane >> 3) * pitch + (uint32_t)(((lane & 7) ^ (4 * i + (lane >> 4))) * 16);
  // the tokens' rows in parts of 128 bytes, a load each: along, the wave's own; across, an eighth
  const int x_lanes = ACROSS ? tp : tp * 8, x_piece = (ACROSS ? wave * tp : 0) + lane;
  const int x_row = x_piece >> 3;
  const uint32_t x_col = (uint32_t)(((x_piece & 7) ^ ((x_row >> 1) & 7)) * 16);
  const int x_dst = x_at + (ACROSS ? wave * tp * 16 : 0);
  // fragments: weights' row c, pieces g and g + 4; the same values of token c's row
  constexpr int kFrags = 2 + 2 * NX;
  uint32_t frag[kFrags];
  {
    auto piece = [&](int row, int p) { return (uint32_t)(row * 128 + ((p ^ ((row >> 1) & 7)) << 4)); };
    const int xr = min(c, tp - 1);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      frag[ks] = ring_lds + w_at + piece(c, ks * 4 + g);
      if constexpr (NX == 1)
        frag[2 + ks] = ring_lds + x_at + piece(xr, ks * 4 + g);
      else
#pragma unroll
        for (int h = 0; h < 2; ++h)
          frag[2 + 2 * ks + h] = ring_lds + x_at + ks * tp * 128 + piece(xr, 2 * g + h);
    }
  }

  typedef FewWalk<ACROSS, DOWN> Walk;
  typedef typename Walk::Place Place;
  constexpr int kStep = Walk::kStep;
  const Walk walk = {items, stride, tiles, per_k, units, chunks, wave};

  // Loading.  Past the last item the loads go nowhere and give zeros, so that every step issues as
  // many loads and the waits count a constant.
  const Place start = walk.start(first);
  Place l = start;
  int l_todo = 0, l_slot = 0;  // units of the run to go; the stage
  uint32_t l_off = 0;          // 128 bytes for each 128 of the rows
  auto rsrc = [](uint64_t base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(base), 0, (int)bytes, 0x00020000);
  };
  const uint64_t x_base = uniform_u64(DOWN ? a.h : a.x);
  // (below 2^31)
  const uint32_t x_bytes = (uint32_t)(DOWN ? a.T * a.k : a.T) * x_pitch;
  const auto rx = rsrc(x_base, x_bytes);
  auto r0 = rx, r1 = rx;
  const char *scale0 = nullptr, *scale1 = nullptr;
  uint32_t v0 = kNone, v1 = kNone, vx = kNone;
  auto find = [&]() __attribute__((always_inline)) {
    const bool live = walk.next_run(l, [](int) {});
    l_todo = live ? l.run : 0x7fffffff;
    l_off = live ? (uint32_t)l.k * (U * 128u) : 0u;
    // (not live: offsets past the resources' ends)
    const int e =
        __builtin_amdgcn_readfirstlane((int)lds_u16(active_tab + walk.entry(l, live) * 2));
    const int col0 =
        __builtin_amdgcn_readfirstlane((int)((uint32_t)l.q % (uint32_t)tiles)) * kCols;
    const int64_t to = (int64_t)e * matrix +
                       (int64_t)(col0 + (ACROSS ? wave * few_columns(DOWN, false) : 0)) * pitch;
    // sixteen rows of down, or eight of gate and eight of up
    const uint64_t base0 = uniform_u64((DOWN ? a.down.q : a.gate.q) + to);
    r0 = rsrc(base0, 0x7fffffff);
    r1 = rsrc(DOWN ? base0 + 8u * pitch : uniform_u64(a.up.q + to), 0x7fffffff);
    v0 = live ? vw[0] : kNone;
    v1 = live ? vw[1] : kNone;
    if constexpr (ES > 0) {
      const int64_t at = live ? ((int64_t)e * (N / 128) + col0 / 128) * (K / 128) * ES : 0;
      scale0 = (DOWN ? a.down.scale : a.gate.scale) + at;
      scale1 = (DOWN ? a.down.scale : a.up.scale) + at;
    }
    if constexpr (DOWN) {
      const int s = (int)lds_u8(slot_tab + e * 16 + min(x_row, kTokens - 1));
      vx = s && live ? (uint32_t)(x_row * a.k + s - 1) * x_pitch + x_col : kNone;
    } else {
      vx = x_row < a.T && live ? (uint32_t)x_row * x_pitch + x_col : kNone;
    }
  };
  auto load_w = [&]() __attribute__((always_inline)) {
    const uint32_t off = __builtin_amdgcn_readfirstlane(l_off);
    lds_char* to = ring + l_slot + w_at;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // each line is read once: past the caches
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r0, to + u * 2048, 16, v0, off + u * 128u, 0, 2);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r1, to + u * 2048 + 1024, 16, v1, off + u * 128u, 0, 2);
    }
  };
  // While h is not ready: the lines of the next units into the L2, a lane for each line.
  auto touch = [&]() __attribute__((always_inline)) {
    if constexpr (!DOWN) return;
    constexpr int kAhead = 8 / U;  // units
    const int piece = lane >> 4;
    uint32_t seen[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int unit = n * (kAhead / 2) + piece / U;
      const uint32_t to = (uint32_t)(lane & 15) * pitch + l_off + (uint32_t)(unit * kStep * U * 128) +
                          (uint32_t)(piece % U) * 128u;
      seen[n] = __builtin_amdgcn_raw_buffer_load_b32(r0, v0 != kNone && unit < l_todo ? to : kNone, 0, 0);
    }
    asm volatile("" ::"v"(seen[0]), "v"(seen[1]));
  };
  auto load_x = [&]() __attribute__((always_inline)) {
    const uint32_t off = __builtin_amdgcn_readfirstlane(l_off);
    if (lane < x_lanes) {
#pragma unroll
      for (int n = 0; n < U * NX; ++n)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, ring + l_slot + x_dst + n * tp * 128, 16, vx,
                                                 off * NX + n * 128u, 0,
                                                 DOWN ? kSharedLoad : 0);
    }
    if constexpr (ES > 0) {
      if (lane < 2 * U) {  // gate or down, up; of each 128 bytes
        const char* p = (lane & 1 ? scale1 : scale0) + (off / 128 + (lane >> 1)) * ES;
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) char*)p,
                                         ring + l_slot + s_at, W::kScale == 1 ? 1 : 4, 0, 0);
      }
    }
  };
  constexpr int kXLoads = U * NX + (ES ? 1 : 0), kLoads = 2 * U + kXLoads;

  // The item's end.  Along: this wave's sums to LDS, and one wave, another one each time, adds them and
  // finishes.  lane (c, g): token c, weight rows 4 g .. 4 g + 3.
  f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
  const uint32_t sums = lds_address(smem) + (ACROSS ? 1 : kWaves) * S * stage;
  auto finish = [&](int q, int nth) __attribute__((always_inline)) {
    f32x4 v = acc;
    acc = f32x4{0.f, 0.f, 0.f, 0.f};
    if constexpr (!ACROSS) {
      const uint32_t buf = sums + (nth & 1) * (kWaves * 1024) + lane * 16;
      lds_write(buf + wave * 1024, v);
      // (the loads under way stay under way)
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      if (wave != (nth & (kWaves - 1))) return;
      v = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWaves; w += 4) {
        u32x4 o[4];
        const uint32_t at[4] = {buf + w * 1024, buf + (w + 1) * 1024, buf + (w + 2) * 1024,
                                buf + (w + 3) * 1024};
        lds_read<4>(o, at);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int b = 0; b < 4; ++b) v[b] += __uint_as_float(o[i][b]);
      }
    }
    const int n = (int)((uint32_t)q / (uint32_t)tiles), tile = q - n * tiles;
    if constexpr (DOWN) {
      const int col = tile * kCols + (ACROSS ? wave * 16 : 0) + 4 * g;
      if (chunks > 1) {
        // the chunk's sums to the workspace; the columns' last chunk adds them in order
        f32x4* at = reinterpret_cast<f32x4*>(a.partial + (int64_t)c * N + col);
        const int64_t chunk = (int64_t)a.T * N / 4;
        if (c < a.T) store_shared(at + n * chunk, v);
        wait_stores();
        int before = 0;
        if (lane == 0)
          before = __hip_atomic_fetch_add(a.tile_done + col / 16, 1, __ATOMIC_RELAXED,
                                          __HIP_MEMORY_SCOPE_AGENT);
        if (__builtin_amdgcn_readfirstlane(before) != chunks - 1) return;
        if (c < a.T) {
          v = load_shared(at);
#pragma unroll 4
          for (int i = 1; i < chunks; ++i) {
            const f32x4 o = load_shared(at + i * chunk);
#pragma unroll
            for (int b = 0; b < 4; ++b) v[b] += o[b];
          }
        }
      }
      if (c < a.T)
        *reinterpret_cast<x4*>(static_cast<X*>(a.out) + (int64_t)c * N + col) =
            x4{Elt<X>::from_f32(v[0]), Elt<X>::from_f32(v[1]), Elt<X>::from_f32(v[2]),
               Elt<X>::from_f32(v[3])};
    } else {
      const int e = __builtin_amdgcn_readfirstlane((int)lds_u16(active_tab + n * 2));
      const int s = (int)lds_u8(slot_tab + e * 16 + c);
      x4 o;
#pragma unroll
      for (int b = 0; b < 4; ++b)  // gate rows 0..7, up rows 8..15 on the lane 32 further
        o[b] = Elt<X>::from_f32(silu_f32(v[b]) * __shfl_xor(v[b], 32, kWave));
      if (s && g < 2)
        store_shared(reinterpret_cast<x4*>(static_cast<X*>(a.h) + (int64_t)(c * a.k + s - 1) * N +
                                           tile * kCols + (ACROSS ? wave * 8 : 0) + 4 * g),
                     o);
    }
  };

  // The unit that is multiplied.
  Place m = start;
  int m_todo = 0, nth = 0;
  uint32_t m_slot = 0;
  float gate = 1.f;
  // One loop, so that there is one copy of everything: a block runs much of its code once, and what
  // it has to fetch it waits for.  First the S - 1 first units' weights, then, h being ready, their
  // rows, then a step for each unit.
  enum { kWeights, kRows, kSteps };
  int phase = kWeights, count = S - 1;
  // loads behind stage u's at step u: those of S - 1 (across: S - 2) stages; at first fewer, since
  // the first stages' rows follow all of their weights
  constexpr int kBehind = ACROSS ? S - 2 : S - 1;
#pragma unroll 1
  for (;;) {
    if (phase == kSteps) {
      if (m_todo == 0) {
        if (!walk.next_run(m, [&](int q) {
              if (q >= 0) finish(q, nth++);
            }))
          break;
        m_todo = m.run;
        if constexpr (DOWN) {
          const int e = __builtin_amdgcn_readfirstlane((int)lds_u16(active_tab + m.at * 2));
          const int s = (int)lds_u8(slot_tab + e * 16 + c);
          // a token that did not choose the expert takes nothing of it, be it infinite or NaN
          gate = s ? lds_f32(gate_tab + (s ? c * a.k + s - 1 : 0) * 4) : -1.f;
        }
      }
      --m_todo;
      if constexpr (ACROSS) {
        if (count > 0)
          wait_loads<(S - 2) * kXLoads>();
        else
          wait_loads<kBehind * kLoads>();
        // everyone's part has landed, and everyone is done with the stage that is loaded again
        asm volatile("s_barrier" ::: "memory");
      }
    }
    if (l_todo == 0) find();
    --l_todo;
    if (phase != kRows) load_w();
    if (phase != kWeights) load_x();
    l_slot = l_slot == (S - 1) * stage ? 0 : l_slot + stage;
    l_off += l.left ? kStep * U * 128u : 0u;
    if (phase != kSteps) {
      if (--count == 0) {
        count = S - 1;
        if (phase++ == kWeights) {
          touch();
          l = start;
          l_todo = l_slot = 0;
          ready();
        }
      }
      continue;
    }
    if constexpr (!ACROSS) {
      if (count > 0)
        wait_loads<(S - 2) * kXLoads + kLoads>();
      else
        wait_loads<kBehind * kLoads>();
    }
    if (count > 0) --count;
    unroll_steps<U>([&](auto UI) {
      constexpr int u = decltype(UI)::value;
      u32x4 f[kFrags];
      uint32_t from[kFrags];
#pragma unroll
      for (int i = 0; i < kFrags; ++i)
        from[i] = frag[i] + m_slot + (i < 2 ? u * 2048 : u * NX * tp * 128);
      lds_read<kFrags>(f, from);
      f32x4 v = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        if constexpr (W::kElt == 1) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            mma_chunk(v, e4m3_to_bf16(f[ks][2 * h], f[ks][2 * h + 1]), f[2 + 2 * ks + h], bf16());
        } else {
          mma_chunk(v, f[ks], f[2 + ks], X());
        }
      }
      // the block's scale, then the gate: their product may be below fp32's normal numbers where the
      // scaled sum is not
      float factor = gate;
      if constexpr (ES > 0) {
        float s = lds_f32(ring_lds + m_slot + s_at + u * 8 + (DOWN || g < 2 ? 0 : 4));
        if constexpr (ES == 1) s = e8m0_value(__float_as_uint(s) & 255u);
        if constexpr (DOWN) {
#pragma unroll
          for (int b = 0; b < 4; ++b) v[b] *= s;
        } else {
          factor = s;
        }
      }
#pragma unroll
      for (int b = 0; b < 4; ++b)
        acc[b] = DOWN && gate < 0.f ? acc[b] : fmaf(v[b], factor, acc[b]);
    });
    m_slot = m_slot == (uint32_t)((S - 1) * stage) ? 0 : m_slot + stage;
  }
  // what is under way goes nowhere, but must not be when the LDS is used again
  wait_loads<0>();
  if constexpr (ACROSS) asm volatile("s_barrier" ::: "memory");
}

// The experts' network: gate/up, then down.  Blocks take tickets, each a run of items, and wait for
// h only when no gate/up ticket is left: all of those are then done or held by blocks that run and
// wait for nothing, so every wait ends, however few of the blocks are on the GPU at once.
template <class W, int U, int S, bool ACROSS>
__global__ void __launch_bounds__(kThreads) few_kernel(const FewKern a) {
  extern __shared__ __attribute__((aligned(1024))) char smem_dyn[];
  __shared__ int ticket;
  const int tid = threadIdx.x;
  int32_t* const take_up = a.counters;
  int32_t* const done_up = a.counters + 32;
  int32_t* const take_down = a.counters + 64;
  auto take = [&](int32_t* p) {
    return __hip_atomic_fetch_add(p, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  };
  int mine = 0, mine_down = 0;
  bool gave_up = false;  // thread 0's
  if (tid == 0) {
    mine = take(take_up);
    mine_down = take(take_down);
  }
  const Routing r = few_routing(a, smem_dyn + a.lds, blockIdx.x == 0);
  const int up_items = r.count * (a.F / few_columns(false, ACROSS));
  const int down_items = r.count > 0 ? a.d / few_columns(true, ACROSS) * a.chunks : 0;
  const int up_tickets = min(up_items, a.tickets), down_tickets = min(down_items, a.tickets);
  auto share = [&](int t) {  // thread 0's ticket, to all threads
    __syncthreads();
    if (tid == 0) ticket = t;
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(ticket);
  };
  for (int t = share(mine); t < up_tickets; t = share(mine)) {
    few_items<W, U, S, ACROSS, false>(a, r, smem_dyn, up_items, t, up_tickets, [] {});
    if (tid == 0) mine = take(take_up);
    wait_stores();
    __syncthreads();  // every wave's part of h has arrived
    if (tid == 0)
      __hip_atomic_fetch_add(done_up, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  for (int t = share(mine_down); t < down_tickets; t = share(mine_down)) {
    few_items<W, U, S, ACROSS, true>(a, r, smem_dyn, down_items, t, down_tickets, [&] {
      if (tid == 0 && !gave_up && !wait_for(done_up, up_tickets, a.polls)) {
        // without h: NaN for every gate makes NaN of every sum that h goes into
        gave_up = true;
        for (int i = 0; i < a.T * a.k; ++i) lds_set(lds_address(r.gate_of + i), 0x7fc00000u);
        if (a.status) atomicOr(a.status, (int)0x80000000u);
      }
      asm volatile("s_barrier" ::: "memory");
    });
    if (tid == 0) mine_down = take(take_down);
  }
}

}  // namespace

// ---------------------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------------------
template <class T, int TT>
static hipError_t run_logits(const FewArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)a.E, (unsigned)std::max<int64_t>(1, (a.T + TT - 1) / TT));
  few_logits_kernel<T, TT><<<grid, 256, 0, s>>>(
      (const T*)a.x, (const T*)a.w_router, a.bias, a.logits, (int)a.T, (int)a.d, (int)a.E,
      a.counters, kFewCounters + (int)(a.d / 16), a.status);
  return hipGetLastError();
}

template <class W, int U, int S, bool ACROSS>
static hipError_t run_few(FewKern k, hipStream_t s) {
  k.lds = ring_bytes<W, U, ACROSS>(k.tp, S) + (ACROSS ? 0 : kSumBytes);
  const int lds = k.lds + few_routing_bytes(k.T, k.k, k.E);
  hipError_t e = hipFuncSetAttribute((const void*)few_kernel<W, U, S, ACROSS>,
                                     hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return e;
  // Down's column tiles are cut along the reduction where they are too few for the CUs, or leave
  // many idle in a last round; each wave keeps two units at least.
  const int tiles = k.d / few_columns(true, ACROSS);
  const int most = std::min<int>(
      kFewChunks, std::max(1, k.k * (k.F * W::kElt / 128) / (2 * (ACROSS ? 4 : kWaves))));
  auto busy = [&](int n) {
    const int rounds = (tiles * n + kSplitCUs - 1) / kSplitCUs;
    return (double)(tiles * n) / (rounds * kSplitCUs);
  };
  k.chunks = 1;
  for (int n = 2; n <= most && busy(k.chunks) < 0.85; ++n)
    if (busy(n) > busy(k.chunks)) k.chunks = n;
  const int64_t up =
      (int64_t)few_active_max(k.T, k.k, k.E) * (k.F / few_columns(false, ACROSS));
  const int64_t items = std::max<int64_t>(up, (int64_t)tiles * k.chunks);
  k.tickets = kSplitCUs;
  const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>(items, kSplitCUs));
  few_kernel<W, U, S, ACROSS><<<k.T ? grid : 1, kThreads, lds, s>>>(k);
  return hipGetLastError();
}

// Whether a ring fits a CU's LDS, beside what the kernel holds in static tables.
template <class W, int U, bool ACROSS>
static bool ring_fits(const FewKern& k, int stages) {
  return ring_bytes<W, U, ACROSS>(k.tp, stages) + (ACROSS ? 0 : kSumBytes) +
             few_routing_bytes(k.T, k.k, k.E) <= 160 * 1024 - 4096;
}

// The deepest ring that fits.  Up to eight tokens the waves divide the reduction, with more, a wave's
// own copy of the rows would take as much of the LDS as its weights (us along and across, bf16: two of
// eight of 4096 / 14336, one token 118 and 137, four 319 and 361, eight 374 and 417; eight of 128 of
// 2048 / 768, one 34 and 45, eight 101 and 120; eight of 256 of 7168 / 2048, eight 797 and 787).  Two
// pieces of 128 bytes a step against one: one token, eight of 256 of 7168 / 2048 121 and 123 us, eight of
// 128 of 2048 / 768 33.7 and 33.8, six of 64 of 2048 / 1408 37.2 and 36.6; sixteen, two of eight of
// 4096 / 14336 422 and 426.
template <class W>
static hipError_t run_few_tokens(FewKern k, hipStream_t s) {
  k.tp = std::max(k.T, 1);
  const bool pairs = (int64_t)k.d * W::kElt % 256 == 0 && (int64_t)k.F * W::kElt % 256 == 0;
  if (k.T > 8) {
    if (pairs && ring_fits<W, 2, kAcross>(k, 4)) return run_few<W, 2, 4, kAcross>(k, s);
    return run_few<W, 1, 6, kAcross>(k, s);
  }
  if (pairs && ring_fits<W, 2, kAlong>(k, 3)) return run_few<W, 2, 3, kAlong>(k, s);
  // (five stages fit beside any tables, but for 8-bit weights, whose rows take two lines a unit)
  if constexpr (W::kScale > 0) {
    if (!ring_fits<W, 1, kAlong>(k, 5))
      return ring_fits<W, 1, kAlong>(k, 4) ? run_few<W, 1, 4, kAlong>(k, s)
                                           : run_few<W, 1, 3, kAlong>(k, s);
  }
  return run_few<W, 1, 5, kAlong>(k, s);
}

// (2^20 looks of about a microsecond: a second)
static std::atomic<int32_t> wait_polls{1 << 20};

int32_t few_wait_polls(int32_t polls) {
  return polls < 0 ? wait_polls.load() : wait_polls.exchange(polls);
}

hipError_t launch_few(const FewArgs& a, hipStream_t s) {
  const bool one = a.T <= 1;
  const hipError_t e = a.dtype == 1 ? one ? run_logits<bf16, 1>(a, s) : run_logits<bf16, 4>(a, s)
                       : one        ? run_logits<float, 1>(a, s)
                                    : run_logits<float, 4>(a, s);
  if (e != hipSuccess) return e;
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
  k.partial = a.partial;
  k.counters = a.counters;
  k.polls = wait_polls.load();
  k.tile_done = a.counters + kFewCounters;
  if (a.scale_type == kScaleF32) return run_few_tokens<W8<4>>(k, s);
  if (a.scale_type == kScaleE8M0) return run_few_tokens<W8<1>>(k, s);
  if (a.dtype == 1) return run_few_tokens<W16>(k, s);
  return run_few_tokens<W32>(k, s);
}

}  // namespace moe
