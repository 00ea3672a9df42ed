// The experts' linear layers: y[r] = act(z[r]) + residual[r], z[r] = x[r] W[e]^T + bias[e] for the
// rows r of expert e, bf16 and fp32, with everything behind the product in its epilogue.
//
// Both operands are rows contiguous along the reduction, which go through LDS in stages of 128 bytes
// of each row (64 bf16 values, 32 fp32), BM activation rows and BN weight rows (256, or 32 and 64 where
// tiles are few), by direct buffer -> LDS loads; the 16-byte piece c of row r lies in slot c ^ ((r >> 1) & 7), which keeps a fragment's
// reads free of bank conflicts.  A stage's weight fragments are read into registers first and their
// LDS is released and loaded again, two steps ahead, while the activations' stream through
// registers.  Sums are fp32 (fp32 operands: fp32 MFMA).  A block fills its CU's LDS and works through
// its share of the tiles; rows past an expert's last load as zeros from nowhere.
//   Epilogue: the sums go through LDS as fp32, so that bias, activation and residual are applied to
// unrounded values and y and z are each rounded once, with 16-byte accesses to whole lines.
//   Few, long tiles: the last partial round's tiles are cut along the reduction, as in the other
// grouped products; the launch that adds their sums applies the epilogue.
//   Large bf16 products are bound by the matrix cores: 8192 rows, 4096 -> 14336, 709 us alone (1357
// TFLOP/s; the library's product 702) and 785 with bias, gelu and z kept, whose stores and slopes the
// next tile's loads do not cover.  Few rows are bound by latency: 33, 2048 -> 7168, 10 us for 29 MB of
// weights, 2.9 TB/s, since each block goes through 32 dependent steps of two barriers, and only half of
// its waves issue loads.
#include <algorithm>

#include "act.h"
#include "gemm_common.h"
#include "kernels.h"

namespace moe {

typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) f32x4 lds_f32x4;

template <class T>
struct LinearOut {
  const float* bias;  // nullable, [E, N]
  const T* residual;  // nullable, [R, N]; may be y
  T* z;               // nullable, [R, N]
  T* y;
  int act;
};

// f(tag of the activation); the same for all lanes, so that one of the copies runs.
template <class F>
__device__ __attribute__((always_inline)) inline void by_act(int act, F&& f) {
  switch (act) {
    case kActRelu: return f(IntC<kActRelu>{});
    case kActSilu: return f(IntC<kActSilu>{});
    case kActGelu: return f(IntC<kActGelu>{});
    case kActGeluTanh: return f(IntC<kActGeluTanh>{});
    default: return f(IntC<kActNone>{});
  }
}

// C consecutive outputs (4 or 8) of row `row` from column `col` on, from their sums.
template <int ACT, class T, int C>
__device__ inline void finish(const LinearOut<T>& o, const float* bias_row, int64_t row, int N,
                              int col, const float (&sum)[C]) {
  typedef T tx __attribute__((ext_vector_type(C)));
  typedef tx txa __attribute__((aligned(sizeof(T) * 4)));
  const int64_t at = row * N + col;
  float v[C];
#pragma unroll
  for (int i = 0; i < C; ++i) v[i] = sum[i];
  if (bias_row) {
#pragma unroll
    for (int i = 0; i < C; i += 4) {
      const f32x4 b = *reinterpret_cast<const f32x4*>(bias_row + col + i);
#pragma unroll
      for (int q = 0; q < 4; ++q) v[i + q] += b[q];
    }
  }
  tx t;
  if (o.z) {
#pragma unroll
    for (int i = 0; i < C; ++i) t[i] = Elt<T>::from_f32(v[i]);
    __builtin_nontemporal_store(t, reinterpret_cast<txa*>(o.z + at));
  }
#pragma unroll
  for (int i = 0; i < C; ++i) v[i] = act_value<ACT>(v[i]);
  if (o.residual) {
    const tx r = *reinterpret_cast<const txa*>(o.residual + at);
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] += Elt<T>::to_f32(r[i]);
  }
#pragma unroll
  for (int i = 0; i < C; ++i) t[i] = Elt<T>::from_f32(v[i]);
  *reinterpret_cast<txa*>(o.y + at) = t;
}

// BM rows x BN weight rows, 8 waves as WM x WN, each MT x NT MFMA tiles of 16 x 16.
template <int BM_, int BN_, int WM_, int WN_, int STAGES_>
struct LinearTile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
  static constexpr int MT = BM / WM / 16, NT = BN / WN / 16;
  static constexpr int kStages = STAGES_;
  static constexpr int kABytes = BM * 128, kBBytes = BN * 128;
  static constexpr int kLds = kStages * (kABytes + kBBytes);
  // direct loads of 1024 bytes (eight rows) per stage and issuing wave (waves 4-7)
  static constexpr int kALoads = BM / 32, kBLoads = BN / 32;
  // pieces of the reduction have their sums laid out for this one
  static constexpr bool kSplits = BN == 256 && WM == 2 && WN == 4;
  static_assert(WM * WN == 8 && MT >= 1 && NT >= 1 && BM % 32 == 0 && BN % 32 == 0, "tile");
  static_assert(kStages >= 2 && kStages <= 6 && kLds <= 160 * 1024, "LDS of one CU");
};

// One tile: `rows` rows of x from A on, `cols` weight rows from B on, the reduction's bytes [0,
// 128 steps) of them, row pitch `pitch` bytes.  slot (nullable): the sums are one piece of the
// reduction and go there.
template <class T, class G>
__device__ __attribute__((always_inline)) inline void linear_body(
    const T* __restrict__ A, int rows, const T* __restrict__ B, int cols, int64_t pitch, int steps,
    const LinearOut<T>& out, const float* bias_row, int64_t row0, int col0, int N,
    f32x4* __restrict__ slot, lds_char* __restrict__ a0, lds_char* __restrict__ a1,
    lds_char* __restrict__ a2, lds_char* __restrict__ a3, lds_char* __restrict__ a4,
    lds_char* __restrict__ a5, lds_char* __restrict__ b0, lds_char* __restrict__ b1,
    lds_char* __restrict__ b2, lds_char* __restrict__ b3, lds_char* __restrict__ b4,
    lds_char* __restrict__ b5) {
  constexpr int MT = G::MT, NT = G::NT, S = G::kStages, nA = G::kALoads, nB = G::kBLoads;
  const int tid = tile_thread(), lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int wm = wave / G::WN, wn = wave % G::WN;
  const int c = lane & 15, g = lane >> 4;
  const bool issuer = wave >= 4;
  const int dslot = wave & 3;

  // Load i of issuing wave d brings rows 32 i + 8 d + L / 8, lane L their piece (L % 8) ^ swizzle:
  // 32 rows on the swizzle is the same, so one lane offset and a scalar for each i.
  const int r0 = dslot * 8 + lane / 8;
  const uint32_t voff =
      (uint32_t)r0 * (uint32_t)pitch + (uint32_t)(((lane & 7) ^ ((r0 >> 1) & 7)) * 16);
  const uint64_t base_a = uniform_u64(A), base_b = uniform_u64(B);
  const auto ra = bounded_rsrc(base_a, (int64_t)rows * pitch);
  const auto rb = bounded_rsrc(base_b, (int64_t)cols * pitch);
  // Stages past the last re-read it into a buffer nobody reads again, so that every step issues
  // as many loads and the waits count a constant.
  auto dma_a = [&](int k, lds_char* buf) {
    if (!issuer) return;
    const uint32_t koff = (uint32_t)min(k, steps - 1) * 128u;
#pragma unroll
    for (int i = 0; i < nA; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, buf + (i * 4 + dslot) * 1024, 16, voff,
                                               koff + (uint32_t)i * 32u * (uint32_t)pitch, 0, 0);
  };
  auto dma_b = [&](int k, lds_char* buf) {
    if (!issuer) return;
    const uint32_t koff = (uint32_t)min(k, steps - 1) * 128u;
#pragma unroll
    for (int i = 0; i < nB; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, buf + (i * 4 + dslot) * 1024, 16, voff,
                                               koff + (uint32_t)i * 32u * (uint32_t)pitch, 0, 0);
  };

  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  int a_at[2], b_at[2];
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
    const int piece = ((ks * 4 + g) ^ ((c >> 1) & 7)) << 4;
    a_at[ks] = (wm * MT * 16 + c) * 128 + piece;
    b_at[ks] = (wn * NT * 16 + c) * 128 + piece;
  }
  // 16-row tiles of this wave's band that hold rows
  const int band_rows = rows - wm * MT * 16;
  const int live = band_rows <= 0 ? 0 : min(MT, (band_rows + 15) / 16);
  // Multiply one stage.  B's fragments of both steps are read first, and mid() releases B's
  // buffer for the stage after next, while A's stream through a ring of three row tiles.
  auto compute = [&](const lds_char* abuf, const lds_char* bbuf, auto live_c, auto mid) {
    constexpr int LIVE = decltype(live_c)::value, RING = 3;
    if constexpr (LIVE == 0) {
      mid();
    } else {
      u32x4 fa[RING][2], fb[2][NT];
      auto ld_a = [&](int i) {
        fa[i % RING][0] = *reinterpret_cast<const lds_u32x4*>(abuf + a_at[0] + i * 2048);
        fa[i % RING][1] = *reinterpret_cast<const lds_u32x4*>(abuf + a_at[1] + i * 2048);
      };
      ld_a(0);
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          fb[ks][j] = *reinterpret_cast<const lds_u32x4*>(bbuf + b_at[ks] + j * 2048);
      if constexpr (LIVE > 1) ld_a(1);
      unroll_steps<LIVE>([&](auto I) {
        constexpr int i = decltype(I)::value;
        if constexpr (i + 2 < LIVE) ld_a(i + 2);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
          for (int j = 0; j < NT; ++j) mma_chunk(acc[i][j], fb[ks][j], fa[i % RING][ks], T());
        if constexpr (i == std::min(1, LIVE - 1)) mid();
        if constexpr (sizeof(T) == 2) {  // the next tile's reads between this one's MFMAs
          constexpr int R = i + 2 < LIVE ? 2 : 0, M = 2 * NT;
          unroll_steps<M>([&](auto MI) {
            constexpr int m = decltype(MI)::value;
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            if constexpr (m < R) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
          });
        }
      });
    }
  };
  auto buf_a = [&](auto I) -> lds_char* {
    constexpr int j = decltype(I)::value % S;
    return j == 0 ? a0 : j == 1 ? a1 : j == 2 ? a2 : j == 3 ? a3 : j == 4 ? a4 : a5;
  };
  auto buf_b = [&](auto I) -> lds_char* {
    constexpr int j = decltype(I)::value % S;
    return j == 0 ? b0 : j == 1 ? b1 : j == 2 ? b2 : j == 3 ? b3 : j == 4 ? b4 : b5;
  };
  // Step k: stage k has landed (own loads waited for, then the barrier); A's stage k + S - 1 goes
  // out into the buffer step k - 1 finished with, B's stage k + S once every wave holds this
  // one's fragments.
  auto step = [&](int k, auto I, auto live_c) {
    if (k >= steps) return;
    constexpr int i = decltype(I)::value;
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((S - 2) * (nA + nB) + nB)
                 : "memory");
    dma_a(k + S - 1, buf_a(IntC<i + S - 1>{}));
    compute(buf_a(I), buf_b(I), live_c, [&] {
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      dma_b(k + S, buf_b(I));
    });
  };
  unroll_steps<S>([&](auto I) {
    dma_b(decltype(I)::value, buf_b(I));
    if constexpr (decltype(I)::value < S - 1) dma_a(decltype(I)::value, buf_a(I));
  });
  if (issuer) __builtin_amdgcn_s_setprio(3);
  // one copy of the loop per count of live row tiles
  unroll_steps<MT + 1>([&](auto V) {
    if (live == decltype(V)::value) {
      for (int k = 0; k < steps; k += S)
        unroll_steps<S>([&](auto I) { step(k + decltype(I)::value, I, V); });
    }
  });
  // drain the loads issued past the last stage before the LDS is used again
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  if constexpr (G::kSplits) {
    if (slot) {
      store_partial(slot, acc, live);
      return;
    }
  }
  __syncthreads();

  // Epilogue through LDS, in passes of the row tiles that fit: B's fragment goes first in the
  // MFMA, so lane (c, g) holds row c of each 16-row tile and columns 4 g .. 4 g + 3.
  constexpr int kRow = G::BN * 4, kMask = std::min(16, kRow / 16) - 1, kEights = G::BN / 8;
  constexpr int IP = std::min(MT, G::kLds / (G::WM * 16 * kRow));  // row tiles of a band per pass
  static_assert(IP >= 1, "a row tile fits");
#pragma unroll
  for (int i0 = 0; i0 < MT; i0 += IP) {
    if (i0) __syncthreads();
#pragma unroll
    for (int ii = 0; ii < IP; ++ii) {
      if (i0 + ii >= MT) break;
      const int r = (wm * IP + ii) * 16 + c;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int piece = (wn * NT + j) * 4 + g;
        *reinterpret_cast<lds_f32x4*>(a0 + r * kRow + ((piece ^ (r & kMask)) << 4)) = acc[i0 + ii][j];
      }
    }
    __syncthreads();
    // eight columns for each thread
    by_act(out.act, [&](auto act) __attribute__((always_inline)) {
      for (int q = tid; q < G::WM * IP * 16 * kEights; q += 512) {
        const int r = q / kEights, p = q % kEights;
        const int band = r / (IP * 16), i = i0 + (r / 16) % IP;
        const int row = (band * MT + i) * 16 + (r & 15), col = p * 8;
        if (i >= MT || row >= rows || col >= cols) continue;
        float v[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const f32x4 u = *reinterpret_cast<const lds_f32x4*>(
              a0 + r * kRow + (((2 * p + h) ^ (r & kMask)) << 4));
#pragma unroll
          for (int b = 0; b < 4; ++b) v[4 * h + b] = u[b];
        }
        finish<decltype(act)::value>(out, bias_row, row0 + row, N, col0 + col, v);
      }
    });
  }
}

template <class T>
struct LinearKern {
  const T* x;
  const T* w;
  const int32_t* offsets;  // nullable: one expert holds all R rows
  const int32_t* table;    // nullable with few experts (RowTiles)
  LinearOut<T> out;
  f32x4* partial;  // slots of partial sums (s_max > 1)
  int R, E, N, K, n_tiles, group_n, s_max;
};

template <class T, class G>
__global__ void __launch_bounds__(512) linear_kernel(const LinearKern<T> a) {
  extern __shared__ __attribute__((aligned(1024))) char smem_dyn[];
  constexpr int S = G::kStages, SA = G::kABytes, SB = G::kBBytes;
  lds_char* base = (lds_char*)smem_dyn;
  lds_char* bb = base + S * SA;
  const RowTiles row_tiles(a.offsets, a.table, a.E, a.R, G::BM);
  const int steps = a.K * (int)sizeof(T) / 128;
  TileWork w;
  for (int j = blockIdx.x >> 3; tile_work(row_tiles, a.n_tiles, a.group_n, a.s_max, j, &w);
       j += gridDim.x >> 3) {
    const int col0 = w.nt * G::BN;
    const int k0 = w.piece * steps / w.pieces, k1 = (w.piece + 1) * steps / w.pieces;
    const int at = k0 * (128 / (int)sizeof(T));
    f32x4* slot = w.slot < 0 ? nullptr : a.partial + (int64_t)w.slot * (G::BM * G::BN / 4);
    // buffers past the ring's stages are never used
    linear_body<T, G>(
        a.x + (int64_t)w.rt.begin * a.K + at, min(w.rt.end - w.rt.begin, G::BM),
        a.w + ((int64_t)w.rt.e * a.N + col0) * a.K + at, min(a.N - col0, G::BN),
        (int64_t)a.K * sizeof(T), k1 - k0, a.out,
        a.out.bias ? a.out.bias + (int64_t)w.rt.e * a.N : nullptr, w.rt.begin, col0, a.N, slot,
        base, base + SA, base + (S > 2 ? 2 : 0) * SA, base + (S > 3 ? 3 : 0) * SA,
        base + (S > 4 ? 4 : 0) * SA, base + (S > 5 ? 5 : 0) * SA, bb, bb + SB,
        bb + (S > 2 ? 2 : 0) * SB, bb + (S > 3 ? 3 : 0) * SB, bb + (S > 4 ? 4 : 0) * SB,
        bb + (S > 5 ? 5 : 0) * SB);
    // every wave's reads of the LDS are done
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  }
}

// The pieces' sums in piece order, and the epilogue: one wave per (tail tile, wave, row tile i),
// grid (kSplitCUs, 8 MT / 4), surplus blocks exit.
template <class T, int BM>
__global__ void __launch_bounds__(256) linear_sum_kernel(const LinearKern<T> a) {
  constexpr int NT = 4, MT = BM / 32;
  const RowTiles rows(a.offsets, a.table, a.E, a.R, BM);
  const TailSplit ts = tail_split_of(rows.count, a.n_tiles, a.s_max);
  if ((int)blockIdx.x >= ts.tail) return;
  int mt, nt;
  dense_tile(ts.whole + blockIdx.x, rows.count, a.n_tiles, a.group_n, &mt, &nt);
  const RowTile rt = rows.at(mt);
  const int unit = blockIdx.y * 4 + threadIdx.x / kWave;  // wave * MT + i
  const int wave = unit / MT, i = unit - wave * MT;
  const int lane = lane_id(), row = ((wave >> 2) * MT + i) * 16 + (lane & 15);
  const int live = min(rt.end - rt.begin, BM);
  if (row - (lane & 15) >= live) return;
  constexpr int kSlot = 8 * MT * NT * kWave;
  const f32x4* src = a.partial + (int64_t)blockIdx.x * ts.pieces * kSlot + unit * NT * kWave + lane;
  const float* bias_row = a.out.bias ? a.out.bias + (int64_t)rt.e * a.N : nullptr;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int col = nt * 256 + (wave & 3) * 64 + j * 16;
    if (col >= a.N) break;
    const f32x4 first = src[j * kWave];
    float v[4] = {first[0], first[1], first[2], first[3]};
    for (int p = 1; p < ts.pieces; ++p) {
      const f32x4 u = src[(int64_t)p * kSlot + j * kWave];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] += u[q];
    }
    if (row < live)
      by_act(a.out.act, [&](auto act) {
        finish<decltype(act)::value>(a.out, bias_row, rt.begin + row, a.N, col + 4 * (lane >> 4), v);
      });
  }
}

// ---------------------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------------------
namespace {
// bf16: 64, 128 or 256 rows by 256 columns by the mean rows of an expert; where 64 rows by 32 columns
// give no more blocks than the CUs hold at once, two each, that (rows, K -> N of one expert, us in
// 64 x 32 tiles and in the best other: 1, 4096 -> 4096 11.3 and 21.0; 33, 2048 -> 7168 9.9 and 19.4;
// 64, 4096 -> 14336 24.3 and 32.5; 128, 4096 -> 4096 15.4 and 27.5; 64, 14336 -> 4096 39.5 and 37.4;
// eight experts, 512 rows, 2048 -> 1408 14.5 and 22.7; 128 rows, 4096 -> 14336, where the rule takes 64
// x 256, 186 and 185).  fp32: 128 x 256, or 64 x 64 where those are fewer than two for each CU
// (eight experts, 1001 rows, 512 -> 1024 14 us in small and 65 in large tiles; 4096 rows, 1024 -> 1024
// 75 and 127; one, 4096 rows, 1024 -> 4096 287 and 255).
enum LinearForm { kRows64, kRows128, kRows256, kFew, kSmall32 };
LinearForm linear_form(int64_t R, int64_t E, int64_t N, int elt) {
  auto row_tiles = [&](int64_t bm) { return E * ((R + bm * E - 1) / (bm * E)); };  // of equal experts
  if (elt == 4)
    return row_tiles(128) * ((N + 255) / 256) < 2 * kSplitCUs ? kSmall32 : kRows128;
  if (row_tiles(64) * (N / 32) <= 2 * kSplitCUs) return kFew;
  return R <= 32 * E ? kRows64 : R <= 128 * E ? kRows128 : kRows256;
}
}  // namespace

GroupPlan linear_plan(int64_t R, int64_t E, int64_t N, int elt) {
  static const int kRows[] = {64, 128, 256, 64, 64};
  GroupPlan p;
  p.bm = kRows[linear_form(R, E, N, elt)];
  p.m_max = (R + E * (p.bm - 1)) / p.bm;
  return p;
}

int64_t linear_columns(int64_t R, int64_t E, int64_t N, int elt) {
  const LinearForm f = linear_form(R, E, N, elt);
  return f == kFew ? 32 : f == kSmall32 ? 64 : 256;
}

GroupSplit linear_split(int64_t R, int64_t E, int64_t N, int64_t K, int elt) {
  const LinearForm f = linear_form(R, E, N, elt);
  if (f == kFew || f == kSmall32) return GroupSplit{1, 0};
  return group_split(linear_plan(R, E, N, elt), E, N, K * elt / 128, 96);
}

template <class T, class G>
static hipError_t run_linear(LinearKern<T> k, int64_t m_max, hipStream_t s) {
  k.n_tiles = (k.N + G::BN - 1) / G::BN;
  k.group_n = G::BM <= 64 ? k.n_tiles : std::min(k.n_tiles, 8);
  k.s_max = linear_split(k.R, k.E, k.N, k.K, sizeof(T)).s_max;
  if (k.s_max > 1 && !k.partial) return hipErrorInvalidValue;
  hipError_t e = hipFuncSetAttribute((const void*)linear_kernel<T, G>,
                                     hipFuncAttributeMaxDynamicSharedMemorySize, G::kLds);
  if (e != hipSuccess) return e;
  // one block for each share of a CU's LDS at most, a multiple of the 8 XCDs
  const int64_t tiles = m_max * k.n_tiles + (k.s_max > 1 ? kSplitCUs : 0);
  const unsigned grid =
      (unsigned)std::min<int64_t>((tiles + 7) / 8 * 8, 160 * 1024 / G::kLds * kSplitCUs);
  linear_kernel<T, G><<<grid, 512, G::kLds, s>>>(k);
  if ((e = hipGetLastError()) != hipSuccess || k.s_max < 2) return e;
  if constexpr (G::kSplits) {
    linear_sum_kernel<T, G::BM><<<dim3(kSplitCUs, 8 * G::MT / 4), 256, 0, s>>>(k);
    return hipGetLastError();
  }
  return hipErrorInvalidValue;
}

template <class T>
static hipError_t run_linear_type(const LinearArgs& a, hipStream_t s) {
  LinearKern<T> k = {};
  k.x = (const T*)a.x;
  k.w = (const T*)a.w;
  k.offsets = a.offsets;
  k.table = a.table;
  k.out = {a.bias, (const T*)a.residual, (T*)a.z, (T*)a.y, a.act};
  k.partial = (f32x4*)a.partial;
  k.R = (int)a.R;
  k.E = (int)a.E;
  k.N = (int)a.N;
  k.K = (int)a.K;
  const int64_t m_max = linear_plan(a.R, a.E, a.N, sizeof(T)).m_max;
  const LinearForm form = linear_form(a.R, a.E, a.N, sizeof(T));
  if constexpr (sizeof(T) == 4) {
    if (form == kSmall32) return run_linear<T, LinearTile<64, 64, 2, 4, 4>>(k, m_max, s);
    return run_linear<T, LinearTile<128, 256, 2, 4, 3>>(k, m_max, s);
  } else {
    if (form == kFew) return run_linear<T, LinearTile<64, 32, 4, 2, 6>>(k, m_max, s);
    if (form == kRows64) return run_linear<T, LinearTile<64, 256, 2, 4, 4>>(k, m_max, s);
    if (form == kRows128) return run_linear<T, LinearTile<128, 256, 2, 4, 3>>(k, m_max, s);
    return run_linear<T, LinearTile<256, 256, 2, 4, 2>>(k, m_max, s);
  }
}

hipError_t launch_linear(const LinearArgs& a, hipStream_t s) {
  if (a.R <= 0) return hipSuccess;
  return a.dtype == 1 ? run_linear_type<bf16>(a, s) : run_linear_type<float>(a, s);
}

}  // namespace moe
