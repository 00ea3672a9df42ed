// Gradients of the product y[r] = x[r] W[e]^T grouped by expert, bf16 and fp32:
//   dgrad  dx[r, k] = sum_n dy[r, n] W[e, n, k]            (rows r of expert e; reduction N)
//   wgrad  dW[e, n, k] = sum_r dy[r, n] x[r, k]            (reduction over e's rows, ragged)
//
// Both are C[m, n] = sum_p A(m, p) B(p, n) with B stored as p rows of contiguous n (dgrad: W[e];
// wgrad: x), and A stored as m rows of contiguous p (dgrad: dy) or as p rows of contiguous m
// (wgrad: dy, "transposed").  The MFMA wants each operand's values along p in a lane, so an
// operand stored by p rows is turned on its way from LDS to registers: bf16 by the
// transposing LDS read (ds_read_b64_tr_b16: sixteen lanes read four rows of sixteen values and
// each gets one column), fp32 by four-byte reads.  Nothing is transposed in memory.
//   - A stage of the LDS ring holds BP values of p (32 KB for each operand), brought by direct
//     buffer -> LDS loads.  wgrad's last stage ends inside the tile: the buffer resource ends
//     with the expert's last row, and loads past its end write zeros, so the neighbour's rows (or
//     what lies behind the last expert) add nothing, whatever they hold.
//   - LDS slots are permuted within a row so that the sixteen or thirty-two rows a wave reads at
//     once fall into different banks.
//   - Sums are fp32 (fp32 operands: fp32 MFMA), in the order of p, rounded once at the end.
// Bounds and measurements (bf16): many rows, the matrix units and the LDS reads that feed them
// (dgrad of 8191 rows, 14336 -> 4096, 8 experts 0.81 to 0.85 ms between cards, matrix units 65 %
// busy at 1.6 GHz; wgrad of 32767 rows, 32 experts of 2048 x 7168 0.95 to 1.27 ms, 40 % busy: 16
// stages a tile, so that its first loads and its stores weigh more; one dense matrix of 4096 x
// 14336 and 8192 rows 1380 and 1240 TFLOP/s); few rows, HBM (86 rows, 32 experts of 13824 x 3328:
// dgrad reads the weights at 6.6 TB/s, wgrad writes them at 5.0).  fp32 (8192 rows, 8 experts of
// 1024 x 4096): dgrad 0.63 ms, matrix units 73 % busy; wgrad 0.67 to 0.91, 44 %.  Where tiles are
// fewer than CUs, fp32 and wgrad leave the others idle: their reductions are not cut.
#include <algorithm>

#include "gemm_common.h"
#include "kernels.h"

namespace moe {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
typedef __attribute__((address_space(3))) uint32_t lds_u32;

// Output tile BM x BN, 8 waves as 2 x 4, each MT x NT MFMA tiles of 16 x 16.  BP: reduction values
// per stage, two MFMA steps.  A "normal" operand is staged as BM rows of BP values (128 bytes), a
// "turned" one as BP rows of BM (or BN) values.
template <class T, int BM_, int BN_, bool A_TURNED_, int STAGES_>
struct GradTile {
  static constexpr int BM = BM_, BN = BN_, WM = 2, WN = 4;
  static constexpr bool kATurned = A_TURNED_;
  static constexpr int kElt = sizeof(T);
  static constexpr int BP = 128 / kElt;  // 64 bf16, 32 fp32
  static constexpr int MT = BM / WM / 16, NT = BN / WN / 16;
  static constexpr int kABytes = BM * BP * kElt, kBBytes = BN * BP * kElt;
  static constexpr int kStages = STAGES_;
  static constexpr int kLds = kStages * (kABytes + kBBytes);
  // direct loads of 1024 bytes per stage and issuing wave (waves 4-7)
  static constexpr int kALoads = kABytes / 4096, kBLoads = kBBytes / 4096;
  // a turned row is 512 bytes: one load covers two of them
  static_assert(BN * kElt == 512 && (!A_TURNED_ || BM * kElt == 512), "turned rows");
  static_assert(kStages >= 2 && kStages <= 4 && kLds <= 160 * 1024, "LDS of one CU");
};

// Slot of 16-byte piece q of row p in a turned operand's stage.  bf16: a wave's transposing reads
// touch rows 8 g + 4 h + 0..3 (g = 0..3) at 32 consecutive bytes; fp32: rows 4 g + i at 64
// consecutive bytes.  The pieces move in those units.
template <class T>
__device__ inline int turned_slot(int p, int q) {
  if (sizeof(T) == 2) return q ^ (((p & 3) | ((p >> 1) & 4)) << 1);
  return q ^ (((p >> 2) & 3) << 2);
}

// One tile.  A: a normal operand's first row, of a_rows rows of pitch a_pitch elements (rows past
// them load as zeros), or a turned operand's first column, of a_rows columns; B: a turned operand's
// first column, of b_cols.  The reduction runs over [0, P): a normal row's values, a turned
// operand's rows.  C: the tile's first output; rows past a_rows and columns past b_cols are not
// stored.  slot (nullable): the sums are one piece of the reduction and go there instead.
template <class T, class G>
__device__ __attribute__((always_inline)) inline void grad_body(
    const T* __restrict__ A, int64_t a_pitch, int a_rows, const T* __restrict__ B,
    int64_t b_pitch, T* __restrict__ C, f32x4* __restrict__ slot, int64_t c_pitch, int64_t P,
    int b_cols, lds_char* __restrict__ a0, lds_char* __restrict__ a1, lds_char* __restrict__ a2,
    lds_char* __restrict__ a3, lds_char* __restrict__ b0, lds_char* __restrict__ b1,
    lds_char* __restrict__ b2, lds_char* __restrict__ b3) {
  constexpr int E = sizeof(T), MT = G::MT, NT = G::NT, S = G::kStages;
  const int tid = tile_thread(), lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int wm = wave >> 2, wn = wave & 3;
  const int c = lane & 15, g = lane >> 4;
  const bool issuer = wave >= 4;
  const int dslot = wave & 3;

  // Direct loads: load i of issuing wave d fills the 1024 bytes 4 i + d of the stage, lane L the 16
  // bytes L of them.  Turned: rows 8 i + 2 d + (L / 32), whose slot permutation depends on i by
  // its lowest bit only; a lane's offset for even and odd i and a scalar for the rows.  Columns
  // past the operand's (the upper half of a last tile) read the lower half again.
  auto turned_lane = [&](int odd, int64_t pitch, int cols) {
    const int p = 8 * odd + 2 * dslot + lane / 32;
    int byte = turned_slot<T>(p, lane % 32) * 16;  // the permutation undoes itself
    if (byte >= cols * E) byte -= 128 * E;
    return (uint32_t)((2 * dslot + lane / 32) * pitch * E) + (uint32_t)byte;
  };
  uint32_t va[2], vb[2];
  if constexpr (G::kATurned) {
    va[0] = turned_lane(0, a_pitch, a_rows);
    va[1] = turned_lane(1, a_pitch, a_rows);
  } else {  // rows 32 i + 8 d + L / 8
    const int r = dslot * 8 + lane / 8;
    va[0] = va[1] =
        (uint32_t)r * (uint32_t)(a_pitch * E) + (uint32_t)(((lane & 7) ^ ((r >> 1) & 7)) * 16);
  }
  vb[0] = turned_lane(0, b_pitch, b_cols);
  vb[1] = turned_lane(1, b_pitch, b_cols);
  const uint64_t base_a = uniform_u64(A), base_b = uniform_u64(B);
  const int steps = (int)((P + G::BP - 1) / G::BP);
  const uint32_t a_row = (uint32_t)(a_pitch * E), b_row = (uint32_t)(b_pitch * E);
  // Stages past the last re-read it into a buffer nobody reads again, so that every step issues
  // as many loads and the waits count a constant.
  auto dma_a = [&](int k, lds_char* buf) {
    if (!issuer) return;
    const int64_t p0 = (int64_t)min(k, steps - 1) * G::BP;
    if constexpr (G::kATurned) {
      const auto r = bounded_rsrc(base_a + p0 * a_row, (P - p0 - 1) * a_row + a_rows * E);
#pragma unroll
      for (int i = 0; i < G::kALoads; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, buf + (i * 4 + dslot) * 1024, 16, va[i & 1],
                                                 (uint32_t)i * 8u * a_row, 0, 0);
    } else {
      const auto r = bounded_rsrc(base_a, (int64_t)a_rows * a_row);
#pragma unroll
      for (int i = 0; i < G::kALoads; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, buf + (i * 4 + dslot) * 1024, 16, va[0],
                                                 (uint32_t)p0 * E + (uint32_t)i * 32u * a_row, 0,
                                                 0);
    }
  };
  auto dma_b = [&](int k, lds_char* buf) {
    if (!issuer) return;
    const int64_t p0 = (int64_t)min(k, steps - 1) * G::BP;
    const auto r = bounded_rsrc(base_b + p0 * b_row, (P - p0 - 1) * b_row + b_cols * E);
#pragma unroll
    for (int i = 0; i < G::kBLoads; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, buf + (i * 4 + dslot) * 1024, 16, vb[i & 1],
                                               (uint32_t)i * 8u * b_row, 0, 0);
  };

  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // Fragment of 16 columns of a turned operand for MFMA step ks of the stage: lane (c, g) gets
  // column c's values p = 8 g .. 8 g + 7 (bf16) or 4 g .. 4 g + 3 (fp32) of the step, as a normal
  // operand's 16-byte piece g holds them.  turned_at: the lane's byte for 16-column tile t; the
  // rows that follow it are constants apart, since the permutation depends on the lane only.
  auto turned_at = [&](int t) {
    if constexpr (E == 2) {
      const int p = 8 * g + c / 4, byte = t * 32 + (c % 4) * 8;
      return p * 512 + (turned_slot<T>(p, byte >> 4) << 4) + (byte & 15);
    } else {
      const int p = 4 * g, byte = t * 64 + c * 4;
      return p * 512 + (turned_slot<T>(p, byte >> 4) << 4) + (byte & 15);
    }
  };
  auto turned_frag = [&](const lds_char* buf, int at, int ks) -> u32x4 {
    u32x4 v;
    if constexpr (E == 2) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const s16x4 t = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_s16x4*)(buf + at + (ks * 32 + 4 * h) * 512));
        typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
        const u32x2 w = __builtin_bit_cast(u32x2, t);
        v[2 * h] = w[0];
        v[2 * h + 1] = w[1];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = *reinterpret_cast<const lds_u32*>(buf + at + (ks * 16 + i) * 512);
    }
    return v;
  };
  int a_at[G::kATurned ? MT : 2], b_at[NT];
  if constexpr (G::kATurned) {
#pragma unroll
    for (int i = 0; i < MT; ++i) a_at[i] = turned_at(wm * MT + i);
  } else {
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
      a_at[ks] = (wm * MT * 16 + c) * 128 + (((ks * 4 + g) ^ ((c >> 1) & 7)) << 4);
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) b_at[j] = turned_at(wn * NT + j);
  auto a_frag = [&](const lds_char* buf, int ks, int i) -> u32x4 {
    if constexpr (G::kATurned)
      return turned_frag(buf, a_at[i], ks);
    else
      return *reinterpret_cast<const lds_u32x4*>(buf + a_at[ks] + i * 2048);
  };
  // 16-row tiles of this wave's band that hold rows
  const int band_rows = a_rows - wm * MT * 16;
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
        fa[i % RING][0] = a_frag(abuf, 0, i);
        fa[i % RING][1] = a_frag(abuf, 1, i);
      };
      ld_a(0);
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int j = 0; j < NT; ++j) fb[ks][j] = turned_frag(bbuf, b_at[j], ks);
      if constexpr (LIVE > 1) ld_a(1);
      unroll_steps<LIVE>([&](auto I) {
        constexpr int i = decltype(I)::value;
        if constexpr (i + 2 < LIVE) ld_a(i + 2);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
          for (int j = 0; j < NT; ++j) mma_chunk(acc[i][j], fb[ks][j], fa[i % RING][ks], T());
        // B's buffer is released behind the fourth row tile: its MFMAs cover the wait (dgrad and
        // wgrad of many rows, as at the top: 870 and 1050 us released at once, 843 and 1009 behind
        // the second row tile, 818 and 953 behind the fourth, 855 and 1005 behind the sixth)
        if constexpr (i == std::min(3, LIVE - 1)) mid();
        if constexpr (E == 2) {  // the next tile's reads between this one's MFMAs
          constexpr int R = i + 2 < LIVE ? (G::kATurned ? 4 : 2) : 0, M = 2 * NT;
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
    return j == 0 ? a0 : j == 1 ? a1 : j == 2 ? a2 : a3;
  };
  auto buf_b = [&](auto I) -> lds_char* {
    constexpr int j = decltype(I)::value % S;
    return j == 0 ? b0 : j == 1 ? b1 : j == 2 ? b2 : b3;
  };
  constexpr int nA = G::kALoads, nB = G::kBLoads;
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
  if (steps > 0) {
    unroll_steps<S>([&](auto I) {
      dma_b(decltype(I)::value, buf_b(I));
      if constexpr (decltype(I)::value < S - 1) dma_a(decltype(I)::value, buf_a(I));
    });
  }
  if (issuer) __builtin_amdgcn_s_setprio(3);
  auto k_loop = [&](auto live_c) {
    for (int k = 0; k < steps; k += S)
      unroll_steps<S>([&](auto I) { step(k + decltype(I)::value, I, live_c); });
  };
  // one copy of the loop per count of live row tiles; a turned operand's columns come in
  // halves of the tile, so a band is whole or empty
  if constexpr (G::kATurned) {
    if (live == 0)
      k_loop(IntC<0>{});
    else
      k_loop(IntC<MT>{});
  } else {
    unroll_steps<MT + 1>([&](auto V) {
      if (live == decltype(V)::value) k_loop(V);
    });
  }
  // drain the loads issued past the last stage before the LDS is used again
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  if constexpr (E == 2 && !G::kATurned) {
    if (slot) {
      store_partial(slot, acc, live);
      return;
    }
  }
  __syncthreads();

  // Epilogue through LDS, in passes of the row tiles that fit: B's fragment goes first in the
  // MFMA, so lane (c, g) holds row c of each 16-row tile and columns 4 g .. 4 g + 3.
  constexpr int kRow = G::BN * E, kPieces = kRow / 16;
  constexpr int IP = std::min(MT, G::kLds / (G::WM * 16 * kRow));  // row tiles of a band per pass
  static_assert(IP >= 1 && kPieces % 16 == 0, "a row tile fits");
#pragma unroll
  for (int i0 = 0; i0 < MT; i0 += IP) {
    if (i0) __syncthreads();
#pragma unroll
    for (int ii = 0; ii < IP; ++ii) {
      if (i0 + ii >= MT) break;
      const int r = (wm * IP + ii) * 16 + c;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int byte = ((wn * NT + j) * 16 + 4 * g) * E;
        lds_char* dst = a0 + r * kRow + (((byte >> 4) ^ (r & 15)) << 4) + (byte & 15);
        const f32x4 v = acc[i0 + ii][j];
        typedef T tx4 __attribute__((ext_vector_type(4)));
        *reinterpret_cast<__attribute__((address_space(3))) tx4*>(dst) =
            tx4{Elt<T>::from_f32(v[0]), Elt<T>::from_f32(v[1]), Elt<T>::from_f32(v[2]),
                Elt<T>::from_f32(v[3])};
      }
    }
    __syncthreads();
    for (int q = tid; q < G::WM * IP * 16 * kPieces; q += 512) {
      const int r = q / kPieces, p = q % kPieces;
      const int band = r / (IP * 16), i = i0 + (r / 16) % IP;
      const int row = (band * MT + i) * 16 + (r & 15);
      const int col = p * (16 / E);
      if (i >= MT || row >= a_rows || col >= b_cols) continue;
      const u32x4 o = *reinterpret_cast<const lds_u32x4*>(a0 + r * kRow + ((p ^ (r & 15)) << 4));
      u32x4* dst = reinterpret_cast<u32x4*>(C + (int64_t)row * c_pitch + col);
      // weight gradients are the larger part of wgrad's traffic and not read again here: past
      // the caches (few rows per expert 640 -> 590 us, fp32 1466 -> 1379 us)
      if constexpr (G::kATurned)
        __builtin_nontemporal_store(o, dst);
      else
        *dst = o;
    }
  }
}

template <class T, class G>
__device__ inline void grad_run(const T* A, int64_t a_pitch, int a_rows, const T* B,
                                int64_t b_pitch, T* C, f32x4* slot, int64_t c_pitch, int64_t P,
                                int b_cols, lds_char* base) {
  constexpr int S = G::kStages, SA = G::kABytes, SB = G::kBBytes;
  lds_char* b = base + S * SA;
  // buffers past the ring's stages are never used
  grad_body<T, G>(A, a_pitch, a_rows, B, b_pitch, C, slot, c_pitch, P, b_cols, base, base + SA,
                  base + (S > 2 ? 2 * SA : 0), base + (S > 3 ? 3 * SA : 0), b, b + SB,
                  b + (S > 2 ? 2 * SB : 0), b + (S > 3 ? 3 * SB : 0));
}

// A block fills its CU's LDS and works through its share of the tiles: the next one's loads go out
// while the stores of the last are under way, where a block for each tile would wait for them.
//
// dgrad: a tile is a row tile of an expert by 256 columns of K, or a piece of its reduction.
template <class T, class G>
__global__ void __launch_bounds__(512)
dgrad_kernel(const T* __restrict__ dy, const int32_t* __restrict__ offsets,
             const int32_t* __restrict__ table, const T* __restrict__ w, T* __restrict__ dx,
             f32x4* __restrict__ partial, int R, int E, int N, int K, int n_tiles, int group_n,
             int s_max) {
  extern __shared__ __attribute__((aligned(1024))) char smem_dyn[];
  const RowTiles rows(offsets, table, E, R, G::BM);
  TileWork k;
  for (int j = blockIdx.x >> 3; tile_work(rows, n_tiles, group_n, s_max, j, &k);
       j += gridDim.x >> 3) {
    const int col0 = k.nt * G::BN, steps = (N + G::BP - 1) / G::BP;
    const int p0 = k.piece * steps / k.pieces * G::BP;
    const int p1 = min((k.piece + 1) * steps / k.pieces * G::BP, N);
    f32x4* slot = k.slot < 0 ? nullptr : partial + (int64_t)k.slot * (G::BM * G::BN / 4);
    grad_run<T, G>(dy + (int64_t)k.rt.begin * N + p0, N, min(k.rt.end - k.rt.begin, G::BM),
                   w + ((int64_t)k.rt.e * N + p0) * K + col0, K,
                   dx + (int64_t)k.rt.begin * K + col0, slot, K, p1 - p0, min(K - col0, G::BN),
                   (lds_char*)smem_dyn);
    // every wave's reads of the LDS are done
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  }
}

// wgrad: a tile is an expert's BM rows of N by BN columns of K.
template <class T, class G>
__global__ void __launch_bounds__(512)
wgrad_kernel(const T* __restrict__ dy, const T* __restrict__ x,
             const int32_t* __restrict__ offsets, T* __restrict__ dw, int R, int E, int N, int K,
             int m_tiles, int n_tiles) {
  extern __shared__ __attribute__((aligned(1024))) char smem_dyn[];
  const int total = E * m_tiles * n_tiles, per = (total + 7) / 8;
  const int first = (blockIdx.x & 7) * per, end = min(first + per, total);
  for (int t = first + (blockIdx.x >> 3); t < end; t += gridDim.x >> 3) {
    const int e = t / (m_tiles * n_tiles), rem = t - e * (m_tiles * n_tiles);
    const int mt = rem / n_tiles, nt = rem - mt * n_tiles;
    const int r0 = offsets ? min(max(offsets[e], 0), R) : 0;
    const int r1 = offsets ? min(max(offsets[e + 1], r0), R) : R;
    const int row0 = mt * G::BM, col0 = nt * G::BN;
    grad_run<T, G>(dy + (int64_t)r0 * N + row0, N, min(N - row0, G::BM),
                   x + (int64_t)r0 * K + col0, K, dw + ((int64_t)e * N + row0) * K + col0,
                   nullptr, K, r1 - r0, min(K - col0, G::BN), (lds_char*)smem_dyn);
    // every wave's reads of the LDS are done
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  }
}

// ---------------------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------------------
// bf16: 128 rows (three stages) where an expert has few, bound by its weight (86 rows, 32 experts
// of 13824 x 3328 470 against 497 us); 256 above (8 experts of 4096 x 4096 with 32 rows 55.0
// against 52.7; 32 of 2048 x 2048 with 128 rows 81 against 56).
GroupPlan dgrad_plan(int64_t R, int64_t E, int elt) {
  GroupPlan p;
  p.bm = elt == 4 || R <= 16 * E ? 128 : 256;
  p.m_max = (R + E * (p.bm - 1)) / p.bm;
  return p;
}

int64_t group_max_tiles(int64_t R, int64_t E, int64_t N, int64_t K, int elt) {
  // row operands: at most (R + 63 E) / 64 row tiles by ceil(columns / 128), at most 2048 blocks of
  // fewer columns in the few-tiles form of the 8-bit product, and a tail's pieces; wgrad: every
  // tile of every expert's weight
  const int64_t rows = (R + E * 63) / 64 * (std::max(N, K) / 128) + 2048 + kSplitCUs;
  const int64_t b = elt == 2 ? 256 : 128;
  return std::max(rows, E * ((N + b - 1) / b) * ((K + b - 1) / b)) + 8;
}

// One block for each share of a CU's LDS at most, a multiple of the 8 XCDs.
static unsigned grid_of(int64_t tiles, int lds) {
  return (unsigned)std::min<int64_t>((tiles + 7) / 8 * 8, 160 * 1024 / lds * kSplitCUs);
}

template <class K>
static hipError_t allow_lds(K kernel, int bytes) {
  return hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize,
                             bytes);
}

GroupSplit dgrad_split(int64_t R, int64_t E, int64_t N, int64_t K, int elt) {
  if (elt != 2) return GroupSplit{1, 0};
  // (8191 rows, 8 experts, N -> 4096, split against whole, two draws of the rows: N = 2048 139 and
  // 144, 145 and 133 us, 4096 263 and 251, 252 and 268; N = 14336 814 and 898)
  return group_split(dgrad_plan(R, E, elt), E, K, N / 64, 96);
}

template <class T, class G>
static hipError_t run_dgrad(const T* dy, const int32_t* offsets, const int32_t* table,
                            const T* w, T* dx, void* partial, int64_t m_max, int64_t R,
                            int64_t E, int64_t N, int64_t K, hipStream_t s) {
  const int n_tiles = (int)((K + G::BN - 1) / G::BN), group_n = std::min(n_tiles, 8);
  const int s_max = dgrad_split(R, E, N, K, sizeof(T)).s_max;
  if (s_max > 1 && !partial) return hipErrorInvalidValue;
  hipError_t e = allow_lds(dgrad_kernel<T, G>, G::kLds);
  if (e != hipSuccess) return e;
  const unsigned grid =
      grid_of(m_max * n_tiles + (s_max > 1 ? kSplitCUs : 0), G::kLds);
  dgrad_kernel<T, G><<<grid, 512, G::kLds, s>>>(dy, offsets, table, w, dx, (f32x4*)partial,
                                                (int)R, (int)E, (int)N, (int)K, n_tiles, group_n,
                                                s_max);
  if ((e = hipGetLastError()) != hipSuccess || s_max < 2) return e;
  if constexpr (sizeof(T) == 2) {
    partial_sum_kernel<G::BM><<<dim3(kSplitCUs, 8 * G::MT / 4), 256, 0, s>>>(
        (const f32x4*)partial, offsets, table, (int)E, (int)R, n_tiles, group_n, s_max, (int)K,
        dx);
    return hipGetLastError();
  }
  return hipErrorInvalidValue;
}

hipError_t launch_dgrad(int dtype, const void* dy, const int32_t* offsets,
                        const int32_t* table, const void* w, void* dx, void* partial, int64_t R,
                        int64_t E, int64_t N, int64_t K, hipStream_t s) {
  if (R <= 0) return hipSuccess;
  const GroupPlan p = dgrad_plan(R, E, dtype == 1 ? 2 : 4);
  if (dtype != 1)
    return run_dgrad<float, GradTile<float, 128, 128, false, 4>>(
        (const float*)dy, offsets, table, (const float*)w, (float*)dx, partial, p.m_max, R, E, N,
        K, s);
  if (p.bm == 128)
    return run_dgrad<bf16, GradTile<bf16, 128, 256, false, 3>>(
        (const bf16*)dy, offsets, table, (const bf16*)w, (bf16*)dx, partial, p.m_max, R, E, N, K,
        s);
  return run_dgrad<bf16, GradTile<bf16, 256, 256, false, 2>>(
      (const bf16*)dy, offsets, table, (const bf16*)w, (bf16*)dx, partial, p.m_max, R, E, N, K,
      s);
}

template <class T, class G>
static hipError_t run_wgrad(const T* dy, const T* x, const int32_t* offsets, T* dw, int64_t R,
                            int64_t E, int64_t N, int64_t K, hipStream_t s) {
  const int64_t mt = (N + G::BM - 1) / G::BM, nt = (K + G::BN - 1) / G::BN;
  hipError_t e = allow_lds(wgrad_kernel<T, G>, G::kLds);
  if (e != hipSuccess) return e;
  wgrad_kernel<T, G><<<grid_of(E * mt * nt, G::kLds), 512, G::kLds, s>>>(
      dy, x, offsets, dw, (int)R, (int)E, (int)N, (int)K, (int)mt, (int)nt);
  return hipGetLastError();
}

hipError_t launch_wgrad(int dtype, const void* dy, const void* x, const int32_t* offsets,
                        void* dw, int64_t R, int64_t E, int64_t N, int64_t K, hipStream_t s) {
  // fp32: two stages, so that two blocks share a CU and one stores while the other multiplies
  // (four stages in one block: 86 rows, 32 experts of 13824 x 3328 1963 against 1466 us; 4096
  // rows, 8 experts of 2048 x 2048 330 against 293 us)
  if (dtype != 1)
    return run_wgrad<float, GradTile<float, 128, 128, true, 2>>(
        (const float*)dy, (const float*)x, offsets, (float*)dw, R, E, N, K, s);
  return run_wgrad<bf16, GradTile<bf16, 256, 256, true, 2>>(
      (const bf16*)dy, (const bf16*)x, offsets, (bf16*)dw, R, E, N, K, s);
}

}  // namespace moe
