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
//   - LDS slots are permuted within a row so that the sixteen or thirty-two rows a wave reads at once
//     fall into different banks.
//   - Sums are fp32 (fp32 operands: fp32 MFMA), in the order of p, rounded once at the end.
#include <algorithm>

#include "gemm_common.h"
#include "kernels.h"

namespace moe {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
typedef __attribute__((address_space(3))) uint32_t lds_u32;

// Output tile BM x BN, 8 waves as WM x WN.  BP: reduction values per stage.
// A "normal" operand is staged as BM rows of BP values (128 bytes), a "turned" one as BP rows of
// BM (or BN) values.
template <class T, int BM_, int BN_, bool A_TURNED_>
struct GradTile {
  static constexpr int BM = BM_, BN = BN_, WM = 2, WN = 4;
  static constexpr bool kATurned = A_TURNED_;
  static constexpr int kElt = sizeof(T);
  static constexpr int BP = 128 / kElt;        // 64 bf16, 32 fp32
  static constexpr int kStep = 64 / kElt;      // p per MFMA step: 32 bf16, 16 fp32
  static constexpr int MT = BM / WM / 16, NT = BN / WN / 16;
  static constexpr int kABytes = BM * BP * kElt, kBBytes = BN * BP * kElt;
  static constexpr int kStages = 2;
  static constexpr int kLds = kStages * (kABytes + kBBytes);
  static constexpr int kALoads = kABytes / 8192, kBLoads = kBBytes / 8192;  // per wave
  static_assert(kLds <= 160 * 1024 && kABytes % 8192 == 0 && kBBytes % 8192 == 0, "tile");
};

// Slot of 16-byte piece q of row p in a turned operand's stage.  bf16: a wave's transposing reads
// touch rows 8 g + 4 h + 0..3 (g = 0..3) at 32 consecutive bytes; fp32: rows 4 g + i at 64
// consecutive bytes.  The pieces move in those units.
template <class T>
__device__ inline int turned_slot(int p, int q) {
  if (sizeof(T) == 2) return q ^ (((p & 3) | ((p >> 1) & 4)) << 1);
  return q ^ (((p >> 2) & 3) << 2);
}

// A buffer resource over [base, base + bytes): loads past its end give zeros.
__device__ inline __amdgpu_buffer_rsrc_t bounded_rsrc(uint64_t base, int64_t bytes) {
  const int n = (int)min(max(bytes, (int64_t)0), (int64_t)0x7fffffff);
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(base), 0, n, 0x00020000);
}

// One tile.  A: normal operand rows a_row0.. (clamped to a_rows of them) of pitch a_pitch
// elements, or turned operand columns a_col0..; B: turned columns b_col0...  p runs over [0, P)
// of rows whose first is A / B themselves.
template <class T, class G>
__device__ __attribute__((always_inline)) inline void grad_body(
    const T* __restrict__ A, int64_t a_pitch, int a_rows, const T* __restrict__ B,
    int64_t b_pitch, T* __restrict__ C, int64_t c_pitch, int64_t P, int64_t a_cols,
    int64_t b_cols, lds_char* __restrict__ a0, lds_char* __restrict__ a1,
    lds_char* __restrict__ b0, lds_char* __restrict__ b1) {
  constexpr int E = sizeof(T), MT = G::MT, NT = G::NT;
  const int tid = threadIdx.x, lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int wm = wave / G::WN, wn = wave % G::WN;
  const int c = lane & 15, g = lane >> 4;

  // direct loads: load i of wave w fills the 1024 bytes i * 8 + w of the stage, lane L the 16
  // bytes L of them
  uint32_t va[G::kALoads], vb[G::kBLoads];
  auto turned_off = [&](int i, int row_bytes, int64_t pitch) {
    const int at = (i * 8 + wave) * 64 + lane, pieces = row_bytes / 16;
    const int p = at / pieces, slot = at % pieces;
    return (uint32_t)(p * pitch * E) + (uint32_t)turned_slot<T>(p, slot) * 16;  // an involution
  };
#pragma unroll
  for (int i = 0; i < G::kALoads; ++i) {
    if constexpr (G::kATurned) {
      va[i] = turned_off(i, G::BM * E, a_pitch);
    } else {
      const int r = (i * 8 + wave) * 8 + lane / 8;
      const int q = (lane & 7) ^ ((r >> 1) & 7);
      va[i] = (uint32_t)min(r, a_rows - 1) * (uint32_t)(a_pitch * E) + q * 16;
    }
  }
#pragma unroll
  for (int i = 0; i < G::kBLoads; ++i) vb[i] = turned_off(i, G::BN * E, b_pitch);
  const uint64_t base_a = uniform_u64(A), base_b = uniform_u64(B);
  const int steps = (int)((P + G::BP - 1) / G::BP);
  auto dma = [&](int k, lds_char* abuf, lds_char* bbuf) {
    if (k >= steps) return;
    const int64_t p0 = (int64_t)k * G::BP;
    // bytes from the stage's first value to the operand's end: rows p0 .. P - 1 of pitch, the
    // last of them only the columns that exist
    const int64_t bb = ((P - p0 - 1) * b_pitch + b_cols) * E;
    const auto rb = bounded_rsrc(base_b + p0 * b_pitch * E, bb);
    if constexpr (G::kATurned) {
      const int64_t ab = ((P - p0 - 1) * a_pitch + a_cols) * E;
      const auto ra = bounded_rsrc(base_a + p0 * a_pitch * E, ab);
#pragma unroll
      for (int i = 0; i < G::kALoads; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, abuf + (i * 8 + wave) * 1024, 16, va[i], 0,
                                                 0, 0);
    } else {
      const auto ra = buffer_rsrc(base_a + p0 * E);
#pragma unroll
      for (int i = 0; i < G::kALoads; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, abuf + (i * 8 + wave) * 1024, 16, va[i], 0,
                                                 0, 0);
    }
#pragma unroll
    for (int i = 0; i < G::kBLoads; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, bbuf + (i * 8 + wave) * 1024, 16, vb[i], 0, 0,
                                               0);
  };

  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // Fragment of 16 columns col0.. of a turned operand for MFMA step ks: lane (c, g) gets column
  // c's values p = 8 g .. 8 g + 7 (bf16) or 4 g .. 4 g + 3 (fp32) of the step, as a normal
  // operand's 16-byte piece g holds them.
  auto turned_frag = [&](const lds_char* buf, int row_bytes, int ks, int col0) -> u32x4 {
    if constexpr (E == 2) {
      u32x4 v;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int p = ks * 32 + 8 * g + 4 * h + c / 4;
        const int byte = col0 * 2 + (c % 4) * 8;
        const s16x4 t = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_s16x4*)(buf + p * row_bytes + (turned_slot<T>(p, byte >> 4) << 4) + (byte & 15)));
        typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
        const u32x2 w = __builtin_bit_cast(u32x2, t);
        v[2 * h] = w[0];
        v[2 * h + 1] = w[1];
      }
      return v;
    } else {
      u32x4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int p = ks * 16 + 4 * g + i;
        const int byte = (col0 + c) * 4;
        v[i] = *reinterpret_cast<const lds_u32*>(buf + p * row_bytes +
                                                 (turned_slot<T>(p, byte >> 4) << 4) + (byte & 15));
      }
      return v;
    }
  };
  auto a_frag = [&](const lds_char* buf, int ks, int i) -> u32x4 {
    const int r = (wm * MT + i) * 16;
    if constexpr (G::kATurned) {
      return turned_frag(buf, G::BM * E, ks, r);
    } else {
      return *reinterpret_cast<const lds_u32x4*>(buf + (r + c) * 128 +
                                                 (((ks * 4 + g) ^ ((c >> 1) & 7)) << 4));
    }
  };
  auto compute = [&](const lds_char* abuf, const lds_char* bbuf) {
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      u32x4 fb[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) fb[j] = turned_frag(bbuf, G::BN * E, ks, (wn * NT + j) * 16);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const u32x4 fa = a_frag(abuf, ks, i);
#pragma unroll
        for (int j = 0; j < NT; ++j) mma_chunk(acc[i][j], fb[j], fa, T());
      }
    }
  };
  dma(0, a0, b0);
  for (int k = 0; k < steps; k += 2) {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    dma(k + 1, a1, b1);
    compute(a0, b0);
    if (k + 1 < steps) {
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      dma(k + 2, a0, b0);
      compute(a1, b1);
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
      *reinterpret_cast<u32x4*>(C + (int64_t)row * c_pitch + col) =
          *reinterpret_cast<const lds_u32x4*>(a0 + r * kRow + ((p ^ (r & 15)) << 4));
    }
  }
}

template <class T, class G>
__device__ inline void grad_run(const T* A, int64_t a_pitch, int a_rows, const T* B,
                                int64_t b_pitch, T* C, int64_t c_pitch, int64_t P,
                                int64_t a_cols, int64_t b_cols, lds_char* base) {
  lds_char* b = base + 2 * G::kABytes;
  grad_body<T, G>(A, a_pitch, a_rows, B, b_pitch, C, c_pitch, P, a_cols, b_cols, base,
                  base + G::kABytes, b, b + G::kBBytes);
}

// dgrad: one block per (row tile of an expert, 256 columns of K).
template <class T, class G>
__global__ void __launch_bounds__(512)
dgrad_kernel(const T* __restrict__ dy, const int32_t* __restrict__ offsets,
             const int32_t* __restrict__ table, const T* __restrict__ w, T* __restrict__ dx,
             int R, int E, int N, int K, int n_tiles, int group_n) {
  extern __shared__ __attribute__((aligned(1024))) char smem_dyn[];
  RowTile rt;
  int nt;
  if (!group_tile(offsets, table, E, R, G::BM, n_tiles, group_n, &rt, &nt)) return;
  const int col0 = nt * G::BN;
  grad_run<T, G>(dy + (int64_t)rt.begin * N, N, min(rt.end - rt.begin, G::BM),
                 w + (int64_t)rt.e * N * K + col0, K, dx + (int64_t)rt.begin * K + col0, K, N, 0,
                 K - col0, (lds_char*)smem_dyn);
}

// wgrad: one block per (expert, BM rows of N, BN columns of K).
template <class T, class G>
__global__ void __launch_bounds__(512)
wgrad_kernel(const T* __restrict__ dy, const T* __restrict__ x,
             const int32_t* __restrict__ offsets, T* __restrict__ dw, int R, int E, int N, int K,
             int m_tiles, int n_tiles) {
  extern __shared__ __attribute__((aligned(1024))) char smem_dyn[];
  const int total = E * m_tiles * n_tiles;
  const int xcd = blockIdx.x & 7, j = blockIdx.x >> 3, per = (total + 7) / 8;
  const int t = xcd * per + j;
  if (j >= per || t >= total) return;
  const int e = t / (m_tiles * n_tiles), rem = t - e * (m_tiles * n_tiles);
  const int mt = rem / n_tiles, nt = rem - mt * n_tiles;
  const int r0 = offsets ? min(max(offsets[e], 0), R) : 0;
  const int r1 = offsets ? min(max(offsets[e + 1], r0), R) : R;
  const int row0 = mt * G::BM, col0 = nt * G::BN;
  grad_run<T, G>(dy + (int64_t)r0 * N + row0, N, min(N - row0, G::BM),
                 x + (int64_t)r0 * K + col0, K, dw + ((int64_t)e * N + row0) * K + col0, K,
                 r1 - r0, N - row0, K - col0, (lds_char*)smem_dyn);
}

// ---------------------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------------------
GroupPlan dgrad_plan(int64_t R, int64_t E, int elt) {
  GroupPlan p;
  p.bm = elt == 4 || R <= 128 * E ? 128 : 256;
  p.m_max = (R + E * (p.bm - 1)) / p.bm;
  return p;
}

int64_t group_max_blocks(int64_t R, int64_t E, int64_t N, int64_t K, int elt) {
  // row operands: at most (R + 63 E) / 64 row tiles by ceil(columns / 128), and up to 2048 blocks
  // where few blocks are split further; wgrad: every tile of every expert's weight
  const int64_t rows = (R + E * 63) / 64 * (std::max(N, K) / 128) + 2048;
  const int64_t b = elt == 2 ? 256 : 128;
  return std::max(rows, E * ((N + b - 1) / b) * ((K + b - 1) / b)) + 8;
}

template <class K>
static hipError_t allow_lds(K kernel, int bytes) {
  return hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize,
                             bytes);
}

template <class T, class G>
static hipError_t run_dgrad(const T* dy, const int32_t* offsets, const int32_t* table,
                            const T* w, T* dx, const GroupPlan& p, int64_t R, int64_t E,
                            int64_t N, int64_t K, hipStream_t s) {
  const int n_tiles = (int)((K + G::BN - 1) / G::BN);
  hipError_t e = allow_lds(dgrad_kernel<T, G>, G::kLds);
  if (e != hipSuccess) return e;
  dgrad_kernel<T, G><<<(unsigned)((p.m_max * n_tiles + 7) / 8 * 8), 512, G::kLds, s>>>(
      dy, offsets, table, w, dx, (int)R, (int)E, (int)N, (int)K, n_tiles, std::min(n_tiles, 8));
  return hipGetLastError();
}

hipError_t launch_dgrad(int dtype, const void* dy, const int32_t* offsets,
                        const int32_t* table, const void* w, void* dx, int64_t R, int64_t E,
                        int64_t N, int64_t K, hipStream_t s) {
  if (R <= 0) return hipSuccess;
  const GroupPlan p = dgrad_plan(R, E, dtype == 1 ? 2 : 4);
  if (dtype != 1)
    return run_dgrad<float, GradTile<float, 128, 128, false>>(
        (const float*)dy, offsets, table, (const float*)w, (float*)dx, p, R, E, N, K, s);
  if (p.bm == 128)
    return run_dgrad<bf16, GradTile<bf16, 128, 256, false>>(
        (const bf16*)dy, offsets, table, (const bf16*)w, (bf16*)dx, p, R, E, N, K, s);
  return run_dgrad<bf16, GradTile<bf16, 256, 256, false>>(
      (const bf16*)dy, offsets, table, (const bf16*)w, (bf16*)dx, p, R, E, N, K, s);
}

template <class T, class G>
static hipError_t run_wgrad(const T* dy, const T* x, const int32_t* offsets, T* dw, int64_t R,
                            int64_t E, int64_t N, int64_t K, hipStream_t s) {
  const int64_t mt = (N + G::BM - 1) / G::BM, nt = (K + G::BN - 1) / G::BN;
  hipError_t e = allow_lds(wgrad_kernel<T, G>, G::kLds);
  if (e != hipSuccess) return e;
  wgrad_kernel<T, G><<<(unsigned)((E * mt * nt + 7) / 8 * 8), 512, G::kLds, s>>>(
      dy, x, offsets, dw, (int)R, (int)E, (int)N, (int)K, (int)mt, (int)nt);
  return hipGetLastError();
}

hipError_t launch_wgrad(int dtype, const void* dy, const void* x, const int32_t* offsets,
                        void* dw, int64_t R, int64_t E, int64_t N, int64_t K, hipStream_t s) {
  if (dtype != 1)
    return run_wgrad<float, GradTile<float, 128, 128, true>>(
        (const float*)dy, (const float*)x, offsets, (float*)dw, R, E, N, K, s);
  return run_wgrad<bf16, GradTile<bf16, 256, 256, true>>(
      (const bf16*)dy, (const bf16*)x, offsets, (bf16*)dw, R, E, N, K, s);
}

}  // namespace moe
