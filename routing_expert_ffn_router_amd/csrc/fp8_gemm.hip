// Products of e4m3 operands with a scale for each block of 128, grouped by expert; with SwiGLU
// and the hidden rows' quantization in the epilogue for the gate and up weights.
//
//   y[r, n] = sum_b xs[r, b] * ws[e, n / 128, b] * (xq[r, b] . wq[e, n, b])
//
// One step of the reduction is one scale block of 128 bytes per row, one
// v_mfma_f32_16x16x128_f8f6f4 for each 16 x 16 tile of outputs.
//   - E8M0 scales are operands of that instruction: a lane gives the exponent byte of its row
//     (the same for the four lanes that hold the row's 128 values).
//   - fp32 scales: the instruction starts from zero and acc += product * (xs * ws) follows in
//     fp32.
// The order of the 128 values within a step is free (both operands use one order and the scale is
// the same for all), so a lane takes the 16-byte pieces g and g + 4 of its row's 128 bytes (g
// = lane / 16).  The weight fragment goes first: a lane then holds one row's four consecutive
// output columns, and the row's scale is one value per lane.
//
// Two kernels.  Few rows per expert (at most 32 on average; decode): every weight is read once
// and bounds the time, so waves load weight fragments straight into registers, a ring of steps
// ahead, and nothing is shared through LDS.  More rows: weights and rows go through LDS.
#include <algorithm>

#include "fp8_common.h"
#include "gemm_common.h"
#include "kernels.h"

namespace moe {

typedef int i32x8 __attribute__((ext_vector_type(8)));

struct Fp8Kern {
  const uint8_t* xq;
  const void* xs;
  const int32_t* src;  // nullable
  int x_rows;
  const uint8_t* b0;
  const void* b0s;
  const uint8_t* b1;
  const void* b1s;
  int R, N, K;
  const int32_t* offsets;  // nullable: one expert holds all R rows
  const int32_t* table;
  bf16* y;
  uint8_t* hq;
  void* hs;
  int n_tiles, group_n;
};

__device__ inline i32x8 join(const u32x4& a, const u32x4& b) {
  return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3],
               (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// A scale as it is used: the exponent byte, or the fp32 value's bits.
template <bool E8M0>
__device__ inline uint32_t load_scale(const void* p, int64_t i) {
  if (E8M0) return static_cast<const uint8_t*>(p)[i];
  return static_cast<const uint32_t*>(p)[i];
}

// acc += (w . x) * 2^(sw - 127) * 2^(sx - 127)
__device__ inline void mma_e8m0(f32x4& acc, const i32x8& w, const i32x8& x, uint32_t sw,
                                uint32_t sx) {
  acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, acc, 0, 0, 0, (int)sw, 0,
                                                         (int)sx);
}
__device__ inline f32x4 mma_zero(const i32x8& w, const i32x8& x) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0,
                                                          0, 0, 0, 0);
}
__device__ inline void add_scaled(f32x4& acc, const f32x4& p, float s) {
#pragma unroll
  for (int q = 0; q < 4; ++q) acc[q] = fmaf(p[q], s, acc[q]);
}

// Row tile and n-tile of this block: the tiles are dealt to the 8 XCDs (blocks go round them in
// turn) in contiguous shares of the tiles there are, so that a share's tiles keep their rows
// and weights in one L2.  False: no tile.
__device__ inline bool fp8_tile(const Fp8Kern& a, int* mt, int* nt) {
  const int m_tiles = a.table[0], total = m_tiles * a.n_tiles;
  const int xcd = blockIdx.x & 7, j = blockIdx.x >> 3, per = (total + 7) / 8;
  const int i = xcd * per + j;
  if (j >= per || i >= total) return false;
  dense_tile(i, m_tiles, a.n_tiles, a.group_n, mt, nt);
  return true;
}

// Row of xq for row r of the grouped rows.
__device__ inline int x_row(const Fp8Kern& a, int r) {
  return a.src ? min(max(a.src[r], 0), a.x_rows - 1) : r;
}

// ---------------------------------------------------------------------------------------
// few rows per expert
// ---------------------------------------------------------------------------------------
// Eight waves; WK of them share a column tile and take every WK-th step of the reduction (their
// sums are added through LDS in wave order), 8 / WK column tiles of 16 per block.  LIVE:
// 16-row tiles that hold rows.  D: steps in flight.
template <bool SWIGLU, bool E8M0, int WK, int LIVE, int D>
__device__ inline void skinny_body(const Fp8Kern& a, int e, int m_begin, int rows, int nt,
                                   float* smem) {
  constexpr int NW = SWIGLU ? 2 : 1, WN = 8 / WK;
  const int lane = lane_id(), wave = threadIdx.x / kWave;
  const int c = lane & 15, g = lane >> 4;
  const int wn = wave % WN, wk = wave / WN;
  const int n0 = (nt * WN + wn) * 16;
  const int KB = a.K / kScaleBlock;
  const uint8_t* wp[NW];
  const void* wsp[NW];
  int64_t wsi;
  {
    const int64_t row = (int64_t)e * a.N + n0 + c;
    wp[0] = a.b0 + row * a.K + g * 16;
    wsp[0] = a.b0s;
    if constexpr (SWIGLU) {
      wp[1] = a.b1 + row * a.K + g * 16;
      wsp[1] = a.b1s;
    }
    wsi = ((int64_t)e * (a.N / kScaleBlock) + __builtin_amdgcn_readfirstlane(n0 / kScaleBlock)) *
          KB;
  }
  const uint8_t* xp[LIVE];
  int64_t xsi[LIVE];
#pragma unroll
  for (int i = 0; i < LIVE; ++i) {
    const int64_t row = x_row(a, m_begin + min(i * 16 + c, rows - 1));
    xp[i] = a.xq + row * a.K + g * 16;
    xsi[i] = row * KB;
  }
  struct Step {
    u32x4 w[NW][2], x[LIVE][2];
    uint32_t ws[NW], xs[LIVE];
  };
  auto load = [&](Step& s, int t) {
    const int kb = min(wk + t * WK, KB - 1);  // past the end: the last step again, not used
    const int64_t off = (int64_t)kb * kScaleBlock;
#pragma unroll
    for (int j = 0; j < NW; ++j) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        s.w[j][h] = __builtin_nontemporal_load(
            reinterpret_cast<const u32x4*>(wp[j] + off + h * 64));
      s.ws[j] = load_scale<E8M0>(wsp[j], wsi + kb);
    }
#pragma unroll
    for (int i = 0; i < LIVE; ++i) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        s.x[i][h] = *reinterpret_cast<const u32x4*>(xp[i] + off + h * 64);
      s.xs[i] = load_scale<E8M0>(a.xs, xsi[i] + kb);
    }
  };
  f32x4 acc[NW][LIVE];
#pragma unroll
  for (int j = 0; j < NW; ++j)
#pragma unroll
    for (int i = 0; i < LIVE; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](const Step& s) {
#pragma unroll
    for (int j = 0; j < NW; ++j) {
      const i32x8 w = join(s.w[j][0], s.w[j][1]);
#pragma unroll
      for (int i = 0; i < LIVE; ++i) {
        const i32x8 x = join(s.x[i][0], s.x[i][1]);
        if constexpr (E8M0)
          mma_e8m0(acc[j][i], w, x, s.ws[j], s.xs[i]);
        else
          add_scaled(acc[j][i], mma_zero(w, x),
                     __uint_as_float(s.ws[j]) * __uint_as_float(s.xs[i]));
      }
    }
  };
  const int steps = (KB - wk + WK - 1) / WK;  // may be 0 for a wave past a short reduction
  Step ring[D];
#pragma unroll
  for (int d = 0; d < D; ++d) load(ring[d], d);
  int t = 0;
  for (; t + D <= steps; t += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      multiply(ring[d]);
      load(ring[d], t + d + D);
    }
  }
#pragma unroll
  for (int d = 0; d < D - 1; ++d)
    if (t + d < steps) multiply(ring[d]);

  if constexpr (SWIGLU) {
    // the block's 128 columns are one scale block of h: the row's largest magnitude over the
    // four lanes that hold its columns in this wave, then over the eight waves through LDS
    uint32_t* wave_max = reinterpret_cast<uint32_t*>(smem);  // [LIVE * 16][8]
    float h[LIVE][4];
#pragma unroll
    for (int i = 0; i < LIVE; ++i) {
      uint32_t m = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        h[i][q] = silu_f32(acc[0][i][q]) * acc[1][i][q];
        m = max(m, abs_bits(h[i][q]));
      }
      m = max(m, (uint32_t)__shfl_xor((int)m, 16, kWave));
      m = max(m, (uint32_t)__shfl_xor((int)m, 32, kWave));
      if (g == 0) wave_max[(i * 16 + c) * 8 + wave] = m;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < LIVE; ++i) {
      if (i * 16 + c >= rows) continue;
      uint32_t m = 0;
#pragma unroll
      for (int w = 0; w < 8; ++w) m = max(m, wave_max[(i * 16 + c) * 8 + w]);
      const bool finite = m < kInfBits;
      const int ex = finite ? scale_exponent(m) : 0;
      const float r = inv_scale(ex);
      const int64_t row = m_begin + i * 16 + c;
      *reinterpret_cast<uint32_t*>(a.hq + row * a.N + n0 + 4 * g) =
          finite ? pack_e4m3(h[i][0] * r, h[i][1] * r, h[i][2] * r, h[i][3] * r) : kNan4;
      if (wave == 0 && g == 0)
        store_scale(a.hs, row * (a.N / kScaleBlock) + nt, E8M0 ? kScaleE8M0 : kScaleF32, ex,
                    finite);
    }
  } else {
    typedef bf16 bf16x4 __attribute__((ext_vector_type(4)));
    auto store = [&](int i, const f32x4& v) {
      if (i * 16 + c < rows)
        *reinterpret_cast<bf16x4*>(a.y + (int64_t)(m_begin + i * 16 + c) * a.N + n0 + 4 * g) =
            bf16x4{(bf16)v[0], (bf16)v[1], (bf16)v[2], (bf16)v[3]};
    };
    if constexpr (WK == 1) {
#pragma unroll
      for (int i = 0; i < LIVE; ++i) store(i, acc[0][i]);
    } else {
      f32x4* part = reinterpret_cast<f32x4*>(smem);  // [wk][wn][LIVE][64]
#pragma unroll
      for (int i = 0; i < LIVE; ++i) part[((wk * WN + wn) * LIVE + i) * kWave + lane] = acc[0][i];
      __syncthreads();
      for (int i = wk; i < LIVE; i += WK) {
        f32x4 v = part[(wn * LIVE + i) * kWave + lane];
#pragma unroll
        for (int w = 1; w < WK; ++w) {
          const f32x4 u = part[((w * WN + wn) * LIVE + i) * kWave + lane];
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] += u[q];
        }
        store(i, v);
      }
    }
  }
}

constexpr int kSkinnyRows = 64;

template <bool SWIGLU, bool E8M0, int WK>
__global__ void __launch_bounds__(512) skinny_kernel(const Fp8Kern a) {
  __shared__ __attribute__((aligned(16))) float smem[WK > 1 ? 8 * 4 * kWave * 4 : kSkinnyRows * 8];
  int mt, nt;
  if (!fp8_tile(a, &mt, &nt)) return;
  const int e = a.table[1 + 2 * mt], m_begin = a.table[2 + 2 * mt];
  const int m_end = a.offsets ? min(a.offsets[e + 1], a.R) : a.R;
  const int rows = min(m_end - m_begin, kSkinnyRows);
  if (rows <= 16)
    skinny_body<SWIGLU, E8M0, WK, 1, 4>(a, e, m_begin, rows, nt, smem);
  else if (rows <= 32)
    skinny_body<SWIGLU, E8M0, WK, 2, 4>(a, e, m_begin, rows, nt, smem);
  else if (rows <= 48)
    skinny_body<SWIGLU, E8M0, WK, 3, 3>(a, e, m_begin, rows, nt, smem);
  else
    skinny_body<SWIGLU, E8M0, WK, 4, 3>(a, e, m_begin, rows, nt, smem);
}

// ---------------------------------------------------------------------------------------
// many rows per expert
// ---------------------------------------------------------------------------------------
// BM rows x 256 weight rows (with SwiGLU 128 gate and the 128 up rows of the same columns),
// eight waves as 2 x 4, each 16-row tiles MT = BM / 32 by four 16-column tiles.  A stage of the
// LDS rings holds one scale block (128 bytes) of each row; slot of 16-byte piece c of row r is
// c ^ ((r >> 1) & 7), which makes a fragment's reads free of bank conflicts.  Waves 4-7 issue
// the direct loads to LDS, waves 0-3 bring the scales: fp32 scales arrive in LDS as the products
// xs * ws of the tile's two weight blocks, E8M0 bytes as words.
template <int BM>
struct Fp8Tile {
  static constexpr int kStages = BM <= 128 ? 3 : 2;
  static constexpr int kABytes = BM * 128, kBBytes = 256 * 128;
  static constexpr int kScaleWords = 2 * BM + 2;
  static constexpr int kRing = kStages * (kABytes + kBBytes);
  static constexpr int kLds = kRing + 2 * ((kScaleWords * 4 + 255) / 256 * 256);
  static_assert(kLds <= 160 * 1024, "LDS of one CU");
};

typedef __attribute__((address_space(3))) uint32_t lds_u32;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) f32x4 lds_f32x4;

template <int BM, bool SWIGLU, bool E8M0>
__device__ __attribute__((always_inline)) inline void fp8_body(
    const Fp8Kern& a, int e, int m_begin, int m_end, int nt, lds_char* __restrict__ a0,
    lds_char* __restrict__ a1, lds_char* __restrict__ a2, lds_char* __restrict__ b0,
    lds_char* __restrict__ b1, lds_char* __restrict__ b2, lds_u32* __restrict__ s0,
    lds_u32* __restrict__ s1) {
  using P = Fp8Tile<BM>;
  constexpr int S = P::kStages, MT = BM / 32, NT = 4;
  constexpr int BN = SWIGLU ? 128 : 256;
  const int tid = threadIdx.x, lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int wm = wave >> 2, wn = wave & 3;
  const int c = lane & 15, g = lane >> 4;
  const int rows = m_end - m_begin, KB = a.K / kScaleBlock;
  const bool issuer = wave >= 4;

  // direct loads: one covers eight rows of 128 bytes; issuing wave d fills blocks 4 i + d
  constexpr int nA = BM / 32, nB = 8;
  const int dslot = wave & 3;
  const int64_t w_row0 = (int64_t)e * a.N + nt * BN;
  const uint64_t base_a = uniform_u64(a.src ? a.xq : a.xq + (int64_t)m_begin * a.K);
  const uint64_t base_b[2] = {uniform_u64(a.b0 + w_row0 * a.K),
                              SWIGLU ? uniform_u64(a.b1 + w_row0 * a.K) : 0};
  uint32_t va[nA], vb[nB];
  auto piece = [&](int r) { return (uint32_t)(((lane & 7) ^ ((r >> 1) & 7)) * 16); };
#pragma unroll
  for (int i = 0; i < nA; ++i) {
    const int r = (i * 4 + dslot) * 8 + lane / 8;
    const int row = min(r, rows - 1);
    va[i] = (uint32_t)(a.src ? x_row(a, m_begin + row) : row) * (uint32_t)a.K + piece(r);
  }
#pragma unroll
  for (int i = 0; i < nB; ++i) {
    const int r = (i * 4 + dslot) * 8 + lane / 8;
    const int row = SWIGLU ? r & 127 : min(r, a.N - 1 - nt * BN);
    vb[i] = (uint32_t)row * (uint32_t)a.K + piece(r);
  }
  auto dma = [&](int kb, lds_char* abuf, lds_char* bbuf) {
    if (!issuer) return;
    const uint32_t koff = (uint32_t)min(kb, KB - 1) * kScaleBlock;
#pragma unroll
    for (int i = 0; i < nA; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer_rsrc(base_a),
                                               abuf + (i * 4 + dslot) * 1024, 16, va[i], koff,
                                               0, 0);
#pragma unroll
    for (int i = 0; i < nB; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer_rsrc(base_b[SWIGLU && i >= 4 ? 1 : 0]),
                                               bbuf + (i * 4 + dslot) * 1024, 16, vb[i], koff,
                                               0, 0);
  };

  // scales: thread t < BM brings row t's, one step ahead in registers, one in LDS
  const bool scaler = tid < BM;
  const int64_t wsi0 = ((int64_t)e * (a.N / 128) + nt * (BN / 128)) * KB;
  // the second block of weights: the up matrix, or the next 128 columns (the last column tile
  // of an odd count repeats its first)
  const int64_t wsi1 = SWIGLU || (nt * 2 + 1) * 128 >= a.N ? wsi0 : wsi0 + KB;
  const int64_t xsi =
      scaler ? (int64_t)x_row(a, m_begin + min(tid, rows - 1)) * KB : 0;
  uint32_t xs = 0, ws0 = 0, ws1 = 0;
  auto scale_load = [&](int kb) {
    if (!scaler) return;
    const int k = min(kb, KB - 1);
    xs = load_scale<E8M0>(a.xs, xsi + k);
    ws0 = load_scale<E8M0>(a.b0s, wsi0 + k);
    ws1 = load_scale<E8M0>(SWIGLU ? a.b1s : a.b0s, wsi1 + k);
  };
  auto scale_put = [&](lds_u32* s) {
    if (!scaler) return;
    if constexpr (E8M0) {
      s[tid] = xs;
      if (tid == 0) {
        s[BM] = ws0;
        s[BM + 1] = ws1;
      }
    } else {
      s[tid] = __float_as_uint(__uint_as_float(xs) * __uint_as_float(ws0));
      s[BM + tid] = __float_as_uint(__uint_as_float(xs) * __uint_as_float(ws1));
    }
  };

  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // 16-row tiles of this wave's band that hold rows
  const int band_rows = rows - wm * MT * 16;
  const int live = band_rows <= 0 ? 0 : min(MT, (band_rows + 15) / 16);
  const int swz = (c >> 1) & 7;
  const int a_frag = (wm * MT * 16 + c) * 128, slot0 = (g ^ swz) * 16, slot1 = ((g + 4) ^ swz) * 16;
  // weight rows of column tile j: with SwiGLU two gate tiles, then the up tiles of the same
  // columns
  auto b_row = [&](int j) {
    return SWIGLU ? (j / 2) * 128 + wn * 32 + (j % 2) * 16 : wn * 64 + j * 16;
  };
  auto frag = [&](const lds_char* p) {
    const u32x4 lo = *reinterpret_cast<const lds_u32x4*>(p + slot0);
    const u32x4 hi = *reinterpret_cast<const lds_u32x4*>(p + slot1);
    return join(lo, hi);
  };
  const int s_row = wm * MT * 16 + c;
  auto compute = [&](const lds_char* abuf, const lds_char* bbuf, const lds_u32* s) {
    i32x8 fb[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) fb[j] = frag(bbuf + (b_row(j) + c) * 128);
    uint32_t w0 = 0, w1 = 0;
    if constexpr (E8M0) {
      w0 = s[BM + (SWIGLU ? 0 : wn >> 1)];
      w1 = SWIGLU ? s[BM + 1] : w0;
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      if (i >= live) break;
      const i32x8 fa = frag(abuf + a_frag + i * 16 * 128);
      if constexpr (E8M0) {
        const uint32_t sx = s[s_row + i * 16];
#pragma unroll
        for (int j = 0; j < NT; ++j) mma_e8m0(acc[i][j], fb[j], fa, j < 2 ? w0 : w1, sx);
      } else {
        const float sa = __uint_as_float(s[(SWIGLU ? 0 : (wn >> 1) * BM) + s_row + i * 16]);
        const float sb = SWIGLU ? __uint_as_float(s[BM + s_row + i * 16]) : sa;
        f32x4 p[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) p[j] = mma_zero(fb[j], fa);
#pragma unroll
        for (int j = 0; j < NT; ++j) add_scaled(acc[i][j], p[j], j < 2 ? sa : sb);
      }
    }
  };

  auto buf_a = [&](auto I) -> lds_char* {
    constexpr int j = decltype(I)::value % S;
    return j == 0 ? a0 : j == 1 ? a1 : a2;
  };
  auto buf_b = [&](auto I) -> lds_char* {
    constexpr int j = decltype(I)::value % S;
    return j == 0 ? b0 : j == 1 ? b1 : b2;
  };
  // Step k: stage k has landed (own loads waited for, then the barrier), the loads of stage
  // k + S - 1 go out into the buffer that step k - 1 finished reading, the scales of step k + 1 go
  // to LDS and those of k + 2 are asked for.
  scale_load(0);
  scale_put(s0);
  scale_load(1);
  unroll_steps<S - 1>([&](auto I) { dma(decltype(I)::value, buf_a(I), buf_b(I)); });
  constexpr int L = S % 2 == 0 ? S : 2 * S;  // the rings repeat
  if (issuer) __builtin_amdgcn_s_setprio(3);
  auto step = [&](int k, auto I) {
    if (k >= KB) return;
    constexpr int i = decltype(I)::value;
    // a wave either issues direct loads or brings scales: the count leaves the direct loads
    // of the S - 2 later stages in flight
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((S - 2) * (nA + nB))
                 : "memory");
    dma(k + S - 1, buf_a(IntC<i + S - 1>{}), buf_b(IntC<i + S - 1>{}));
    scale_put(i % 2 ? s0 : s1);
    scale_load(k + 2);
    compute(buf_a(I), buf_b(I), i % 2 ? s1 : s0);
  };
  for (int k = 0; k < KB; k += L)
    unroll_steps<L>([&](auto I) { step(k + decltype(I)::value, I); });
  // drain the loads issued past the last stage before the LDS is used again
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();

  // Epilogue through LDS: a lane holds four consecutive columns of row c of each 16-row tile.
  // The 16-byte piece p of row r lands in slot p ^ (r & 15).
  if constexpr (SWIGLU) {
    constexpr int kRow = 128 * 4;  // fp32
    static_assert(BM * kRow <= P::kRing, "the tile of h fits the rings");
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int r = (wm * MT + i) * 16 + c;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int p = (wn * 32 + j * 16 + 4 * g) / 4;
        f32x4 v;
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = silu_f32(acc[i][j][q]) * acc[i][j + 2][q];
        *reinterpret_cast<lds_f32x4*>(a0 + r * kRow + ((p ^ (r & 15)) << 4)) = v;
      }
    }
    __syncthreads();
    // eight lanes per row, each four pieces of four columns
    const int sub = tid & 7;
    for (int r = tid / 8; r < min(BM, rows); r += 64) {
      f32x4 v[4];
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = *reinterpret_cast<const lds_f32x4*>(a0 + r * kRow +
                                                   (((j * 8 + sub) ^ (r & 15)) << 4));
#pragma unroll
        for (int q = 0; q < 4; ++q) m = max(m, abs_bits(v[j][q]));
      }
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, 8));
      const bool finite = m < kInfBits;
      const int ex = finite ? scale_exponent(m) : 0;
      const float k = inv_scale(ex);
      uint8_t* dst = a.hq + (int64_t)(m_begin + r) * a.N + nt * 128 + sub * 4;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint32_t*>(dst + j * 32) =
            finite ? pack_e4m3(v[j][0] * k, v[j][1] * k, v[j][2] * k, v[j][3] * k) : kNan4;
      if (sub == 0)
        store_scale(a.hs, (int64_t)(m_begin + r) * (a.N / 128) + nt,
                    E8M0 ? kScaleE8M0 : kScaleF32, ex, finite);
    }
  } else {
    constexpr int kRow = 256 * 2;  // bf16
    static_assert(BM * kRow <= P::kRing, "the tile of y fits the rings");
    typedef bf16 bf16x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int r = (wm * MT + i) * 16 + c;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int b = (wn * 64 + j * 16 + 4 * g) * 2;
        *reinterpret_cast<lds_bf16x4*>(a0 + r * kRow + (((b >> 4) ^ (r & 15)) << 4) + (b & 15)) =
            bf16x4{(bf16)acc[i][j][0], (bf16)acc[i][j][1], (bf16)acc[i][j][2],
                   (bf16)acc[i][j][3]};
      }
    }
    __syncthreads();
    for (int q = tid; q < min(BM, rows) * 32; q += 512) {
      const int r = q / 32, p = q % 32, col = nt * 256 + p * 8;
      if (col >= a.N) continue;
      *reinterpret_cast<u32x4*>(a.y + (int64_t)(m_begin + r) * a.N + col) =
          *reinterpret_cast<const lds_u32x4*>(a0 + r * kRow + ((p ^ (r & 15)) << 4));
    }
  }
}

template <int BM, bool SWIGLU, bool E8M0>
__device__ inline void fp8_run(const Fp8Kern& a, int e, int m_begin, int m_end, int nt,
                               lds_char* base) {
  using P = Fp8Tile<BM>;
  constexpr int A = P::kABytes, B = P::kBBytes;
  lds_char* b = base + P::kStages * A;
  lds_u32* s = reinterpret_cast<lds_u32*>(base + P::kRing);
  // a third buffer exists only where the ring has three stages
  fp8_body<BM, SWIGLU, E8M0>(a, e, m_begin, m_end, nt, base, base + A,
                             base + (P::kStages > 2 ? 2 * A : 0), b, b + B,
                             b + (P::kStages > 2 ? 2 * B : 0), s,
                             s + (P::kScaleWords * 4 + 255) / 256 * 64);
}

// BM: the tile height of the table; tiles of at most 128 rows run the 128-row tile.
template <int BM, bool SWIGLU, bool E8M0>
__global__ void __launch_bounds__(512) fp8_kernel(const Fp8Kern a) {
  extern __shared__ __attribute__((aligned(1024))) char smem_dyn[];
  int mt, nt;
  if (!fp8_tile(a, &mt, &nt)) return;
  const int e = a.table[1 + 2 * mt], m_begin = a.table[2 + 2 * mt];
  const int m_end = a.offsets ? min(a.offsets[e + 1], a.R) : a.R;
  lds_char* base = (lds_char*)smem_dyn;
  if constexpr (BM > 128) {
    if (m_end - m_begin > 128) {
      fp8_run<BM, SWIGLU, E8M0>(a, e, m_begin, m_end, nt, base);
      return;
    }
  }
  fp8_run<128, SWIGLU, E8M0>(a, e, m_begin, m_end, nt, base);
}

// ---------------------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------------------
GroupPlan fp8_plan(int64_t R, int64_t E) {
  GroupPlan p;
  p.small = R <= 32 * E;
  p.bm = p.small ? kSkinnyRows : R <= 128 * E ? 128 : 256;
  p.m_max = (R + E * (p.bm - 1)) / p.bm;
  return p;
}

template <bool SWIGLU, bool E8M0, int WK>
static hipError_t run_skinny(Fp8Kern k, int64_t m_max, hipStream_t s) {
  k.n_tiles = k.N / (128 / WK);
  k.group_n = k.n_tiles;
  skinny_kernel<SWIGLU, E8M0, WK>
      <<<(unsigned)((m_max * k.n_tiles + 7) / 8 * 8), 512, 0, s>>>(k);
  return hipGetLastError();
}

template <int BM, bool SWIGLU, bool E8M0>
static hipError_t run_tiles(Fp8Kern k, int64_t m_max, hipStream_t s) {
  constexpr int BN = SWIGLU ? 128 : 256;
  k.n_tiles = (k.N + BN - 1) / BN;
  k.group_n = std::min(k.n_tiles, 8);
  constexpr int lds = std::max(Fp8Tile<BM>::kLds, Fp8Tile<128>::kLds);
  hipError_t e = hipFuncSetAttribute((const void*)fp8_kernel<BM, SWIGLU, E8M0>,
                                     hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return e;
  fp8_kernel<BM, SWIGLU, E8M0>
      <<<(unsigned)((m_max * k.n_tiles + 7) / 8 * 8), 512, lds, s>>>(k);
  return hipGetLastError();
}

template <bool SWIGLU, bool E8M0>
static hipError_t run_fp8(const Fp8Kern& k, const GroupPlan& p, hipStream_t s) {
  if (p.small) {
    if constexpr (!SWIGLU) {
      // a block of 128 columns for each row tile would leave most CUs idle: split the reduction
      // over the block's waves and take fewer columns
      const int64_t blocks = p.m_max * (k.N / 128);
      if (blocks < 256) return run_skinny<SWIGLU, E8M0, 8>(k, p.m_max, s);
      if (blocks < 1024) return run_skinny<SWIGLU, E8M0, 2>(k, p.m_max, s);
    }
    return run_skinny<SWIGLU, E8M0, 1>(k, p.m_max, s);
  }
  if (p.bm == 128) return run_tiles<128, SWIGLU, E8M0>(k, p.m_max, s);
  return run_tiles<256, SWIGLU, E8M0>(k, p.m_max, s);
}

hipError_t launch_fp8_gemm(const Fp8Args& a, hipStream_t s) {
  if (a.R <= 0) return hipSuccess;
  const GroupPlan p = fp8_plan(a.R, a.E);
  Fp8Kern k;
  k.xq = (const uint8_t*)a.xq;
  k.xs = a.x_scale;
  k.src = a.src_rows;
  k.x_rows = (int)a.x_rows;
  k.b0 = (const uint8_t*)a.b0;
  k.b0s = a.b0_scale;
  k.b1 = (const uint8_t*)a.b1;
  k.b1s = a.b1_scale;
  k.R = (int)a.R;
  k.N = (int)a.N;
  k.K = (int)a.K;
  k.offsets = a.offsets;
  k.table = a.table;
  k.y = (bf16*)a.y;
  k.hq = (uint8_t*)a.hq;
  k.hs = a.h_scale;
  k.n_tiles = k.group_n = 0;
  const bool e8m0 = a.scale_type == kScaleE8M0;
  if (a.b1) return e8m0 ? run_fp8<true, true>(k, p, s) : run_fp8<true, false>(k, p, s);
  return e8m0 ? run_fp8<false, true>(k, p, s) : run_fp8<false, false>(k, p, s);
}

}  // namespace moe
