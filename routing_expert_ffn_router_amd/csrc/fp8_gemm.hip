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
//     fp32.  Where an xs * ws is past fp32's largest number (2^100 and 2^30), though the block's
//     dot product may be 0 or small, a tile is computed again with the exponents given to the
//     instruction, which adds them in a wider range, and only what is left of each scale, 1 <= m
//     < 4, multiplied in fp32 (a product where every tile is: 530 -> 1243 us, 638 -> 1297; that
//     form alone in place of the usual one costs 8 to 17 % of every product; the check costs 1 to
//     2 % of gate/up in 256-row tiles and nothing elsewhere).  The few-tiles form below always
//     takes it: its loads hide the difference (16 rows, K = 4096, N = 16384 21.1 and 21.3 us).
// The order of the 128 values within a step is free (both operands use one order and the scale is
// the same for all), so a lane takes the 16-byte pieces g and g + 4 of its row's 128 bytes (g
// = lane / 16).  The weight fragment goes first: a lane then holds one row's four consecutive
// output columns, and the row's scale is one value per lane.
//
// Weights and rows go through LDS in tiles of 64, 128 or 256 rows by 256 weight rows; a product
// with too few tiles for the CUs splits its reduction over the waves of a block instead.
//   64 rows (at most 32 rows per expert on average; decode): bound by HBM, every weight is read
//   once (256 experts of 7168 / 2048 with 256 tokens, E8M0: gate/up 1.09 ms, down 0.65 ms, 6.5
//   TB/s; the same weights straight into registers reached 3.6-4.1 TB/s).
//   256 rows (more than 128 on average; prefill): 64 KB of LDS writes and 192 KB of reads a step
//   against 2048 cycles of its MFMAs, and two barriers: matrix units 41-45 % busy at 2.0-2.2 GHz
//   (8 experts of 4096 / 14336 with 4096 tokens of 2: gate/up 1.01 ms with E8M0 scales and
//   1.07 ms with fp32 ones, down 0.52 ms; one dense expert of 8192 rows, 14336 -> 4096 2460-2600
//   and 2370-2450 TFLOP/s).
//   128 rows: between the two, 85 flop per loaded byte, three stages.
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
  int R, E, N, K;
  const int32_t* offsets;  // nullable: one expert holds all R rows
  const int32_t* table;    // nullable with few experts (RowTiles)
  bf16* y;
  uint8_t* hq;
  void* hs;
  f32x4* partial;  // slots of partial sums (s_max > 1)
  int n_tiles, group_n, s_max;
};

__device__ inline i32x8 join(const u32x4& a, const u32x4& b) {
  return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3],
               (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
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
__device__ inline f32x4 mma_zero(const i32x8& w, const i32x8& x, uint32_t sw, uint32_t sx) {
  f32x4 p = f32x4{0.f, 0.f, 0.f, 0.f};
  mma_e8m0(p, w, x, sw, sx);
  return p;
}
// An fp32 scale as 2^(e - 127) * m: its exponent byte e, kept within 1 and 253 so that 2^(127 - e)
// is a normal number, and m, which is exact: 1 <= |m| < 4, less for a subnormal scale (an infinity
// or a NaN stays one).
__device__ inline uint32_t scale_byte(uint32_t bits) {
  return min(max((bits >> 23) & 255u, 1u), 253u);
}
__device__ inline float scale_rest(uint32_t bits) {
  return __uint_as_float(bits) * __uint_as_float((254u - scale_byte(bits)) << 23);
}
__device__ inline void add_scaled(f32x4& acc, const f32x4& p, float s) {
#pragma unroll
  for (int q = 0; q < 4; ++q) acc[q] = fmaf(p[q], s, acc[q]);
}

// ---------------------------------------------------------------------------------------
// few tiles
// ---------------------------------------------------------------------------------------
// A product whose column tiles are too few for the 256 CUs (a shared expert and a few tokens) is
// bound by latency: 16 NT columns per block, every wave of the eight takes each eighth step of
// the reduction with its weight and row fragments loaded straight into registers, D steps ahead,
// and the sums are added through LDS in wave order.  Each block reads all of its rows, so more rows
// take more columns per block.  LIVE: 16-row tiles that hold rows.
constexpr int kSplitRows = 64, kSplitWaves = 8;

template <bool E8M0, int NT, int LIVE, int D>
__device__ inline void split_body(const Fp8Kern& a, const RowTile& rt, int rows, int nt,
                                  f32x4* part) {
  constexpr int ES = E8M0 ? 1 : 4;
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane & 15, g = lane >> 4;
  const int n0 = nt * 16 * NT, KB = a.K / kScaleBlock;
  const auto rw = buffer_rsrc(uniform_u64(a.b0 + ((int64_t)rt.e * a.N + n0) * a.K));
  const auto rx = buffer_rsrc(uniform_u64(a.xq + (int64_t)rt.begin * a.K));
  const auto rws = buffer_rsrc(uniform_u64(
      static_cast<const char*>(a.b0s) +
      ((int64_t)rt.e * (a.N / kScaleBlock) + n0 / kScaleBlock) * KB * ES));
  const auto rxs =
      buffer_rsrc(uniform_u64(static_cast<const char*>(a.xs) + (int64_t)rt.begin * KB * ES));
  uint32_t vw[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) vw[j] = (uint32_t)(j * 16 + c) * (uint32_t)a.K + g * 16;
  uint32_t vx[LIVE], vs[LIVE];
#pragma unroll
  for (int i = 0; i < LIVE; ++i) {
    const uint32_t row = min(i * 16 + c, rows - 1);
    vx[i] = row * (uint32_t)a.K + g * 16;
    vs[i] = row * (uint32_t)(KB * ES);
  }
  struct Step {
    u32x4 w[NT][2], x[LIVE][2];
    uint32_t ws, xs[LIVE];
  };
  auto scale_at = [&](const __amdgpu_buffer_rsrc_t& r, uint32_t voff, int kb) -> uint32_t {
    if constexpr (E8M0)
      return __builtin_amdgcn_raw_buffer_load_b8(r, voff, kb, 0);
    else
      return __builtin_amdgcn_raw_buffer_load_b32(r, voff, kb * 4, 0);
  };
  auto load = [&](Step& s, int t) {
    const int kb = wave + t * kSplitWaves;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        s.w[j][h] =
            __builtin_amdgcn_raw_buffer_load_b128(rw, vw[j], kb * kScaleBlock + h * 64, 2);
#pragma unroll
    for (int i = 0; i < LIVE; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        s.x[i][h] = __builtin_amdgcn_raw_buffer_load_b128(rx, vx[i], kb * kScaleBlock + h * 64, 0);
    s.ws = scale_at(rws, 0, kb);
#pragma unroll
    for (int i = 0; i < LIVE; ++i) s.xs[i] = scale_at(rxs, vs[i], kb);
  };
  f32x4 acc[LIVE][NT];
#pragma unroll
  for (int i = 0; i < LIVE; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](const Step& s) {
#pragma unroll
    for (int i = 0; i < LIVE; ++i) {
      const i32x8 x = join(s.x[i][0], s.x[i][1]);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const i32x8 w = join(s.w[j][0], s.w[j][1]);
        if constexpr (E8M0)
          mma_e8m0(acc[i][j], w, x, s.ws, s.xs[i]);
        else
          add_scaled(acc[i][j], mma_zero(w, x, scale_byte(s.ws), scale_byte(s.xs[i])),
                     scale_rest(s.ws) * scale_rest(s.xs[i]));
      }
    }
  };
  const int steps = (KB - wave + kSplitWaves - 1) / kSplitWaves;  // 0 past a short reduction
  Step ring[D];
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (d < steps) load(ring[d], d);
  for (int t = 0; t < steps; t += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      // keep the order: the loads of a slot right behind its last use, D steps ahead
      __builtin_amdgcn_sched_barrier(0);
      if (t + d < steps) multiply(ring[d]);
      if (t + d + D < steps) load(ring[d], t + d + D);
    }
  }
  constexpr int TILES = LIVE * NT;
#pragma unroll
  for (int i = 0; i < TILES; ++i) part[(wave * TILES + i) * kWave + lane] = acc[i / NT][i % NT];
  __syncthreads();
  if (wave < TILES) {
    const int i = wave / NT, j = wave % NT;
    f32x4 v = part[wave * kWave + lane];
#pragma unroll
    for (int w = 1; w < kSplitWaves; ++w) {
      const f32x4 u = part[(w * TILES + wave) * kWave + lane];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] += u[q];
    }
    typedef bf16 bf16x4 __attribute__((ext_vector_type(4)));
    if (i * 16 + c < rows)
      *reinterpret_cast<bf16x4*>(a.y + (int64_t)(rt.begin + i * 16 + c) * a.N + n0 + j * 16 +
                                 4 * g) =
          bf16x4{(bf16)v[0], (bf16)v[1], (bf16)v[2], (bf16)v[3]};
  }
}

template <bool E8M0, int NT>
__global__ void __launch_bounds__(512) split_kernel(const Fp8Kern a) {
  __shared__ f32x4 part[kSplitWaves * (kSplitRows / 16) * NT * kWave];
  TileWork w;
  if (!tile_work(RowTiles(a.offsets, a.table, a.E, a.R, kSplitRows), a.n_tiles, a.group_n, 1,
                 blockIdx.x >> 3, &w))
    return;
  const RowTile rt = w.rt;
  const int nt = w.nt;
  const int rows = min(rt.end - rt.begin, kSplitRows);
  if (rows <= 16)
    split_body<E8M0, NT, 1, 4>(a, rt, rows, nt, part);
  else if (rows <= 32)
    split_body<E8M0, NT, 2, 3>(a, rt, rows, nt, part);
  else
    split_body<E8M0, NT, 4, NT == 1 ? 3 : 2>(a, rt, rows, nt, part);
}

// ---------------------------------------------------------------------------------------
// tiles through LDS
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
  static constexpr int kScaleBytes = (kScaleWords * 4 + 255) / 256 * 256;
  // rings, two buffers of scales, the rows' offsets, the word that asks for exact scales
  static constexpr int kLds = kRing + 2 * kScaleBytes + BM * 4 + 16;
  static_assert(kLds <= 160 * 1024, "LDS of one CU");
};

typedef __attribute__((address_space(3))) uint32_t lds_u32;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) f32x4 lds_f32x4;

// A block fills its CU's LDS and works through its share of the tiles.  While the outputs of one
// tile leave through the activations' part of the LDS, the first weight stages of the next
// arrive in theirs.
template <int BM, bool SWIGLU, bool E8M0>
__device__ __attribute__((always_inline)) inline void fp8_body(
    const Fp8Kern& a, lds_char* __restrict__ a0, lds_char* __restrict__ a1,
    lds_char* __restrict__ a2, lds_char* __restrict__ b0, lds_char* __restrict__ b1,
    lds_char* __restrict__ b2, lds_u32* __restrict__ s0, lds_u32* __restrict__ s1,
    lds_u32* __restrict__ row_offset, lds_u32* __restrict__ exact_word) {
  using P = Fp8Tile<BM>;
  constexpr int S = P::kStages, MT = BM / 32, NT = 4;
  constexpr int BN = SWIGLU ? 128 : 256;
  constexpr int nA = BM / 32, nB = 8;  // direct loads per stage and issuing wave
  constexpr int ES = E8M0 ? 1 : 4;     // bytes of a scale
  // Few rows per expert: each weight line is read by one tile, and the non-temporal hint keeps
  // it from displacing the activation rows (decode experts 1853 -> 1735 us).
  constexpr bool kStreamW = BM <= 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave >> 2, wn = wave & 3;
  const int KB = a.K / kScaleBlock;
  const bool issuer = wave >= 4, scaler = wave < BM / 64;
  const int dslot = wave & 3;

  auto buf_a = [&](auto I) -> lds_char* {
    constexpr int j = decltype(I)::value % S;
    return j == 0 ? a0 : j == 1 ? a1 : a2;
  };
  auto buf_b = [&](auto I) -> lds_char* {
    constexpr int j = decltype(I)::value % S;
    return j == 0 ? b0 : j == 1 ? b1 : b2;
  };

  const RowTiles row_tiles(a.offsets, a.table, a.E, a.R, BM);
  TileWork w;
  int work = blockIdx.x >> 3;
  if (!tile_work(row_tiles, a.n_tiles, a.group_n, a.s_max, work, &w)) return;

  // Direct loads: one covers eight rows of 128 bytes; issuing wave d fills blocks 4 i + d.  The
  // rows of blocks i and i + 1 are 32 apart, which leaves the lane's piece the same: one lane
  // offset and a scalar for each i (weights; those past N, the upper half of a last column tile,
  // read the lower half again).
  auto direct_row = [&] { return dslot * 8 + (tile_thread() & (kWave - 1)) / 8; };
  auto piece_of = [&](int dr) {
    return (uint32_t)(((tile_thread() & 7) ^ ((dr >> 1) & 7)) * 16);
  };
  const int dr0 = direct_row();
  const uint32_t vb = (uint32_t)dr0 * (uint32_t)a.K + piece_of(dr0);
  // the weights' side of a tile
  struct Weights {
    uint64_t b, b2;
    int k_first, steps;  // the steps of the reduction it takes: all of them, or one piece
  };
  auto weights_of = [&](const TileWork& t) {
    Weights r;
    const int64_t row0 = (int64_t)t.rt.e * a.N + t.nt * BN;
    r.b = uniform_u64(a.b0 + row0 * a.K);
    r.b2 = SWIGLU ? uniform_u64(a.b1 + row0 * a.K)
                  : r.b + (t.nt * BN + 128 < a.N ? (uint64_t)128 * a.K : 0);
    r.k_first = t.piece * KB / t.pieces;
    r.steps = (t.piece + 1) * KB / t.pieces - r.k_first;
    return r;
  };
  auto dma_b = [&](const Weights& r, int kb, lds_char* bbuf) {
    if (!issuer) return;
    const uint32_t koff = (uint32_t)(r.k_first + min(kb, r.steps - 1)) * kScaleBlock;
#pragma unroll
    for (int i = 0; i < nB; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer_rsrc(i < 4 ? r.b : r.b2),
                                               bbuf + (i * 4 + dslot) * 1024, 16, vb,
                                               koff + (uint32_t)(i & 3) * 32u * (uint32_t)a.K, 0,
                                               kStreamW ? 2 : 0);
  };
  // The rows' side.  Gathered rows (gate and up only) have an offset each, kept in LDS (registers
  // are short), else they lie one behind the other.  Rows past the expert's get offsets past
  // the resource's end: they load as zeros, from nowhere.  Thread t < BM looks after row t: its
  // source is asked for (row_source) well before its offset is needed (rows_of).
  int src = 0;
  uint32_t vxs = 0;
  uint64_t base_a = 0, base_xs = 0;
  auto row_source = [&](const TileWork& t) {
    if (SWIGLU && a.src && scaler) src = a.src[min(t.rt.begin + tile_thread(), t.rt.end - 1)];
  };
  auto rows_of = [&](const TileWork& t) {
    const bool gather = SWIGLU && a.src;
    base_a = uniform_u64(gather ? a.xq : a.xq + (int64_t)t.rt.begin * a.K);
    // (rows of a tile, or all gathered rows, lie within 2^31 bytes of scales)
    base_xs = uniform_u64(static_cast<const char*>(a.xs) +
                          (gather ? 0 : (int64_t)t.rt.begin * KB * ES));
    const int row_t = tile_thread();
    const int row = gather ? min(max(src, 0), a.x_rows - 1)
                           : min(row_t, t.rt.end - t.rt.begin - 1);
    vxs = (uint32_t)row * (uint32_t)(KB * ES);
    if (SWIGLU && scaler)
      row_offset[row_t] =
          row_t < t.rt.end - t.rt.begin ? (uint32_t)row * (uint32_t)a.K : 0x80000000u;
  };

  Weights wt = weights_of(w);
  row_source(w);
  unroll_steps<S>([&](auto I) { dma_b(wt, decltype(I)::value, buf_b(I)); });
  rows_of(w);
  if (!E8M0 && tile_thread() == 0) *exact_word = 0;
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // the rows' offsets
  if (issuer) __builtin_amdgcn_s_setprio(3);

  for (;;) {
    // (what the last tile left, in scalar registers again)
    base_a = uniform_u64(base_a);
    base_xs = uniform_u64(base_xs);
    wt.b = uniform_u64(wt.b);
    wt.b2 = uniform_u64(wt.b2);
    const int rows = w.rt.end - w.rt.begin, m_begin = w.rt.begin, nt = w.nt;
    const int tid = tile_thread(), c = tid & 15, g = (tid >> 4) & 3;
    auto dma_a = [&](int kb, lds_char* abuf) {
      if (!issuer) return;
      const uint32_t koff = (uint32_t)(wt.k_first + min(kb, wt.steps - 1)) * kScaleBlock;
      uint32_t va[nA];
      if constexpr (SWIGLU) {
        const int dr = direct_row();
        const uint32_t piece = piece_of(dr);
#pragma unroll
        for (int i = 0; i < nA; ++i) va[i] = row_offset[i * 32 + dr] + piece;
      }
#pragma unroll
      for (int i = 0; i < nA; ++i)
        if constexpr (SWIGLU)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer_rsrc(base_a),
                                                   abuf + (i * 4 + dslot) * 1024, 16, va[i],
                                                   koff, 0, 0);
        else
          __builtin_amdgcn_raw_ptr_buffer_load_lds(
              bounded_rsrc(base_a, (int64_t)min(rows, BM) * a.K), abuf + (i * 4 + dslot) * 1024,
              16, vb, koff + (uint32_t)i * 32u * (uint32_t)a.K, 0, 0);
    };
    // Scales: thread t < BM brings row t's, one step ahead in registers, one in LDS.  The second
    // block of weights: the up matrix, or the next 128 columns (the last column tile of an odd
    // count repeats its first).
    const int64_t wsi = ((int64_t)w.rt.e * (a.N / 128) + nt * (BN / 128)) * KB;
    const uint64_t base_ws0 = uniform_u64(static_cast<const char*>(a.b0s) + wsi * ES);
    const uint64_t base_ws1 = SWIGLU ? uniform_u64(static_cast<const char*>(a.b1s) + wsi * ES)
                                     : base_ws0 + (nt * BN + 128 < a.N ? (uint64_t)KB * ES : 0);
    uint32_t xs = 0, ws0 = 0, ws1 = 0;
    float largest = 0.0f;  // of the products of scales
    auto scale_at = [&](uint64_t base, uint32_t voff, int k) -> uint32_t {
      if constexpr (E8M0)
        return __builtin_amdgcn_raw_buffer_load_b8(buffer_rsrc(base), voff, k, 0);
      else
        return __builtin_amdgcn_raw_buffer_load_b32(buffer_rsrc(base), voff, k * 4, 0);
    };
    auto scale_load = [&](int kb) {
      if (!scaler) return;
      const int k = wt.k_first + min(kb, wt.steps - 1);
      xs = scale_at(base_xs, vxs, k);
      ws0 = scale_at(base_ws0, 0, k);
      ws1 = scale_at(base_ws1, 0, k);
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
        const float p0 = __uint_as_float(xs) * __uint_as_float(ws0);
        const float p1 = __uint_as_float(xs) * __uint_as_float(ws1);
        s[tid] = __float_as_uint(p0);
        s[BM + tid] = __float_as_uint(p1);
        largest = fmaxf(largest, fmaxf(fabsf(p0), fabsf(p1)));
      }
    };

    f32x4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    // 16-row tiles of this wave's band that hold rows
    const int band_rows = rows - wm * MT * 16;
    const int live = band_rows <= 0 ? 0 : min(MT, (band_rows + 15) / 16);  // uniform
    const int swz = (c >> 1) & 7;
    // a fragment's two pieces: byte offsets of the lane's row, row tiles and column tiles a
    // constant apart; with SwiGLU a wave's column tiles are two gate tiles and the up tiles of
    // the same columns
    const int slot0 = (g ^ swz) * 16, slot1 = ((g + 4) ^ swz) * 16;
    const int af0 = (wm * MT * 16 + c) * 128 + slot0, af1 = af0 - slot0 + slot1;
    const int bf0 = (wn * (SWIGLU ? 32 : 64) + c) * 128 + slot0, bf1 = bf0 - slot0 + slot1;
    auto frag = [&](const lds_char* buf, int o0, int o1, int rows_on) {
      const u32x4 lo = *reinterpret_cast<const lds_u32x4*>(buf + o0 + rows_on * 128);
      const u32x4 hi = *reinterpret_cast<const lds_u32x4*>(buf + o1 + rows_on * 128);
      return join(lo, hi);
    };
    auto b_rows_on = [](int j) { return SWIGLU ? (j / 2) * 128 + (j % 2) * 16 : j * 16; };
    const int s_row = wm * MT * 16 + c;
    // Multiply one stage.  The row fragments stream through a ring of three, each read two row
    // tiles ahead of its MFMAs; the reads are spread between the MFMAs.  LIVE: the band's
    // 16-row tiles that hold rows (compile-time; k_loop picks the copy).  fp32 scales: a row
    // tile's four products are added to its sums behind the next tile's MFMAs.
    auto compute = [&](const lds_char* abuf, const lds_char* bbuf, const lds_u32* s,
                       auto live_c, auto mid) {
      constexpr int LIVE = decltype(live_c)::value, RING = 3;
      if constexpr (LIVE == 0) mid();
      if constexpr (LIVE > 0) {
        i32x8 fa[RING], fb[NT];
        uint32_t sx[RING];
        auto ld_a = [&](int i) {
          fa[i % RING] = frag(abuf, af0, af1, i * 16);
          if constexpr (E8M0) sx[i % RING] = s[s_row + i * 16];
        };
        // fp32 scales: read at their row tile's MFMAs, used behind the next one's
        float sa[2], sb[2];
        auto ld_s = [&](int i) {
          sa[i & 1] = __uint_as_float(s[(SWIGLU ? 0 : (wn >> 1) * BM) + s_row + i * 16]);
          sb[i & 1] = SWIGLU ? __uint_as_float(s[BM + s_row + i * 16]) : sa[i & 1];
        };
        uint32_t w0 = 0, w1 = 0;
        if constexpr (E8M0) {
          w0 = s[BM + (SWIGLU ? 0 : wn >> 1)];
          w1 = SWIGLU ? s[BM + 1] : w0;
        }
        ld_a(0);
#pragma unroll
        for (int j = 0; j < NT; ++j) fb[j] = frag(bbuf, bf0, bf1, b_rows_on(j));
        if constexpr (LIVE > 1) ld_a(1);
        if constexpr (!SWIGLU) mid();
        f32x4 p[2][NT];
        unroll_steps<LIVE>([&](auto I) {
          constexpr int i = decltype(I)::value;
          if constexpr (i + 2 < LIVE) ld_a(i + 2);
          if constexpr (!E8M0) ld_s(i);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            if constexpr (E8M0) {
              mma_e8m0(acc[i][j], fb[j], fa[i % RING], j < 2 ? w0 : w1, sx[i % RING]);
            } else {
              p[i & 1][j] = mma_zero(fb[j], fa[i % RING]);
              if constexpr (i > 0)
                add_scaled(acc[i - 1][j], p[(i - 1) & 1][j],
                           j < 2 ? sa[(i - 1) & 1] : sb[(i - 1) & 1]);
            }
          }
          // gate and up release the weights behind the second row tile: its MFMAs cover the wait
          // (fp32 scales 1550 -> 1510 us over the experts' network; no gain without SwiGLU)
          if constexpr (SWIGLU && i == std::min(1, LIVE - 1)) mid();
          // the reads and the previous tile's additions between this tile's MFMAs (scaled ones
          // count as vector instructions)
          constexpr int R = (i + 2 < LIVE ? (E8M0 ? 3 : 2) : 0) + (E8M0 ? 0 : SWIGLU ? 2 : 1);
          unroll_steps<NT>([&](auto J) {
            constexpr int j = decltype(J)::value;
            __builtin_amdgcn_sched_group_barrier(E8M0 ? 0x002 : 0x008, 1, 0);
            if constexpr (R > j) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            if constexpr (!E8M0 && i > 0) __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
          });
        });
        if constexpr (!E8M0) {
#pragma unroll
          for (int j = 0; j < NT; ++j)
            add_scaled(acc[LIVE - 1][j], p[(LIVE - 1) & 1][j],
                       j < 2 ? sa[(LIVE - 1) & 1] : sb[(LIVE - 1) & 1]);
        }
      }
    };

    // Step k: stage k has landed (own loads waited for, then the barrier); the activations' stage
    // k + S - 1 goes out into the buffer step k - 1 finished with and, once every wave holds this
    // step's weight fragments, the weights' stage k + S into theirs.  The scales of step k + 1 go
    // to LDS and those of k + 2 are asked for.
    //
    // Loads a wave may leave in flight at the top of step k: those of the S - 2 later stages and
    // one more of weights; in the first steps, whose weights all went out before the first
    // activations, the later activations and a weight stage for each step made.
    auto wait = [&](auto N) {
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(decltype(N)::value)
                   : "memory");
    };
    constexpr int L = S % 2 == 0 ? S : 2 * S;  // the rings repeat
    auto step = [&](int k, auto I, auto live_c) {
      if (k >= wt.steps) return;
      constexpr int i = decltype(I)::value;
      if (i == 0 && k == 0)
        wait(IntC<(S - 2) * nA>{});
      else if (S == 3 && i == 1 && k == 1)
        wait(IntC<(S - 2) * nA + nB>{});
      else
        wait(IntC<(S - 2) * (nA + nB) + nB>{});
      dma_a(k + S - 1, buf_a(IntC<i + S - 1>{}));
      scale_put(i % 2 ? s0 : s1);
      scale_load(k + 2);
      compute(buf_a(I), buf_b(I), i % 2 ? s1 : s0, live_c, [&] {
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        dma_b(wt, k + S, buf_b(I));
      });
    };
    unroll_steps<S - 1>([&](auto I) { dma_a(decltype(I)::value, buf_a(I)); });
    scale_load(0);
    scale_put(s0);
    scale_load(1);
    // one copy of the loop per count of live row tiles, so that nothing is tested between MFMAs
    auto k_loop = [&](auto live_c) {
      for (int k = 0; k < wt.steps; k += L)
        unroll_steps<L>([&](auto I) { step(k + decltype(I)::value, I, live_c); });
    };
    unroll_steps<MT + 1>([&](auto V) {
      if (live == decltype(V)::value) k_loop(V);
    });
    if (!E8M0 && largest > 0x1.fffffep127f) *exact_word = 1;
    // drain the loads issued past the last stage; every wave is done with the rings
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");

    // A product of scales past fp32's largest number: the tile again, a stage at a time, with the
    // exponents in the instruction.
    if constexpr (!E8M0) {
      if (__builtin_expect(__builtin_amdgcn_readfirstlane(*exact_word), 0)) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int k = 0; k < wt.steps; ++k) {
          dma_b(wt, k, b0);
          dma_a(k, a0);
          scale_load(k);
          if (scaler) s0[tid] = xs;
          const uint32_t w0 = scale_at(SWIGLU || wn < 2 ? base_ws0 : base_ws1, 0, wt.k_first + k);
          const uint32_t w1 = SWIGLU ? scale_at(base_ws1, 0, wt.k_first + k) : w0;
          asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
          i32x8 fb[NT];
#pragma unroll
          for (int j = 0; j < NT; ++j) fb[j] = frag(b0, bf0, bf1, b_rows_on(j));
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            const i32x8 fa = frag(a0, af0, af1, i * 16);
            const uint32_t x = s0[s_row + i * 16];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              const uint32_t u = j < 2 ? w0 : w1;
              add_scaled(acc[i][j], mma_zero(fb[j], fa, scale_byte(u), scale_byte(x)),
                         scale_rest(u) * scale_rest(x));
            }
          }
          asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        }
      }
    }

    // the next tile's sources and first weights
    TileWork next;
    work += gridDim.x >> 3;
    const bool more = tile_work(row_tiles, a.n_tiles, a.group_n, a.s_max, work, &next);
    if (more) {
      wt = weights_of(next);
      row_source(next);
      unroll_steps<S>([&](auto I) { dma_b(wt, decltype(I)::value, buf_b(I)); });
    }

    // Epilogue through the activations' rings, in passes of IP row tiles of both bands: a lane
    // holds four consecutive columns of row c of each 16-row tile.  Row r of a pass has its
    // 16-byte piece p in slot p ^ (r & 15).
    constexpr int kRow = 512;  // 128 fp32 values of h, or 256 bf16 ones of y
    const int tid_e = tile_thread(), c_e = tid_e & 15, g_e = (tid_e >> 4) & 3;
    constexpr int IP = std::min(MT, S * P::kABytes / (32 * kRow));
    static_assert(IP >= 1, "one row tile of both bands fits");
    if (w.slot >= 0) {  // one piece of the reduction: its partial sums
      if constexpr (!SWIGLU) store_partial(a.partial + (int64_t)w.slot * (BM * 64), acc, live);
    } else {
#pragma unroll
      for (int i0 = 0; i0 < MT; i0 += IP) {
        if (i0) asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
        for (int ii = 0; ii < IP; ++ii) {
          if (i0 + ii >= MT) break;
          const int r = (wm * IP + ii) * 16 + c_e;
          lds_char* row = a0 + r * kRow;
          const f32x4(&v)[NT] = acc[i0 + ii];
          if constexpr (SWIGLU) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              f32x4 h;
#pragma unroll
              for (int q = 0; q < 4; ++q) h[q] = silu_f32(v[j][q]) * v[j + 2][q];
              *reinterpret_cast<lds_f32x4*>(row + (((wn * 8 + j * 4 + g_e) ^ (r & 15)) << 4)) = h;
            }
          } else {
            typedef bf16 bf16x4 __attribute__((ext_vector_type(4)));
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              const int b = (wn * 64 + j * 16 + 4 * g_e) * 2;
              *reinterpret_cast<__attribute__((address_space(3))) bf16x4*>(
                  row + (((b >> 4) ^ (r & 15)) << 4) + (b & 15)) =
                  bf16x4{(bf16)v[j][0], (bf16)v[j][1], (bf16)v[j][2], (bf16)v[j][3]};
            }
          }
        }
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        // staged row r of the pass is row at(r) of the tile
        auto at = [&](int r) {
          return ((r / (IP * 16)) * MT + i0) * 16 + r % (IP * 16);
        };
        auto in_tile = [&](int r) {
          return (i0 + (r / 16) % IP) < MT && at(r) < min(rows, BM);
        };
        if constexpr (SWIGLU) {
          // eight lanes per row, each four pieces of four columns
          const int sub = tid_e & 7;
          for (int r = tid_e / 8; r < 32 * IP; r += 64) {
            if (!in_tile(r)) continue;
            f32x4 v[4];
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              v[j] = *reinterpret_cast<const lds_f32x4*>(
                  a0 + r * kRow + (((j * 8 + sub) ^ (r & 15)) << 4));
#pragma unroll
              for (int q = 0; q < 4; ++q) m = max(m, abs_bits(v[j][q]));
            }
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, 8));
            const bool finite = m < kInfBits;
            const int ex = finite ? scale_exponent(m) : 0;
            const float k = inv_scale(ex);
            const int64_t row = m_begin + at(r);
            uint8_t* dst = a.hq + row * a.N + nt * 128 + sub * 4;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<uint32_t*>(dst + j * 32) =
                  finite ? pack_e4m3(v[j][0] * k, v[j][1] * k, v[j][2] * k, v[j][3] * k) : kNan4;
            if (sub == 0)
              store_scale(a.hs, row * (a.N / 128) + nt, E8M0 ? kScaleE8M0 : kScaleF32, ex,
                          finite);
          }
        } else {
          for (int q = tid_e; q < 32 * IP * 32; q += 512) {
            const int r = q / 32, p = q % 32, col = nt * 256 + p * 8;
            if (!in_tile(r) || col >= a.N) continue;
            *reinterpret_cast<u32x4*>(a.y + (int64_t)(m_begin + at(r)) * a.N + col) =
                *reinterpret_cast<const lds_u32x4*>(a0 + r * kRow + ((p ^ (r & 15)) << 4));
          }
        }
      }
    }
    if (!more) return;
    w = next;
    rows_of(w);
    // every wave has read the staged rows, and the offsets of the next ones are there
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (!E8M0 && tile_thread() == 0) *exact_word = 0;  // (read by all, set behind the next loop)
  }
}

// BM: the tile height of the table.
template <int BM, bool SWIGLU, bool E8M0>
__global__ void __launch_bounds__(512) fp8_kernel(const Fp8Kern a) {
  extern __shared__ __attribute__((aligned(1024))) char smem_dyn[];
  using P = Fp8Tile<BM>;
  constexpr int A = P::kABytes, B = P::kBBytes;
  lds_char* base = (lds_char*)smem_dyn;
  lds_char* b = base + P::kStages * A;
  lds_u32* s = reinterpret_cast<lds_u32*>(base + P::kRing);
  // a third buffer exists only where the ring has three stages
  fp8_body<BM, SWIGLU, E8M0>(a, base, base + A, base + (P::kStages > 2 ? 2 * A : 0), b, b + B,
                             b + (P::kStages > 2 ? 2 * B : 0), s, s + P::kScaleBytes / 4,
                             s + P::kScaleBytes / 2, s + P::kScaleBytes / 2 + BM);
}

// ---------------------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------------------
// Row-tile heights by rows per expert (256 experts of 2048 x 2048, E8M0): 64 against 128 at 31 rows
// 206 and 210 us, at 48 rows 230 and 218; 128 against 256 at 100 rows 246 and 253 us, at 160 rows
// 353 and 287.
GroupPlan fp8_plan(int64_t R, int64_t E) {
  GroupPlan p;
  p.bm = R <= 32 * E ? 64 : R <= 128 * E ? 128 : 256;
  p.m_max = (R + E * (p.bm - 1)) / p.bm;
  return p;
}

GroupSplit group_split(const GroupPlan& p, int64_t E, int64_t columns, int64_t steps,
                       int64_t least) {
  GroupSplit g = {1, 0};
  const int64_t n_tiles = (columns + 255) / 256, tiles = p.m_max * n_tiles;
  // Worth a second launch and the partial sums' way through memory when a tile is long (at least
  // `least` steps) and the last partial round is a good part of all rounds.  That round is known
  // for a single expert's rows, and where all tiles are fewer than the CUs.  One expert's last
  // round that is whole, or too full to cut any tile in two, has nothing to split (8192 rows, 8192
  // -> 4096 220 us with the launch, 215 without; 2048 rows, 4096 -> 5120, 160 tiles, 59 and 56).
  const int64_t last = E == 1 || tiles < kSplitCUs ? tiles % kSplitCUs : kSplitCUs;
  if (E == 1 && (last == 0 || last > kSplitCUs / 2)) return g;
  // Few tiles in the last round leave most CUs idle through it: split from 32 steps.  Whole against
  // split, dgrad: 256 rows, 4096 -> 2048 (8 tiles of 64 steps) 77 and 39 us; 1024 rows, 2048 ->
  // 5120 (80 tiles of 32) 45.4 and 44.5; 4096 rows, 2048 -> 2048 (128 tiles of 32) 46.2 and 53.6;
  // 4096 rows, 4096 -> 5120 (320 tiles) 173 and 148; 8 experts, 1024 rows, 2048 -> 2048 (at most
  // 88 tiles) 34.5 and 32.4, 2048 -> 5120 (at most 220) 35.6 and 38.7.  8-bit, one expert, 256
  // rows, 4096 -> 2048 53 and 35, 1024 rows, 4096 -> 5120 (80 tiles) 55 and 48.
  if (last <= 3 * kSplitCUs / 8) least = std::min<int64_t>(least, 32);
  if (steps >= least && tiles > 0 && tiles < 8 * kSplitCUs) {
    g.s_max = (int)std::min<int64_t>(8, steps / 8);
    g.bytes = std::min<int64_t>(kSplitCUs, tiles * g.s_max) * p.bm * 256 * 4;
  }
  return g;
}

// (8192 rows, 8 experts, K -> 4096, E8M0, split against whole: K = 4096 169 and 168 us, 6144 254
// and 267, 7168 266 and 283, 14336 496 and 570; 2048 rows, K = 4096 61 and 57)
GroupSplit fp8_split(int64_t R, int64_t E, int64_t N, int64_t K) {
  return group_split(fp8_plan(R, E), E, N, K / kScaleBlock, 48);
}

// Bound on the blocks that hold a tile, of m_max x n_tiles, rounded up to the 8 XCDs' shares.
static unsigned grid_of(int64_t m_max, int64_t n_tiles) {
  return (unsigned)((m_max * n_tiles + 7) / 8 * 8);
}

template <bool E8M0, int NT>
static hipError_t run_split(Fp8Kern k, int64_t m_max, hipStream_t s) {
  k.n_tiles = k.group_n = k.N / (16 * NT);
  split_kernel<E8M0, NT><<<grid_of(m_max, k.n_tiles), 512, 0, s>>>(k);
  return hipGetLastError();
}

template <int BM, bool SWIGLU, bool E8M0>
static hipError_t run_tiles(Fp8Kern k, int64_t m_max, hipStream_t s) {
  constexpr int BN = SWIGLU ? 128 : 256;
  k.n_tiles = (k.N + BN - 1) / BN;
  // tiles are cut along the reduction where the plan has room for their partial sums
  const GroupSplit split = fp8_split(k.R, k.E, k.N, k.K);
  k.s_max = SWIGLU ? 1 : split.s_max;
  if (k.s_max > 1 && !k.partial) return hipErrorInvalidValue;
  // few rows: the activations are what tiles share, so an expert's column tiles run together
  // (decode experts 1735 -> 1726 us)
  k.group_n = BM <= 64 ? k.n_tiles : std::min(k.n_tiles, 8);
  constexpr int lds = Fp8Tile<BM>::kLds;
  hipError_t e = hipFuncSetAttribute((const void*)fp8_kernel<BM, SWIGLU, E8M0>,
                                     hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return e;
  // one block per CU at most (a multiple of the 8 XCDs)
  const unsigned grid = std::min<unsigned>(
      grid_of(m_max, k.n_tiles) + (k.s_max > 1 ? kSplitCUs : 0), kSplitCUs);
  fp8_kernel<BM, SWIGLU, E8M0><<<grid, 512, lds, s>>>(k);
  if ((e = hipGetLastError()) != hipSuccess || k.s_max < 2) return e;
  partial_sum_kernel<BM><<<dim3(kSplitCUs, 8 * (BM / 32) / 4), 256, 0, s>>>(
      k.partial, k.offsets, k.table, k.E, k.R, k.n_tiles, k.group_n, k.s_max, k.N, k.y);
  return hipGetLastError();
}

template <bool SWIGLU, bool E8M0>
static hipError_t run_fp8(const Fp8Kern& k, const GroupPlan& p, hipStream_t s) {
  if constexpr (!SWIGLU) {
    // Few tiles and at most 64 rows per expert on average; every block reads all its rows, so
    // more rows need fewer columns (one expert, K = 4096, E8M0, split against tiles: 16 rows N =
    // 16384 21 and 25 us, N = 28672 37 and 29; 32 rows N = 16384 26 and 27; 64 rows N = 16384
    // 36 and 27; K = 2048, fp32 scales, 64 rows N = 7168 11.5 and 17.8).
    const int64_t m64 = (k.R + (int64_t)k.E * (kSplitRows - 1)) / kSplitRows;
    const int64_t most = k.R > 32 * (int64_t)k.E ? 96 : 192;
    if (!group_needs_table(k.E) && k.R <= kSplitRows * (int64_t)k.E && m64 * (k.N / 128) < most)
      // 16 columns a block while 32 would leave CUs idle (64 rows: N = 4096 16.4 against 18.3 us,
      // N = 7168 18.2 against 11.5)
      return m64 * (k.N / 32) < 192 ? run_split<E8M0, 1>(k, m64, s)
                                    : run_split<E8M0, 2>(k, m64, s);
  }
  if (p.bm == 64) return run_tiles<64, SWIGLU, E8M0>(k, p.m_max, s);
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
  k.E = (int)a.E;
  k.N = (int)a.N;
  k.K = (int)a.K;
  k.offsets = a.offsets;
  k.table = group_needs_table(a.E) ? a.table : nullptr;
  k.y = (bf16*)a.y;
  k.hq = (uint8_t*)a.hq;
  k.hs = a.h_scale;
  k.partial = (f32x4*)a.partial;
  k.n_tiles = k.group_n = 0;
  k.s_max = 1;
  const bool e8m0 = a.scale_type == kScaleE8M0;
  if (a.b1) return e8m0 ? run_fp8<true, true>(k, p, s) : run_fp8<true, false>(k, p, s);
  return e8m0 ? run_fp8<false, true>(k, p, s) : run_fp8<false, false>(k, p, s);
}

}  // namespace moe
