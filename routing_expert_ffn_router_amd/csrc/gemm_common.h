// Building blocks shared by the grouped GEMMs: buffer resources and direct buffer -> LDS loads,
// compile-time unrolling, the waits of the LDS rings and the order of the tiles.
#pragma once

#include <type_traits>
#include <utility>

#include "common.h"
#include "kernels.h"

namespace moe {

// silu(g) = g / (1 + e^-g) with the hardware reciprocal (about 1 ulp) instead of a correctly
// rounded division: the SwiGLU epilogue evaluates it for every output of the gate/up GEMM,
// and the division's ten instructions made that epilogue several percent of a tile.  For
// g < -88 the reciprocal of +inf gives -0.0 where the exact value is below 1e-36.
__device__ inline float silu_f32(float g) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g));
}

typedef __attribute__((address_space(3))) char lds_char;

// A wave-uniform 64-bit address, moved to scalar registers.
__device__ inline uint64_t uniform_u64(uint64_t a) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
  return ((uint64_t)hi << 32) | lo;
}
__device__ inline uint64_t uniform_u64(const void* p) {
  return uniform_u64(reinterpret_cast<uint64_t>(p));
}
// Raw buffer resource for byte offsets below 2^31 from a uniform base address.  Selecting
// between bases (scalar) rather than between descriptors keeps the descriptor in scalar
// registers; a descriptor the compiler cannot prove uniform turns every buffer load into a
// serialised per-lane loop.
__device__ inline __amdgpu_buffer_rsrc_t buffer_rsrc(uint64_t base) {
  constexpr int kFlags = 0x00020000;  // raw buffer, 32-bit data format (gfx9 family)
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(base), 0, 0x7fffffff,
                                           kFlags);
}

// A buffer resource over [base, base + bytes): loads past its end give zeros.  (Loads lie within
// 2^31 bytes of the base, so an end beyond that needs no exact value.)
__device__ inline __amdgpu_buffer_rsrc_t bounded_rsrc(uint64_t base, int64_t bytes) {
  const int n = (int)min(max(bytes, (int64_t)0), (int64_t)0x7fffffff);
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(base), 0, n, 0x00020000);
}

template <int N>
using IntC = std::integral_constant<int, N>;
// f(IntC<0>{}), ..., f(IntC<L-1>{}), with compile-time indices
template <class F, int... Is>
__device__ inline void unroll_steps_impl(F&& f, std::integer_sequence<int, Is...>) {
  (f(IntC<Is>{}), ...);
}
template <int L, class F>
__device__ inline void unroll_steps(F&& f) {
  unroll_steps_impl(f, std::make_integer_sequence<int, L>{});
}

// wait until at most N direct loads of this wave are outstanding, then block barrier
template <int N>
__device__ inline void wait_vm_barrier() {
  static_assert(N >= 0 && N < 64, "vmcnt immediate");
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(N) : "memory");
}

// (m-tile, n-tile) of dense tile number i: groups of m_tiles x group_n tiles, n fastest
// within a group; the last group holds the n_tiles mod group_n remaining n-tiles.
__device__ inline void dense_tile(int i, int m_tiles, int n_tiles, int group_n, int* mt,
                                  int* nt) {
  const int per_group = m_tiles * group_n, full = n_tiles / group_n;
  if (i < full * per_group) {
    const int grp = i / per_group, rem = i - grp * per_group;
    *mt = rem / group_n;
    *nt = grp * group_n + rem % group_n;
  } else {
    const int rem = i - full * per_group, gw = n_tiles - full * group_n;
    *mt = rem / gw;
    *nt = full * group_n + rem % gw;
  }
}

// The thread's index, opaque to the compiler: what a tile derives from it is computed again for
// each tile, not kept in registers around the loop over tiles.
__device__ inline int tile_thread() {
  int t = threadIdx.x;
  asm volatile("" : "+v"(t));
  return t;
}

// Tiles of rows grouped by expert.  With at most kScanExperts experts a wave finds its row tile
// from the offsets themselves, one expert per lane, which saves the launch that writes the tile
// table (about 2 us of its own and a gap before it); more experts take the table.
static_assert(kScanExperts <= kWave, "one expert per lane");

// A grouped product with few, long tiles: the tail split.  The t = m-tiles x n-tiles tiles (m-tiles
// counted on the device) are numbered densely, n fastest within groups of group_n n-tiles.
// The first floor(t / cus) * cus tiles run whole; the tail of t mod cus tiles, which would
// leave most CUs idle through a last partial round, is split along the reduction into
// S = min(s_max, cus / tail) pieces, each storing its tile of fp32 partial sums in a slot of
// its own for another launch to add in piece order (deterministic).  S < 2: nothing splits.
struct TailSplit {
  int tiles, whole, tail, pieces;
};
__device__ inline TailSplit tail_split_of(int m_tiles, int n_tiles, int s_max) {
  TailSplit p;
  p.tiles = m_tiles * n_tiles;
  p.whole = p.tiles / kSplitCUs * kSplitCUs;
  p.tail = p.tiles - p.whole;
  p.pieces = p.tail ? min(s_max, kSplitCUs / p.tail) : 1;
  if (p.pieces < 2) {
    p.whole = p.tiles;
    p.tail = 0;
    p.pieces = 1;
  }
  return p;
}

struct RowTile {
  int e, begin, end;  // expert, first row, end of the expert's rows
};
// What a block computes: a row tile and column tile, whole (slot < 0) or `piece` of `pieces` of its
// reduction, whose partial sums go to slot `slot`.
struct TileWork {
  RowTile rt;
  int nt, slot, piece, pieces;
};

// The row tiles of the experts, as a wave holds them: from the table, or one expert per lane.
struct RowTiles {
  const int32_t* offsets;  // nullable: one expert holds all R rows
  const int32_t* table;    // launch_tile_table's, or null (E <= kScanExperts)
  int R, bm, count;
  int row0, tiles, inc;  // lane's expert: first row, row tiles, row tiles up to and with it

  __device__ inline RowTiles(const int32_t* offsets_, const int32_t* table_, int E, int R_,
                             int bm_)
      : offsets(offsets_), table(table_), R(R_), bm(bm_), row0(0), tiles(0), inc(0) {
    if (table) {
      count = table[0];
    } else {
      const int l = lane_id();
      int row1 = 0;
      if (l < E) {  // offsets are clamped to [0, R]
        row0 = offsets ? min(max(offsets[l], 0), R) : 0;
        row1 = offsets ? min(offsets[l + 1], R) : R;
      }
      tiles = (max(row1 - row0, 0) + bm - 1) / bm;
      inc = wave_inclusive_scan(tiles);
      // at most GroupPlan::m_max, as the table: offsets that decrease would count rows twice, and
      // the slots of partial sums are laid out for m_max tiles
      count = min(__builtin_amdgcn_readlane(inc, kWave - 1),
                  (int)(((uint32_t)R + (uint32_t)(E * (bm - 1))) / (uint32_t)bm));
    }
  }
  __device__ inline RowTile at(int mt) const {
    RowTile t;
    if (table) {
      t.e = table[1 + 2 * mt];
      t.begin = table[2 + 2 * mt];
    } else {
      t.e = __builtin_ctzll(__ballot(mt < inc));
      t.begin = __builtin_amdgcn_readlane(row0, t.e) +
                (mt - (__builtin_amdgcn_readlane(inc, t.e) -
                       __builtin_amdgcn_readlane(tiles, t.e))) * bm;
    }
    t.end = offsets ? min(offsets[t.e + 1], R) : R;
    return t;
  }
};

// Work j of this block's XCD.  Blocks go round the 8 XCDs in turn; each XCD takes a contiguous
// share of the tiles there are, so that its tiles keep their rows and weights in one L2, then
// (s_max > 1) its share of the tail's pieces.  False: no such work, nor any after it.
__device__ inline bool tile_work(const RowTiles& rows, int n_tiles, int group_n, int s_max, int j,
                                 TileWork* w) {
  const int xcd = blockIdx.x & 7;
  TailSplit ts;
  if (s_max > 1) {
    ts = tail_split_of(rows.count, n_tiles, s_max);
  } else {
    ts.whole = rows.count * n_tiles;
    ts.tail = 0;
  }
  const int w8 = (ts.whole + 7) / 8;
  int tile;
  w->slot = -1;
  w->piece = 0;
  w->pieces = 1;
  if (j < w8 && xcd * w8 + j < ts.whole) {
    tile = xcd * w8 + j;
  } else {
    if (ts.tail == 0) return false;
    // (with a tail, the whole tiles are a multiple of the CUs: every XCD has w8 of them)
    const int all = ts.tail * ts.pieces, q8 = (all + 7) / 8, q = xcd * q8 + (j - w8);
    if (j < w8 || j - w8 >= q8 || q >= all) return false;
    w->piece = q / ts.tail;
    w->pieces = ts.pieces;
    const int i = q - w->piece * ts.tail;
    w->slot = i * ts.pieces + w->piece;
    tile = ts.whole + i;
  }
  int mt;
  dense_tile(tile, rows.count, n_tiles, group_n, &mt, &w->nt);
  w->rt = rows.at(mt);
  return true;
}

// Stores of partial sums and their sum, for tiles of eight waves as 2 x 4 whose wave (wm, wn)
// holds MT x NT tiles of 16 x 16, lane l holding row l % 16 and columns 4 (l / 16) .. + 3 of each:
// the slot keeps the registers as they are, 1 KB for each 16 x 16 tile of each wave.
template <int MT, int NT>
__device__ inline void store_partial(f32x4* slot, const f32x4 (&acc)[MT][NT], int live) {
  const int wave = threadIdx.x / kWave;
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    if (i >= live) break;
#pragma unroll
    for (int j = 0; j < NT; ++j)
      slot[((wave * MT + i) * NT + j) * kWave + lane_id()] = acc[i][j];
  }
}

// The slots' sum, rounded to bf16: one wave per (tail tile, wave, row tile i), grid (kSplitCUs, 8 *
// MT / 4), surplus blocks exit.  Bound by HBM and its launch (256 slots of 256 KB in 16-20 us).
template <int BM>
__global__ void __launch_bounds__(256)
partial_sum_kernel(const f32x4* __restrict__ acc, const int32_t* __restrict__ offsets,
                   const int32_t* __restrict__ table, int E, int R, int n_tiles, int group_n,
                   int s_max, int N, bf16* __restrict__ y) {
  constexpr int NT = 4, MT = BM / 32;
  const RowTiles rows(offsets, table, E, R, BM);
  const TailSplit ts = tail_split_of(rows.count, n_tiles, s_max);
  if ((int)blockIdx.x >= ts.tail) return;
  int mt, nt;
  dense_tile(ts.whole + blockIdx.x, rows.count, n_tiles, group_n, &mt, &nt);
  const RowTile rt = rows.at(mt);
  const int unit = blockIdx.y * 4 + threadIdx.x / kWave;  // wave * MT + i
  const int wave = unit / MT, i = unit - wave * MT;
  const int lane = lane_id(), row = ((wave >> 2) * MT + i) * 16 + (lane & 15);
  if (row - (lane & 15) >= min(rt.end - rt.begin, BM)) return;
  const bool stored = row < min(rt.end - rt.begin, BM);
  constexpr int kSlot = 8 * MT * NT * kWave;
  const f32x4* src = acc + (int64_t)blockIdx.x * ts.pieces * kSlot + unit * NT * kWave + lane;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int col = nt * 256 + (wave & 3) * 64 + j * 16;
    if (col >= N) break;
    f32x4 v = src[j * kWave];
    for (int p = 1; p < ts.pieces; ++p) {
      const f32x4 u = src[(int64_t)p * kSlot + j * kWave];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] += u[q];
    }
    typedef bf16 bf16x4 __attribute__((ext_vector_type(4)));
    if (stored)
      *reinterpret_cast<bf16x4*>(y + (int64_t)(rt.begin + row) * N + col + 4 * (lane >> 4)) =
          bf16x4{(bf16)v[0], (bf16)v[1], (bf16)v[2], (bf16)v[3]};
  }
}

}  // namespace moe
