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
__device__ inline uint64_t uniform_u64(const void* p) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
  return ((uint64_t)hi << 32) | lo;
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

// Tiles of rows grouped by expert.  With at most kScanExperts experts a wave finds its row tile
// from the offsets themselves, one expert per lane, which saves the launch that writes the tile
// table (about 2 us of its own and a gap before it); more experts take the table.
static_assert(kScanExperts <= kWave, "one expert per lane");

struct RowTile {
  int e, begin, end;  // expert, first row, end of the expert's rows
};

// Block -> (row tile, column tile): the tiles are dealt to the 8 XCDs (blocks go round them in
// turn) in contiguous shares of the tiles there are, so that a share's tiles keep their rows and
// weights in one L2.  table: launch_tile_table's, or null (E <= kScanExperts).  offsets null: one
// expert holds all R rows.  Offsets are clamped to [0, R].  False: no tile for this block.
__device__ inline bool group_tile(const int32_t* offsets, const int32_t* table, int E, int R,
                                  int bm, int n_tiles, int group_n, RowTile* rt, int* nt) {
  int m_tiles, row0 = 0, tiles = 0, inc = 0;
  if (table) {
    m_tiles = table[0];
  } else {
    const int l = lane_id();
    int row1 = 0;
    if (l < E) {
      row0 = offsets ? min(max(offsets[l], 0), R) : 0;
      row1 = offsets ? min(offsets[l + 1], R) : R;
    }
    tiles = (max(row1 - row0, 0) + bm - 1) / bm;
    inc = wave_inclusive_scan(tiles);
    m_tiles = __builtin_amdgcn_readlane(inc, kWave - 1);
  }
  const int total = m_tiles * n_tiles;
  const int xcd = blockIdx.x & 7, j = blockIdx.x >> 3, per = (total + 7) / 8;
  const int i = xcd * per + j;
  if (j >= per || i >= total) return false;
  int mt;
  dense_tile(i, m_tiles, n_tiles, group_n, &mt, nt);
  if (table) {
    rt->e = table[1 + 2 * mt];
    rt->begin = table[2 + 2 * mt];
  } else {
    rt->e = __builtin_ctzll(__ballot(mt < inc));
    rt->begin = __builtin_amdgcn_readlane(row0, rt->e) +
                (mt - (__builtin_amdgcn_readlane(inc, rt->e) -
                       __builtin_amdgcn_readlane(tiles, rt->e))) * bm;
  }
  rt->end = offsets ? min(offsets[rt->e + 1], R) : R;
  return true;
}

}  // namespace moe
