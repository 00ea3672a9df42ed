// The order in which a wave of few_kernel works through the units of its items, and the chosen
// expert that each unit belongs to.  Plain arithmetic, so that it runs on the host as well.
#pragma once

#ifdef __HIPCC__
#include <hip/hip_runtime.h>
#define MOE_WALK __host__ __device__ __attribute__((always_inline)) inline
#else
#define MOE_WALK inline
#endif

#include <algorithm>
#include <cstdint>

namespace moe {

constexpr int kWaves = 8;  // of a block

// The same in all lanes, which the compiler does not know of a quotient: kept in a scalar register.
MOE_WALK int walk_uniform(int v) {
#ifdef __HIP_DEVICE_COMPILE__
  return __builtin_amdgcn_readfirstlane(v);
#else
  return v;
#endif
}

// Items first, first + stride, ... below `items`; an item is `tiles` column tiles of an expert's gate and
// up, or of a chunk of down's reduction over all chosen experts.  Each expert has per_k units of the
// reduction.  ACROSS: every wave goes through all units of an item; else every eighth, from its own
// number on (together the waves then read whole kilobytes of each row).
template <bool ACROSS, bool DOWN>
struct FewWalk {
  int items, stride, tiles, per_k;
  int units;   // of an item's whole reduction
  int chunks;  // of it
  int wave;
  static constexpr int kStep = ACROSS ? 1 : kWaves;

  // A place in the stream of units: item q, `left` units to go when the run began, unit k of the rows
  // of the at-th expert there; a run ends with the item or the expert.
  struct Place {
    int q, left, run, at, k;
  };
  MOE_WALK Place start(int first) const { return Place{first - stride, 0, 0, 0, 0}; }

  // how many units of an item this wave has, and the first
  MOE_WALK int item_units(int q, int* u0) const {
    int from = 0, len = units;
    if constexpr (DOWN) {  // (at most 2^24 units and 32 chunks)
      const uint32_t n = (uint32_t)q / (uint32_t)tiles;
      from = (int)(n * (uint32_t)units / (uint32_t)chunks);
      len = (int)((n + 1) * (uint32_t)units / (uint32_t)chunks) - from;
    }
    if constexpr (!ACROSS) {
      from += wave;
      len = (len > wave ? len - wave + kWaves - 1 : 0) / kWaves;
    }
    *u0 = walk_uniform(from);
    return walk_uniform(len);
  }

  // From the end of a run to the next one; false: no item has units any more.  done(q): item q ended.
  template <class Done>
  MOE_WALK bool next_run(Place& p, Done&& done) const {
    p.left -= p.run;
    p.k += p.run * kStep;
#pragma unroll 1
    while (p.left == 0) {
      done(p.q);
      p.q += stride;
      if (p.q >= items) return false;
      int u0;
      p.left = item_units(p.q, &u0);
      p.at = walk_uniform(
          (int)(DOWN ? (uint32_t)u0 / (uint32_t)per_k : (uint32_t)p.q / (uint32_t)tiles));
      p.k = DOWN ? u0 - p.at * per_k : u0;
    }
    if constexpr (DOWN) {
#pragma unroll 1
      while (p.k >= per_k) {
        p.k -= per_k;
        ++p.at;
      }
      const int here = (int)((uint32_t)(per_k - p.k + kStep - 1) / kStep);
      p.run = p.left < here ? p.left : here;
    } else {
      p.run = p.left;
    }
    return true;
  }

  // The entry of the list of chosen experts for a place; where next_run found no more units (`live`
  // false) the place may lie past the list, and the first entry stands in.
  MOE_WALK int entry(const Place& p, bool live) const { return live ? p.at : 0; }
};

}  // namespace moe
