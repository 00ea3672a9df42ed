"""The walk of the few-token layer's waves through their units, on the host: every unit of every item is
taken once, and no place that is looked up lies past the list of chosen experts."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "routing_expert_ffn_router_amd", "csrc")

DRIVER = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "few_walk.h"
using namespace moe;

static long walks = 0;
#define REQUIRE(c)                                                                            \
  if (!(c)) {                                                                                 \
    std::printf("%s: across %d down %d experts %d per_k %d tiles %d chunks %d stride %d first %d wave %d\n", \
                #c, ACROSS, DOWN, experts, per_k, tiles, chunks, stride, first, wave);        \
    std::exit(1);                                                                             \
  }

// All items of one launch: `blocks` runs of items, each worked through by eight waves.
template <bool ACROSS, bool DOWN>
void launch(int experts, int per_k, int tiles, int chunks, int blocks) {
  const int units = DOWN ? experts * per_k : per_k;
  const int items = DOWN ? tiles * chunks : experts * tiles;
  const int stride = items < blocks ? items : blocks;
  // the unit counts of one column tile: [expert][unit], the same for all tiles
  std::vector<int> taken((size_t)tiles * experts * per_k, 0);
  for (int first = 0; first < stride; ++first)
    for (int wave = 0; wave < kWaves; ++wave) {
      if (ACROSS && wave) break;  // all waves go the same way
      const FewWalk<ACROSS, DOWN> w = {items, stride, tiles, per_k, units, chunks, wave};
      auto p = w.start(first);
      int ended = first - stride;
      for (;;) {
        const bool live = w.next_run(p, [&](int q) {
          REQUIRE(q == ended);
          ended += stride;
        });
        const int at = w.entry(p, live);
        REQUIRE(at >= 0 && at < experts);
        if (!live) break;
        REQUIRE(p.run > 0 && p.run <= p.left && p.q >= 0 && p.q < items);
        for (int i = 0; i < p.run; ++i) {
          const int k = p.k + i * w.kStep;
          REQUIRE(k >= 0 && k < per_k);
          ++taken[((size_t)(p.q % tiles) * experts + at) * per_k + k];
        }
      }
      REQUIRE(ended >= items);  // every item of the run has ended, with units or without
      ++walks;
    }
  const int wave = -1, first = -1;
  for (int n : taken) REQUIRE(n == 1);
}

int main() {
  const int experts[] = {1, 2, 3, 7, 16, 61}, per_k[] = {1, 2, 3, 4, 7, 8, 9, 11, 16, 56, 112};
  const int tiles[] = {1, 2, 8, 23}, chunks[] = {1, 2, 3, 5, 8, 31, 32}, blocks[] = {1, 3, 256};
  for (int e : experts)
    for (int k : per_k)
      for (int t : tiles)
        for (int b : blocks) {
          launch<false, false>(e, k, t, 1, b);
          launch<true, false>(e, k, t, 1, b);
          for (int c : chunks) {
            launch<false, true>(e, k, t, c, b);
            launch<true, true>(e, k, t, c, b);
          }
        }
  std::printf("walks %ld\n", walks);
}
"""


def test_every_unit_once_and_no_expert_past_the_list(tmp_path):
    src, exe = tmp_path / "walk.cpp", tmp_path / "walk"
    src.write_text(DRIVER)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-Wno-unknown-pragmas",
                    "-fsanitize=undefined", "-fno-sanitize-recover=undefined", "-I", CSRC, str(src),
                    "-o", str(exe)], check=True, timeout=120)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.startswith("walks ")
