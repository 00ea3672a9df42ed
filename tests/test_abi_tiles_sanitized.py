"""The host code that tells a linear layer's tiles and sets the few-token layer's waits under
AddressSanitizer and UndefinedBehaviorSanitizer, in a child process with the sanitizers' copy of the
library.  No kernel is launched."""
import os
import subprocess
import sys

import pytest

from routing_expert_ffn_router_amd import _build
from test_abi_sanitized import _fresh, _runtime

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import ctypes, itertools, sys
sys.path.insert(0, ROOT)
import routing_expert_ffn_router_amd as moe
lib = moe.load_library(LIB)
tiles = (ctypes.c_int64 * 3)()
n = ok = 0
for rows, E, N, K in itertools.product([-(1 << 62), -1, 0, 1, 16, 63, 64, 65, 1000, 1 << 16, (1 << 20) + 7,
                                        (1 << 31) - 1, 1 << 31, (1 << 62) + 5],
                                       [-1, 0, 1, 8, 64, 65, 1024, 1025],
                                       [-128, 0, 100, 128, 384, 4096, 1 << 20, (1 << 20) + 128],
                                       [0, 128, 4096, 1 << 20, 1 << 40]):
    for dt in (-1, 0, 1, 2):
        g = ctypes.byref(moe.MoeGroupShape(rows, E, N, K, dt, 0))
        tiles[0] = tiles[1] = tiles[2] = -9
        rc = lib.moe_linear_tiles(g, tiles)
        if rc == 0:
            assert tiles[0] in (64, 128, 256) and tiles[1] in (32, 64, 256) and 1 <= tiles[2] <= 8
            assert lib.moe_linear_workspace_size(g) > 0
            ok += 1
        else:
            assert list(tiles) == [-9] * 3 and lib.moe_linear_workspace_size(g) == 0
        assert lib.moe_linear_tiles(g, None) != 0
        n += 1
assert lib.moe_linear_tiles(None, tiles) != 0
for polls in (0, 1, (1 << 31) - 1, -1, -(1 << 31)):
    lib.moe_few_wait_polls(polls)
assert lib.moe_few_wait_polls(-1) == (1 << 31) - 1
print("calls", n, ok)
"""


def test_host_code_under_the_sanitizers():
    rt = _runtime()
    if rt is None:
        pytest.skip("no AddressSanitizer runtime in this ROCm install")
    lib = _build.LIB_SANITIZED
    if not _fresh(lib):
        _build.build(sanitize=True)
    code = CHILD.replace("ROOT", repr(ROOT)).replace("load_library(LIB)", f"load_library({lib!r})")
    env = dict(os.environ, LD_PRELOAD=rt, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, (r.stdout[-2000:], r.stderr[-4000:])
    words = r.stdout.split()
    assert words[0] == "calls" and int(words[2]) > 100
