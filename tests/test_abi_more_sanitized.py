"""The host code of the few-token layer, the linear layers and the clipping under AddressSanitizer and
UndefinedBehaviorSanitizer: extreme shapes through every host function, and arguments that fail
validation through every entry point, in a child process with the sanitizers' copy of the library.  No
kernel is launched."""
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
P, W = 1 << 40, 1 << 40  # never dereferenced: every call below fails validation first
big = [-(1 << 62), -1, 0, 1, 2, 16, 17, 127, 1000, (1 << 20) + 128, (1 << 31) - 1, 1 << 31, 1 << 40,
       (1 << 62) + 5]
n = 0
for rows, E, N, K in itertools.product(big, [-1, 0, 1, 8, 1024, 1025],
                                       [-128, 0, 100, 128, 1 << 20, (1 << 20) + 128],
                                       [0, 128, 4096, 1 << 20, 1 << 40]):
    for dt in (-1, 0, 1, 2):
        g = ctypes.byref(moe.MoeGroupShape(rows, E, N, K, dt, 0))
        lib.moe_linear_workspace_size(g)
        for act in (-7, 0, 3, 5, 1 << 30):
            assert lib.moe_grouped_linear(g, act, P, P, P, P, P, None, W, P, P, None) != 0
            assert lib.moe_grouped_linear_grad(g, act, P, P, P, None, W, P, P, None) != 0
        n += 1
for T, E, k, d, F in itertools.product(big, [0, 1, 8, 1024, 1 << 40], [-1, 1, 2, 64, 65],
                                       [128, 100, 1 << 20, 1 << 40], [128, 1 << 20, -128]):
    for dt, cap, fl in ((0, 0, 0), (1, 3, 2), (1, 1 << 62, 1), (2, -5, 8)):
        s = ctypes.byref(moe.shape(T, d, E, k, F, cap, dt, fl))
        lib.moe_few_workspace_size(s)
        assert lib.moe_layer_few(s, P, P, None, P, P, P, None, W, P, None, None, None, None, None) != 0
        w = ctypes.byref(moe.MoeFp8Tensor(P, P))
        assert lib.moe_layer_few_fp8(s, 1, P, P, None, w, w, w, None, W, P, None, None, None, None,
                                     None) != 0
        n += 1
for count in big:
    lib.moe_grad_workspace_size(count)
for words in itertools.product([0, 1, 2, P], [0, 3, P], big, [-1, 0, 1, 2, 1 << 40]):
    g = (ctypes.c_int64 * 8)(P, P, 64, 1, *words)
    assert lib.moe_grad_norm(2, g, None, W, P, None) != 0
    assert lib.moe_grad_clip(2, g, float("nan"), P, None) != 0
    assert lib.moe_grad_clip(2, g, -1.0, P, None) != 0
    n += 1
for f in (lib.moe_linear_workspace_size, lib.moe_few_workspace_size):
    assert f(None) == 0
print("calls", n)
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
    assert r.stdout.split()[0] == "calls"
