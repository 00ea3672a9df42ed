"""The layer for a few tokens where a block gives up waiting for the others' part of h: forced by a
number of looks of zero, with which no block waits at all and every kernel ends as ever."""
import contextlib

import pytest
import torch

import _few as ref
import routing_expert_ffn_router_amd as moe
from test_gpu_few import _args, _call, _case, _ints, _setup

pytestmark = pytest.mark.gpu


@contextlib.contextmanager
def _polls(n):
    before = moe.few_wait_polls(n)
    try:
        yield
    finally:
        moe.few_wait_polls(before)


# waves along the reduction and across the columns; down's reduction whole and in chunks
@pytest.mark.parametrize("kind", ["bf16", "f32", "e4m3-f32", "e4m3-e8m0"])
@pytest.mark.parametrize("T,E,k,d,F", [(1, 8, 2, 256, 384), (5, 16, 4, 640, 256), (16, 4, 2, 1152, 256),
                                       (3, 4, 2, 4096, 256), (12, 2, 2, 128, 4096), (1, 1, 1, 128, 128)])
def test_a_wait_that_is_given_up_shows(T, E, k, d, F, kind):
    c = _case(T, E, k, d, F, kind, seed=T + d)
    s, ws, out = _setup(c)
    args, ints, good_ints = _args(c), _ints(c), _ints(c)
    good = torch.empty_like(out)
    _call(c, s, ws, good, good_ints, args)
    assert bool(good.isfinite().all()) and int(good_ints[3]) == 0
    with _polls(0):
        _call(c, s, ws, out, ints, args)
        torch.cuda.synchronize()
    assert bool(out.isnan().all())
    assert int(ints[3]) == -(1 << 31)
    for a, b in zip(ints[:3], good_ints[:3]):
        assert torch.equal(a, b)
    # nothing of it is left to the next call
    _call(c, s, ws, out, ints, args)
    assert torch.equal(out, good) and int(ints[3]) == 0


def test_status_still_counts_tokens():
    c = _case(6, 8, 2, 256, 256, "bf16", seed=3)
    c["x"][[2, 5], 7] = float("nan")
    s, ws, out = _setup(c)
    ints = _ints(c)
    with _polls(0):
        _call(c, s, ws, out, ints)
        torch.cuda.synchronize()
    assert int(ints[3]) == -(1 << 31) + 2 and bool(out.isnan().all())
    with _polls(0):
        _call(c, s, ws, out, [None] * 4)  # without a status the outputs alone show it
    assert bool(out.isnan().all())
    _call(c, s, ws, out, ints)
    assert int(ints[3]) == 2


def test_no_tokens_wait_for_nothing():
    c = _case(0, 8, 2, 128, 128, "bf16", seed=1)
    s, ws, out = _setup(c)
    ints = _ints(c)
    with _polls(0):
        _call(c, s, ws, out, ints)
    assert all(bool((v == 0).all()) for v in ints)


def test_a_captured_call_keeps_its_number():
    c = _case(4, 8, 2, 256, 384, "bf16", seed=17)
    s, ws, out = _setup(c)
    ints, args = _ints(c), _args(c)
    _call(c, s, ws, out, ints, args)
    want = out.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _call(c, s, ws, out, ints, args)
    with _polls(0):
        for _ in range(3):
            out.fill_(3)
            ints[3].fill_(-5)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want) and int(ints[3]) == 0
    idx = ref.route(c["x"], c["w_router"], c["b"], 2)[0]
    assert torch.equal(ints[0].cpu(), torch.bincount(idx.flatten(), minlength=8).int())
