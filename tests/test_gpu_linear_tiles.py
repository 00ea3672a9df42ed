"""Every tile of the linear layers, whole and cut along the reduction, with few experts and with many,
against the 64-bit form."""
import pytest
import torch

import routing_expert_ffn_router_amd as moe
from _fp8 import offsets_of
from _linear import ACTS, DTYPES
from _linear_tiles import CASES, FIRST, SLACK, pieces_of, shape_of
from test_gpu_linear import SENTINEL, _check

pytestmark = pytest.mark.gpu

IDS = [f"{c[0]}-{c[1]}x{c[2]}-{'cut' if c[3] else 'whole'}-E{len(c[4])}-K{c[5]}-N{c[6]}" for c in CASES]


def _case(case, seed):
    dtype, _, _, _, counts, K, N = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[dtype][0]
    E, R = len(counts), FIRST + sum(counts) + SLACK
    made = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.float32)
    c = {"x": made(R, K).to(dt), "w": torch.stack([(made(N, K) / K ** 0.5).to(dt) for _ in range(E)]),
         "bias": made(E, N), "res": made(R, N).to(dt), "offsets": offsets_of(counts, FIRST), "R": R,
         "E": E, "N": N, "K": K, "dtype": dtype}
    for n, bad in (("x", float("nan")), ("res", float("inf"))):  # rows of no expert
        c[n][:FIRST] = bad
        c[n][R - SLACK:] = bad
    return c


def _run(case, c, act, bias=True, res=True, keep=True, in_place=False, byte=255):
    g, dt = shape_of(case), DTYPES[c["dtype"]][0]
    ws = torch.full((moe.linear_workspace_size(g),), byte, dtype=torch.uint8, device="cuda")
    new = lambda: torch.full((c["R"], c["N"]), SENTINEL, dtype=dt, device="cuda")
    z = new() if keep else None
    y = c["res"].clone() if in_place else new()
    r = (y if in_place else c["res"]) if res else None
    moe.grouped_linear(g, ACTS[act], c["x"], c["offsets"].cuda(), c["w"], c["bias"] if bias else None,
                       r, ws, y, z)
    return z, y


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_tiles(case):
    assert moe.linear_tiles(shape_of(case))[:2] == (case[1], case[2])
    assert (pieces_of(case) > 1) == case[3]
    c = _case(case, seed=case[5] + case[6])
    z, y = _run(case, c, "gelu")
    _check(c, "gelu", z, y)
    again = _run(case, c, "gelu", byte=0)
    a, b = int(c["offsets"][0]), int(c["offsets"][-1])
    assert torch.equal(z[a:b], again[0][a:b]) and torch.equal(y[a:b], again[1][a:b])


@pytest.mark.parametrize("case", [c for c in CASES if c[2] == 256], ids=[
    i for i, c in zip(IDS, CASES) if c[2] == 256])
def test_residual_in_place(case):
    c = _case(case, seed=3)
    want = _run(case, c, "silu", keep=False)[1]
    got = _run(case, c, "silu", keep=False, in_place=True)[1]
    a, b = int(c["offsets"][0]), int(c["offsets"][-1])
    assert torch.equal(got[a:b], want[a:b])
    bits = torch.int16 if c["dtype"] == "bf16" else torch.int32
    for rows in (slice(0, a), slice(b, None)):
        assert torch.equal(got[rows].view(bits), c["res"][rows].view(bits))


SOME = [i for i, c in enumerate(CASES) if c[2] == 256 and len(c[4]) <= 8]


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("bias,res,keep", [(True, False, True), (False, True, False),
                                           (False, False, False)])
@pytest.mark.parametrize("which", [1, 6, 11, 16])  # a cut case of each large tile
def test_every_epilogue_of_a_cut_tile(which, bias, res, keep, act):
    case = CASES[which]
    assert case[2] == 256 and case[3] and which in SOME
    c = _case(case, seed=11)
    z, y = _run(case, c, act, bias, res, keep)
    _check(c, act, z, y, bias, res)
