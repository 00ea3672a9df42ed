"""The experts' linear layers against their 64-bit form."""
import pytest
import torch

import routing_expert_ffn_router_amd as moe
from _fp8 import offsets_of
from _linear import ACTS, DTYPES, value, value_error

pytestmark = pytest.mark.gpu

SENTINEL = 777.0


def _case(counts, K, N, dtype, seed, slack=3, first=2):
    g = torch.Generator().manual_seed(seed)
    dt = DTYPES[dtype][0]
    E, R = len(counts), first + sum(counts) + slack
    c = {"x": torch.randn((R, K), generator=g).to(dt),
         "w": (torch.randn((E, N, K), generator=g) / K ** 0.5).to(dt),
         "bias": torch.randn((E, N), generator=g), "res": torch.randn((R, N), generator=g).to(dt),
         "offsets": offsets_of(counts, first), "R": R, "E": E, "N": N, "K": K, "dtype": dtype}
    # rows that belong to no expert hold anything at all
    for n, bad in (("x", float("nan")), ("res", float("inf"))):
        c[n][:first] = bad
        c[n][first + sum(counts):] = bad
    return c


def _run(c, act, bias=True, res=True, keep=True, in_place=False, ws_byte=255):
    dt = DTYPES[c["dtype"]]
    g = moe.group_shape(c["R"], c["E"], c["N"], c["K"], dt[1])
    ws = torch.empty(moe.linear_workspace_size(g), dtype=torch.uint8, device="cuda").fill_(ws_byte)
    z = torch.full((c["R"], c["N"]), SENTINEL, dtype=dt[0], device="cuda") if keep else None
    y = c["res"].cuda() if in_place else torch.full((c["R"], c["N"]), SENTINEL, dtype=dt[0],
                                                    device="cuda")
    r = (y if in_place else c["res"].cuda()) if res else None
    moe.grouped_linear(g, ACTS[act], c["x"].cuda(), c["offsets"].cuda(), c["w"].cuda(),
                       c["bias"].cuda() if bias else None, r, ws, y, z)
    return z.cpu() if keep else None, y.cpu()


def _over(err, bound):
    return float((err - bound).max()) if err.numel() else 0.0


def _check(c, act, z, y, bias=True, res=True):
    half, off = DTYPES[c["dtype"]][2], c["offsets"].tolist()
    for e, (a, b) in enumerate(zip(off, off[1:])):
        if a == b:
            continue
        x, w = c["x"][a:b].cuda().double(), c["w"][e].cuda().double()
        want = x @ w.t()
        # a rounding for each product and addition, the bias's with them
        err = (c["K"] + 2) * 2.0 ** -24 * (x.abs() @ w.abs().t())
        if bias:
            want = want + c["bias"][e].cuda().double()
            err = err + 2.0 ** -24 * (want.abs() + c["bias"][e].cuda().double().abs())
        if z is not None:
            assert _over((z[a:b].cuda().double() - want).abs(), half * (want.abs() + err) + err) <= 0, e
        # no slope of the activations passes 1.13
        err = 1.13 * err + value_error(want, act)
        want = value(want, act)
        if res:
            want = want + c["res"][a:b].cuda().double()
            err = err + 2.0 ** -24 * (want.abs() + err)
        assert _over((y[a:b].cuda().double() - want).abs(), half * (want.abs() + err) + err) <= 0, e
    for t in (z, y):
        if t is not None:
            for part in (t[:off[0]], t[off[-1]:]):
                assert bool((part == SENTINEL).all())


CASES = [([1], 128, 128), ([0, 1, 0], 128, 256), ([2, 0, 31, 32, 33], 384, 128),
         ([63, 64, 65, 0], 256, 384), ([127, 128, 129], 256, 256), ([300, 5, 0, 257], 384, 640),
         ([700], 640, 384), ([1, 0, 2, 3] * 17, 128, 128), ([5], 8192, 128), ([40], 128, 8192),
         ([0] * 1000 + [2] * 24, 128, 128)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("counts,K,N", CASES)
def test_linear(counts, K, N, dtype):
    c = _case(counts, K, N, dtype, seed=N + sum(counts))
    _check(c, "gelu", *_run(c, "gelu"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("bias,res,keep", [(True, False, True), (False, True, False),
                                           (False, False, False), (True, True, True)])
def test_every_epilogue(act, bias, res, keep, dtype):
    c = _case([40, 0, 130, 3], 256, 384, dtype, seed=11)
    _check(c, act, *_run(c, act, bias, res, keep), bias, res)


@pytest.mark.parametrize("counts,K,N", [
    # the last round's tiles in pieces; a whole round, then pieces
    ([256], 4096, 2048), ([9], 8192, 1152), ([300], 6144, 384), ([60, 0, 9], 6144, 512),
    ([0, 300, 1, 20], 6272, 640), ([4200], 2048, 5120), ([33], 2048, 7168), ([1], 16384, 128),
    ([1, 2, 0, 5], 4096, 128)])
def test_few_long_tiles(counts, K, N):
    c = _case(counts, K, N, "bf16", seed=K + N)
    z, y = _run(c, "silu")
    _check(c, "silu", z, y)
    again = _run(c, "silu", ws_byte=0)
    assert torch.equal(z, again[0]) and torch.equal(y, again[1])


@pytest.mark.parametrize("dtype,counts,K,N", [
    # blocks that work through several tiles
    ("bf16", [20, 300, 0, 5], 128, 16768), ("bf16", [9, 0, 16, 1, 3], 128, 22912),
    ("bf16", [1, 300, 0, 257, 20] * 13, 256, 1152), ("f32", [130, 1, 70], 384, 11392),
    ("f32", [1, 130, 0, 17, 20] * 13, 128, 1152), ("bf16", [4200, 0, 9000], 256, 1152)])
def test_many_tiles(counts, K, N, dtype):
    c = _case(counts, K, N, dtype, seed=N + sum(counts))
    _check(c, "gelu_tanh", *_run(c, "gelu_tanh"))


@pytest.mark.parametrize("counts,K,N", [([40, 0, 130], 256, 384), ([33], 2048, 1152),
                                        ([300], 6144, 384)])
def test_residual_in_place(counts, K, N):
    c = _case(counts, K, N, "bf16", seed=3)
    want = _run(c, "none", keep=False)[1]
    got = _run(c, "none", keep=False, in_place=True)[1]
    a, b = c["offsets"][0], c["offsets"][-1]
    assert torch.equal(got[a:b], want[a:b])
    assert torch.equal(got[:a].view(torch.int16), c["res"][:a].view(torch.int16))
    assert torch.equal(got[b:].view(torch.int16), c["res"][b:].view(torch.int16))


def test_one_expert_without_offsets_and_no_rows():
    c = _case([100], 256, 384, "bf16", seed=6, slack=0, first=0)
    want = _run(c, "relu")[1]
    g = moe.group_shape(100, 1, 384, 256, moe.MOE_BF16)
    ws = torch.empty(moe.linear_workspace_size(g), dtype=torch.uint8, device="cuda")
    y = torch.empty((100, 384), dtype=torch.bfloat16, device="cuda")
    moe.grouped_linear(g, ACTS["relu"], c["x"].cuda(), None, c["w"].cuda(), c["bias"].cuda(),
                       c["res"].cuda(), ws, y)
    assert torch.equal(y.cpu(), want)
    g = moe.group_shape(0, 1, 384, 256, moe.MOE_BF16)
    none = torch.empty((0, 384), dtype=torch.bfloat16, device="cuda")
    moe.grouped_linear(g, 0, torch.empty((0, 256), dtype=torch.bfloat16, device="cuda"), None,
                       c["w"].cuda(), None, None, ws, none)


def test_infinities_and_nans_reach_their_rows_alone():
    c = _case([20, 30], 256, 256, "bf16", seed=9)
    clean = _run(c, "none", res=False)[1]
    c["x"][5, 7], c["x"][30, 0] = float("inf"), float("nan")
    got = _run(c, "none", res=False)[1]
    rows = [r for r in range(c["R"]) if r not in (5, 30)]
    assert torch.equal(got[rows], clean[rows])
    assert not bool(got[[5, 30]].isfinite().any())


def test_refusals_of_the_binding():
    c = _case([40], 256, 384, "bf16", seed=3, slack=0, first=0)
    g = moe.group_shape(40, 1, 384, 256, moe.MOE_BF16)
    ws = torch.empty(moe.linear_workspace_size(g), dtype=torch.uint8, device="cuda")
    y = torch.empty((40, 384), dtype=torch.bfloat16, device="cuda")
    x, w, b, o = c["x"].cuda(), c["w"].cuda(), c["bias"].cuda(), c["offsets"].cuda()
    good = dict(x=x, expert_offsets=o, w=w, bias=b, residual=None, workspace=ws, y=y, z=None)
    for bad in (dict(x=x[:39]), dict(x=x.float()), dict(x=x.t().contiguous().t()), dict(w=w[0]),
                dict(bias=b.bfloat16()), dict(residual=y[:, :128]), dict(y=None),
                dict(z=y.float()), dict(expert_offsets=o.long()), dict(x=x.cpu())):
        with pytest.raises(ValueError):
            moe.grouped_linear(g, 0, **{**good, **bad})
    for act in (-1, 5):
        with pytest.raises(moe.MoeError):
            moe.grouped_linear(g, act, **good)
    with pytest.raises(moe.MoeError):
        moe.grouped_linear(g, 0, **{**good, "workspace": ws[:256]})
