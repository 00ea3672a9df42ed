"""The backward pass of the experts' linear layers up to their products, against its 64-bit form."""
import pytest
import torch

import routing_expert_ffn_router_amd as moe
from _fp8 import offsets_of
from _linear import ACTS, DTYPES, slope, slope_error, value

pytestmark = pytest.mark.gpu

SENTINEL = 777.0


def _case(counts, N, dtype, seed, slack=3, first=2):
    g = torch.Generator().manual_seed(seed)
    dt = DTYPES[dtype][0]
    R = first + sum(counts) + slack
    c = {"dy": torch.randn((R, N), generator=g).to(dt),
         "z": (torch.randn((R, N), generator=g) * 2).to(dt), "offsets": offsets_of(counts, first),
         "R": R, "E": len(counts), "N": N, "dtype": dtype}
    # rows that belong to no expert hold anything at all
    for n, bad in (("dy", float("nan")), ("z", float("inf"))):
        c[n][:first] = bad
        c[n][first + sum(counts):] = bad
    return c


def _run(c, act, dz=True, db=True, z=True):
    dt = DTYPES[c["dtype"]]
    g = moe.group_shape(c["R"], c["E"], c["N"], 128, dt[1])
    ws = torch.empty(moe.linear_workspace_size(g), dtype=torch.uint8, device="cuda").fill_(255)
    out = torch.full((c["R"], c["N"]), SENTINEL, dtype=dt[0], device="cuda") if dz else None
    bias = torch.full((c["E"], c["N"]), float("nan"), device="cuda") if db else None
    moe.grouped_linear_grad(g, ACTS[act], c["dy"].cuda(), c["z"].cuda() if z else None,
                            c["offsets"].cuda(), ws, out, bias)
    return out.cpu() if dz else None, bias.cpu() if db else None


def _over(err, bound):
    return float((err - bound).max()) if err.numel() else 0.0


def _check(c, act, dz, db):
    half = DTYPES[c["dtype"]][2]
    off = c["offsets"].tolist()
    for e, (a, b) in enumerate(zip(off, off[1:])):
        dy, z = c["dy"][a:b].double(), c["z"][a:b].double()
        want, err = dy * slope(z, act), dy.abs() * slope_error(z, act)
        # the product's rounding to fp32, and to the type
        err = err + 2.0 ** -24 * want.abs()
        if dz is not None:
            assert _over((dz[a:b].double() - want).abs(), half * (want.abs() + err) + err) <= 0, e
        if db is not None:
            # one rounding for each addition, within the sum of magnitudes
            n = b - a
            bound = err.sum(0) + (n + 1) * 2.0 ** -24 * (want.abs() + err).sum(0)
            assert _over((db[e].double() - want.sum(0)).abs(), bound) <= 0, e
    if dz is not None:
        assert bool((dz[:off[0]] == SENTINEL).all()) and bool((dz[off[-1]:] == SENTINEL).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("counts,N", [
    ([1], 128), ([0, 1, 0], 256), ([63, 64, 65, 0, 1], 384), ([300, 0, 5, 129], 640),
    ([2, 1, 0, 0, 3] * 20, 128), ([1500], 1152)])
def test_linear_grad(counts, N, act, dtype):
    c = _case(counts, N, dtype, seed=N + sum(counts))
    _check(c, act, *_run(c, act))


@pytest.mark.parametrize("counts", [[0] * 1000 + [70] * 24, [1] * 1024, [0] * 3, [5000, 1]])
def test_many_and_empty_experts(counts):
    c = _case(counts, 128, "bf16", seed=len(counts))
    dz, db = _run(c, "silu")
    _check(c, "silu", dz, db)
    assert bool((db[[i for i, n in enumerate(counts) if n == 0]] == 0).all())


def test_no_rows():
    g = moe.group_shape(0, 3, 256, 128, moe.MOE_BF16)
    ws = torch.empty(moe.linear_workspace_size(g), dtype=torch.uint8, device="cuda")
    db = torch.full((3, 256), float("nan"), device="cuda")
    dy = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    moe.grouped_linear_grad(g, moe.MOE_ACT_GELU, dy, dy, torch.zeros(4, dtype=torch.int32).cuda(),
                            ws, dy, db)
    assert bool((db == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_each_output_alone_in_place_and_without_z(dtype):
    c = _case([70, 0, 9], 384, dtype, seed=4)
    both = _run(c, "gelu")
    assert torch.equal(_run(c, "gelu", db=False)[0], both[0])
    assert torch.equal(_run(c, "gelu", dz=False)[1], both[1])
    dz, db = _run(c, "none", z=False)
    _check(c, "none", dz, db)
    g = moe.group_shape(c["R"], c["E"], c["N"], 128, DTYPES[dtype][1])
    ws = torch.empty(moe.linear_workspace_size(g), dtype=torch.uint8, device="cuda")
    dy, off = c["dy"].cuda(), c["offsets"].cuda()
    moe.grouped_linear_grad(g, ACTS["gelu"], dy, c["z"].cuda(), off, ws, dy)
    a, b = c["offsets"][0], c["offsets"][-1]
    assert torch.equal(dy[a:b].cpu(), both[0][a:b])


def test_one_expert_without_offsets():
    c = _case([100], 256, "bf16", seed=6, slack=0, first=0)
    want = _run(c, "relu")
    g = moe.group_shape(100, 1, 256, 128, moe.MOE_BF16)
    ws = torch.empty(moe.linear_workspace_size(g), dtype=torch.uint8, device="cuda")
    dz = torch.empty((100, 256), dtype=torch.bfloat16, device="cuda")
    db = torch.empty((1, 256), device="cuda")
    moe.grouped_linear_grad(g, ACTS["relu"], c["dy"].cuda(), c["z"].cuda(), None, ws, dz, db)
    assert torch.equal(dz.cpu(), want[0]) and torch.equal(db.cpu(), want[1])


@pytest.mark.parametrize("act", list(ACTS))
def test_slopes_of_extreme_values(act):
    inf = float("inf")
    z = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 20.0, -20.0, 1e4, -1e4, 1e20, -1e20, 3e38, -3e38,
                      inf, -inf, float("nan")])
    zs = torch.zeros((1, 128))
    zs[0, :len(z)] = z
    g = moe.group_shape(1, 1, 128, 128, moe.MOE_F32)
    ws = torch.empty(moe.linear_workspace_size(g), dtype=torch.uint8, device="cuda")
    dz = torch.empty((1, 128), device="cuda")
    moe.grouped_linear_grad(g, ACTS[act], torch.ones((1, 128)).cuda(), zs.cuda(), None, ws, dz)
    got = dz.cpu()[0, :len(z)].double()
    want = slope(z[:12].clamp(-1e3, 1e3).double(), act)
    assert bool(((got[:12] - want).abs() <= 20 * 2.0 ** -24).all())
    assert got[12] == 1 and got[13] == (1 if act == "none" else 0)
    assert act == "none" or bool(got[14].isnan())


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_slopes_equal_differences(act):
    z = torch.linspace(-6, 6, 128)
    g = moe.group_shape(1, 1, 128, 128, moe.MOE_F32)
    ws = torch.empty(moe.linear_workspace_size(g), dtype=torch.uint8, device="cuda")
    dz = torch.empty((1, 128), device="cuda")
    moe.grouped_linear_grad(g, ACTS[act], torch.ones((1, 128)).cuda(), z.view(1, 128).cuda(), None,
                            ws, dz)
    h = 1e-4
    d = (value(z.double() + h, act) - value(z.double() - h, act)) / (2 * h)
    # third derivatives of these are below 3: h^2 / 6 of that, and fp32's 16 units
    assert float((dz.cpu()[0].double() - d).abs().max()) <= h * h / 2 + 20 * 2.0 ** -24
