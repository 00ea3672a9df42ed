"""Argument checks, workspace sizes and refusals of the linear layers and of gradient clipping on
the host.  Nothing here launches a kernel: every call is refused before the first HIP
call."""
import ctypes

import pytest

import routing_expert_ffn_router_amd as moe

lib = moe.load_library()
P = 4096  # a 256-byte aligned address that is never read
INVALID, UNSUPPORTED = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
ALIGNMENT, WORKSPACE = moe.MOE_ERR_ALIGNMENT, moe.MOE_ERR_WORKSPACE


def group(**kw):
    a = dict(rows=100, E=4, N=256, K=128, dtype=moe.MOE_BF16, scale_type=moe.MOE_SCALE_F32)
    a.update(kw)
    return moe.MoeGroupShape(**a)


def linear(g, **kw):
    a = dict(act=moe.MOE_ACT_GELU, x=P, off=P, w=P, bias=P, res=P, work=P, n=1 << 40, z=P, y=P)
    a.update(kw)
    return lib.moe_grouped_linear(None if g is None else ctypes.byref(g), a["act"], a["x"],
                                  a["off"], a["w"], a["bias"], a["res"], a["work"], a["n"],
                                  a["z"], a["y"], None)


def linear_grad(g, **kw):
    a = dict(act=moe.MOE_ACT_GELU, dy=P, z=P, off=P, work=P, n=1 << 40, dz=P, db=P)
    a.update(kw)
    return lib.moe_grouped_linear_grad(None if g is None else ctypes.byref(g), a["act"], a["dy"],
                                       a["z"], a["off"], a["work"], a["n"], a["dz"], a["db"], None)


BAD_GROUPS = [
    (dict(rows=-1), INVALID), (dict(E=0), INVALID), (dict(N=0), INVALID), (dict(K=-1), INVALID),
    (dict(E=1025), UNSUPPORTED), (dict(N=200), UNSUPPORTED), (dict(K=64), UNSUPPORTED),
    (dict(N=(1 << 20) + 128), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED),
    (dict(dtype=7), UNSUPPORTED), (dict(rows=(1 << 31) - 1, N=1 << 20), UNSUPPORTED)]
BAD_CALLS = [
    (dict(act=-1), UNSUPPORTED), (dict(act=5), UNSUPPORTED), (dict(off=None), INVALID),
    (dict(work=None), WORKSPACE), (dict(n=0), WORKSPACE), (dict(work=P + 128), ALIGNMENT)]


@pytest.mark.parametrize("call", [linear, linear_grad])
@pytest.mark.parametrize("kw,want", BAD_GROUPS)
def test_group_shapes_are_refused(call, kw, want):
    assert call(group(**kw)) == want
    assert moe.linear_workspace_size(group(**kw)) == 0


@pytest.mark.parametrize("call", [linear, linear_grad])
@pytest.mark.parametrize("kw,want", BAD_CALLS)
def test_calls_are_refused(call, kw, want):
    assert call(group(), **kw) == want
    assert call(None) == INVALID


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID),
    (dict(x=P + 8), ALIGNMENT), (dict(w=P + 8), ALIGNMENT), (dict(bias=P + 4), ALIGNMENT),
    (dict(res=P + 2), ALIGNMENT), (dict(z=P + 8), ALIGNMENT), (dict(y=P + 8), ALIGNMENT)])
def test_linear_operands(kw, want):
    assert linear(group(), **kw) == want


def test_linear_of_no_rows_needs_no_operands():
    assert linear(group(rows=0), x=None, w=None, y=None) == moe.MOE_OK


@pytest.mark.parametrize("kw,want", [
    (dict(dy=None), INVALID), (dict(z=None), INVALID), (dict(dy=P + 8), ALIGNMENT),
    (dict(z=P + 4), ALIGNMENT), (dict(dz=P + 2), ALIGNMENT), (dict(db=P + 4), ALIGNMENT)])
def test_linear_grad_operands(kw, want):
    assert linear_grad(group(), **kw) == want


def test_workspace_is_what_the_call_asks_for():
    for rows in (0, 1, 5000):
        g = group(rows=rows)
        n = moe.linear_workspace_size(g)
        assert n > 0 and n % 256 == 0
        assert linear_grad(g, n=n - 1) == WORKSPACE
        assert linear(g, n=n - 1) == WORKSPACE


def grads(*items):
    words = [w for it in items for w in it]
    return (ctypes.c_int64 * len(words))(*words)


def norm(count, g, work=P, n=1 << 40, out=P):
    return lib.moe_grad_norm(count, g, work, n, out, None)


def clip(count, g, limit=1.0, size=P):
    return lib.moe_grad_clip(count, g, limit, size, None)


GOOD = (P, P, 64, 1)


@pytest.mark.parametrize("item,want", [
    ((P, P, -1, 1), INVALID), ((P, P, 64, 2), UNSUPPORTED), ((P, P, 64, -1), UNSUPPORTED),
    ((P, P, 1 << 36, 1), UNSUPPORTED), ((0, P, 64, 1), INVALID), ((P + 1, P, 64, 1), ALIGNMENT),
    ((P + 2, P, 64, 0), ALIGNMENT)])
def test_gradients_are_refused(item, want):
    assert norm(2, grads(GOOD, item)) == want
    assert clip(2, grads(GOOD, item)) == want


def test_outputs_are_checked_by_clip_alone():
    assert clip(1, grads((P, 0, 64, 1))) == INVALID
    assert clip(1, grads((P, P + 1, 64, 1))) == ALIGNMENT
    assert norm(1, grads((P, 0, 64, 1)), n=0) == WORKSPACE  # passed over


def test_counts_and_scalars_are_refused():
    g = grads(GOOD)
    for call in (norm, clip):
        assert call(-1, g) == INVALID
        assert call(1, None) == INVALID
        assert call((1 << 20) + 1, g) == UNSUPPORTED
    assert norm(1, g, out=None) == INVALID
    assert norm(1, g, out=P + 2) == ALIGNMENT
    assert norm(1, g, work=None) == WORKSPACE
    assert norm(1, g, work=P + 8) == ALIGNMENT
    assert norm(1, g, n=moe.grad_workspace_size(1) - 1) == WORKSPACE
    assert clip(1, g, size=None) == INVALID
    assert clip(1, g, size=P + 1) == ALIGNMENT
    for limit in (-1.0, float("nan"), float("inf")):
        assert clip(1, g, limit=limit) == INVALID


def test_clipping_nothing_needs_no_launch():
    assert clip(0, None) == moe.MOE_OK
    assert clip(1, grads((0, 0, 0, 1))) == moe.MOE_OK


def test_grad_workspace_size():
    assert moe.grad_workspace_size(-1) == 0 and moe.grad_workspace_size((1 << 20) + 1) == 0
    sizes = [moe.grad_workspace_size(n) for n in (0, 1, 192, 193, 1 << 20)]
    assert all(n > 0 and n % 256 == 0 for n in sizes) and sizes == sorted(sizes)
