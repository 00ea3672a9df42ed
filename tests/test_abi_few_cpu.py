"""Argument checks, workspace sizes and refusals of the layer for a few tokens on the host.  Nothing
here launches a kernel: every call is refused before the first HIP call."""
import ctypes

import pytest

import routing_expert_ffn_router_amd as moe

lib = moe.load_library()
P = 4096  # a 256-byte aligned address that is never read
INVALID, UNSUPPORTED = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
ALIGNMENT, WORKSPACE = moe.MOE_ERR_ALIGNMENT, moe.MOE_ERR_WORKSPACE


def shape(T=4, d=256, E=8, k=2, F=384, capacity=0, dtype=moe.MOE_BF16, flags=0, n_groups=0,
          topk_groups=0):
    return moe.shape(T, d, E, k, F, capacity, dtype, flags, n_groups, topk_groups)


def few(s, **kw):
    a = dict(x=P, wr=P, b=P, g=P, u=P, w=P, ws=P, n=1 << 40, out=P)
    a.update(kw)
    return lib.moe_layer_few(None if s is None else ctypes.byref(s), a["x"], a["wr"], a["b"], a["g"],
                             a["u"], a["w"], a["ws"], a["n"], a["out"], None, None, None, None, None)


def pair(v):
    return None if v is None else ctypes.byref(moe.MoeFp8Tensor(*v))


def few_fp8(s, **kw):
    a = dict(x=P, wr=P, b=P, g=P, u=P, w=P, ws=P, n=1 << 40, out=P, kind=moe.MOE_SCALE_F32, scale=P)
    a.update(kw)
    w = [pair((a[n], a["scale"])) if a[n] is not None else None for n in "guw"]
    return lib.moe_layer_few_fp8(None if s is None else ctypes.byref(s), a["kind"], a["x"], a["wr"],
                                 a["b"], *w, a["ws"], a["n"], a["out"], None, None, None, None, None)


BAD_SHAPES = [
    (dict(T=-1), INVALID), (dict(k=9), INVALID), (dict(d=0), INVALID), (dict(flags=64), INVALID),
    (dict(T=17), UNSUPPORTED), (dict(d=100), UNSUPPORTED), (dict(F=64), UNSUPPORTED),
    (dict(E=1025), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED),
    (dict(T=16, E=64, k=33), UNSUPPORTED),  # 528 pairs
    (dict(T=16, E=64, k=64, F=1 << 20), UNSUPPORTED),
    (dict(T=16, E=64, k=32, F=1 << 20, dtype=moe.MOE_F32), UNSUPPORTED),  # h past 2^31 bytes
    (dict(n_groups=3), INVALID), (dict(n_groups=4, topk_groups=5), INVALID)]


@pytest.mark.parametrize("call", [few, few_fp8])
@pytest.mark.parametrize("kw,want", BAD_SHAPES)
def test_shapes_are_refused(call, kw, want):
    assert call(shape(**kw)) == want
    assert moe.few_workspace_size(shape(**kw)) == 0


@pytest.mark.parametrize("call", [few, few_fp8])
@pytest.mark.parametrize("kw,want", [
    (dict(x=None), INVALID), (dict(wr=None), INVALID), (dict(g=None), INVALID),
    (dict(u=None), INVALID), (dict(w=None), INVALID), (dict(out=None), INVALID),
    (dict(x=P + 8), ALIGNMENT), (dict(wr=P + 2), ALIGNMENT), (dict(g=P + 8), ALIGNMENT),
    (dict(u=P + 8), ALIGNMENT), (dict(w=P + 8), ALIGNMENT), (dict(out=P + 8), ALIGNMENT),
    (dict(ws=None), WORKSPACE), (dict(n=0), WORKSPACE), (dict(ws=P + 128), ALIGNMENT)])
def test_operands_are_refused(call, kw, want):
    assert call(shape(), **kw) == want
    assert call(None) == INVALID


@pytest.mark.parametrize("kw,want", [(dict(kind=2), UNSUPPORTED), (dict(kind=-1), UNSUPPORTED),
                                     (dict(scale=0), INVALID), (dict(scale=P + 2), ALIGNMENT)])
def test_scales_are_refused(kw, want):
    assert few_fp8(shape(), **kw) == want


def test_eight_bits_beside_fp32_are_refused():
    assert few_fp8(shape(dtype=moe.MOE_F32)) == UNSUPPORTED


def test_workspace_sizes():
    for kw in (dict(T=0), dict(T=1), dict(T=16, E=256, k=8), dict(dtype=moe.MOE_F32),
               dict(T=16, E=1024, k=32, F=16384)):
        s = shape(**kw)
        n = moe.few_workspace_size(s)
        assert n > 0 and n % 256 == 0
        assert few(s, n=n - 1) == WORKSPACE
        if s.T:
            assert n >= s.T * s.E * 4 + s.T * s.k * s.F * (2 if s.dtype == moe.MOE_BF16 else 4)
