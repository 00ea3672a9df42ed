"""Argument checks, workspace sizes and refusals of the 8-bit operators and the gradients on the
host.  Nothing here launches a kernel: every call is refused before the first HIP call."""
import ctypes

import pytest
import torch

import _fp8 as ref
import routing_expert_ffn_router_amd as moe

lib = moe.load_library()
P = 4096  # a 256-byte aligned address that is never read
INVALID, UNSUPPORTED = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
ALIGNMENT, WORKSPACE = moe.MOE_ERR_ALIGNMENT, moe.MOE_ERR_WORKSPACE


def group(**kw):
    a = dict(rows=100, E=4, N=256, K=128, dtype=moe.MOE_BF16, scale_type=moe.MOE_SCALE_F32)
    a.update(kw)
    return moe.MoeGroupShape(**a)


def quantize(rows=128, K=256, block=1, dtype=1, kind=0, x=P, q=P, scale=P):
    return lib.moe_quantize(rows, K, block, dtype, kind, x, q, scale, None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INVALID), (dict(K=0), INVALID), (dict(K=-128), INVALID),
    (dict(block=2), INVALID), (dict(block=0), INVALID), (dict(rows=100, block=128), INVALID),
    (dict(K=100), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED),
    (dict(kind=2), UNSUPPORTED), (dict(kind=-1), UNSUPPORTED),
    (dict(rows=1 << 30, K=128), UNSUPPORTED), (dict(rows=1 << 62, K=1 << 61), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(q=None), INVALID), (dict(scale=None), INVALID),
    (dict(x=P + 8), ALIGNMENT), (dict(q=P + 4), ALIGNMENT), (dict(scale=P + 2), ALIGNMENT)])
def test_quantize_refusals(kw, want):
    assert quantize(**kw) == want


def test_quantize_of_no_rows_needs_no_pointers():
    assert quantize(rows=0, x=None, q=None, scale=None) == moe.MOE_OK


BAD_GROUPS = [
    (dict(rows=-1), INVALID), (dict(E=0), INVALID), (dict(N=0), INVALID), (dict(K=-1), INVALID),
    (dict(E=1025), UNSUPPORTED), (dict(N=200), UNSUPPORTED), (dict(K=64), UNSUPPORTED),
    (dict(N=(1 << 20) + 128), UNSUPPORTED), (dict(K=1 << 21), UNSUPPORTED),
    (dict(rows=1 << 31), UNSUPPORTED), (dict(dtype=7), UNSUPPORTED),
    (dict(scale_type=2), UNSUPPORTED),
    (dict(rows=(1 << 31) - 1, N=1 << 20, K=1 << 20), UNSUPPORTED),  # a grid past the limit
    (dict(E=1024, N=1 << 17, K=1 << 17), UNSUPPORTED)]


def gemm(g, **kw):
    a = dict(xq=P, xs=P, off=P, wq=P, ws=P, work=P, n=1 << 30, y=P)
    a.update(kw)
    return lib.moe_grouped_gemm_fp8(None if g is None else ctypes.byref(g), a["xq"], a["xs"],
                                    a["off"], a["wq"], a["ws"], a["work"], a["n"], a["y"], None)


def dgrad(g, **kw):
    a = dict(dy=P, off=P, w=P, work=P, n=1 << 30, dx=P)
    a.update(kw)
    return lib.moe_grouped_dgrad(None if g is None else ctypes.byref(g), a["dy"], a["off"],
                                 a["w"], a["work"], a["n"], a["dx"], None)


def wgrad(g, **kw):
    a = dict(dy=P, x=P, off=P, work=P, n=1 << 30, dw=P)
    a.update(kw)
    return lib.moe_grouped_wgrad(None if g is None else ctypes.byref(g), a["dy"], a["x"],
                                 a["off"], a["work"], a["n"], a["dw"], None)


@pytest.mark.parametrize("call", [gemm, dgrad, wgrad])
@pytest.mark.parametrize("kw,want", BAD_GROUPS)
def test_group_shapes_are_refused(call, kw, want):
    assert call(group(**kw)) == want
    assert moe.group_workspace_size(group(**kw)) == 0


@pytest.mark.parametrize("call", [gemm, dgrad, wgrad])
def test_group_calls_check_workspace_and_offsets(call):
    g = group()
    need = moe.group_workspace_size(g)
    assert need > 0
    assert call(None) == INVALID
    assert call(g, off=None) == INVALID  # only one expert does without
    assert call(g, work=None) == WORKSPACE
    assert call(g, n=need - 1) == WORKSPACE
    assert call(g, work=P + 16) == ALIGNMENT


@pytest.mark.parametrize("name,want", [("xq", ALIGNMENT), ("wq", ALIGNMENT), ("y", ALIGNMENT)])
def test_gemm_operands(name, want):
    assert gemm(group(), **{name: None}) == INVALID
    assert gemm(group(), **{name: P + 8}) == want


def test_gemm_scales_and_types():
    assert gemm(group(), xs=None) == INVALID and gemm(group(), ws=None) == INVALID
    assert gemm(group(), xs=P + 2) == ALIGNMENT and gemm(group(), ws=P + 1) == ALIGNMENT
    # outputs are bf16 only: the 8-bit instruction does not hold a sum to fp32's precision
    assert gemm(group(dtype=moe.MOE_F32)) == UNSUPPORTED


@pytest.mark.parametrize("call,names", [(dgrad, ("dy", "w", "dx")), (wgrad, ("dy", "x", "dw"))])
def test_gradient_operands(call, names):
    for n in names:
        assert call(group(), **{n: None}) == INVALID
        assert call(group(), **{n: P + 4}) == ALIGNMENT


def test_no_rows_need_no_operands():
    g = group(rows=0)
    assert gemm(g, xq=None, xs=None, wq=None, ws=None, y=None) == moe.MOE_OK
    assert dgrad(g, dy=None, w=None, dx=None) == moe.MOE_OK
    assert wgrad(g, dw=None) == INVALID  # its zeros have to go somewhere


def tiles(rows, E):
    """Row tiles of at most 256 rows when all experts but one hold a single row."""
    return rows if rows <= E else E - 1 + -(-(rows - E + 1) // 256)


@pytest.mark.parametrize("rows", [0, 1, 63, 64, 100, 4096, 32768, 1 << 20])
@pytest.mark.parametrize("E", [1, 8, 256, 1024])
def test_group_workspace_holds_every_tile_table(rows, E):
    need = moe.group_workspace_size(group(rows=rows, E=E))
    assert need % 256 == 0 and need >= 4 * (1 + 2 * tiles(rows, E))


@pytest.mark.parametrize("kw,slots", [
    # one expert's few tiles leave most CUs idle: pieces from 32 steps of the reduction.  dgrad
    # takes N in steps of 64, tiles of 256 rows (128 up to 16 rows) by 256 columns of K
    (dict(rows=256, E=1, N=4096, K=2048), 8 * 8), (dict(rows=1024, E=1, N=2048, K=5120), 80 * 4),
    (dict(rows=300, E=1, N=1920, K=1024), 0),
    # whole rounds before a short last one; a last round of more than half the CUs has no pieces
    (dict(rows=4096, E=1, N=2048, K=5120), 320 * 4), (dict(rows=4096, E=1, N=4096, K=2176), 0),
    (dict(rows=4096, E=1, N=10240, K=4096), 0),
    # the 8-bit product takes K in steps of 128, and columns of N
    (dict(rows=256, E=1, N=1920, K=4096), 8 * 4), (dict(rows=4096, E=1, N=1024, K=5120), 64 * 5),
])
def test_few_tiles_have_room_for_pieces(kw, slots):
    have = moe.group_workspace_size(group(**kw))
    assert have - min(slots, 256) * 256 * 256 * 4 in range(256, 4096)


# -------------------------------------------------------------- experts' network and layer
def fp8(q=P, scale=P):
    return moe.MoeFp8Tensor(q, scale)


def ffn(s, kind=0, n=1 << 40, x=P, src=P, off=P, wg=None, wu=None, wd=None, work=P, y=P,
        null_weight=False):
    w = [ctypes.byref(t or fp8()) for t in (wg, wu, wd)]
    if null_weight:
        w[1] = None
    return lib.moe_expert_ffn_fp8(ctypes.byref(s), kind, x, src, off, w[0], w[1], w[2], work, n,
                                  y, None)


def layer(s, kind=0, n=1 << 40, x=P, wr=P, wg=None, work=P, out=P):
    return lib.moe_layer_fp8(ctypes.byref(s), kind, x, wr, None, ctypes.byref(wg or fp8()),
                             ctypes.byref(fp8()), ctypes.byref(fp8()), work, n, out, None, None,
                             None, None, None)


OK_SHAPE = (64, 256, 8, 2, 384)


@pytest.mark.parametrize("call", [ffn, layer])
def test_fp8_shapes(call):
    s = moe.shape(*OK_SHAPE)
    need = moe.fp8_workspace_size(s, 0)
    assert need > 0
    assert call(s, kind=2) == UNSUPPORTED and moe.fp8_workspace_size(s, 2) == 0
    f32 = moe.shape(*OK_SHAPE, dtype=moe.MOE_F32)
    assert call(f32) == UNSUPPORTED and moe.fp8_workspace_size(f32, 0) == 0
    assert call(moe.shape(64, 200, 8, 2, 384)) == UNSUPPORTED
    assert call(moe.shape(64, 256, 8, 9, 384)) == INVALID
    assert call(s, n=need - 1) == WORKSPACE
    assert call(s, work=None) == WORKSPACE
    assert call(s, work=P + 128) == ALIGNMENT
    assert call(s, x=None) == INVALID
    assert call(s, x=P + 8) == ALIGNMENT
    assert call(s, wg=fp8(q=None)) == INVALID and call(s, wg=fp8(scale=None)) == INVALID
    assert call(s, wg=fp8(q=P + 1)) == ALIGNMENT
    assert call(s, wg=fp8(scale=P + 2)) == ALIGNMENT
    # gathered rows are addressed with 32 bits
    wide = moe.shape(1 << 20, 1 << 11, 8, 1, 128)
    assert call(wide) == UNSUPPORTED


def test_ffn_operands():
    s = moe.shape(*OK_SHAPE)
    assert ffn(s, off=None) == INVALID and ffn(s, y=None) == INVALID
    assert ffn(s, y=P + 4) == ALIGNMENT
    assert ffn(s, null_weight=True) == INVALID
    assert ffn(moe.shape(0, 256, 8, 2, 384), x=None, src=None, y=None) == moe.MOE_OK


def test_layer_operands():
    s = moe.shape(*OK_SHAPE)
    assert layer(s, wr=None) == INVALID and layer(s, out=None) == INVALID
    assert layer(s, out=P + 2) == ALIGNMENT and layer(s, wr=P + 2) == ALIGNMENT


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("T,d,E,k,F,C,flags", [
    (0, 128, 4, 2, 128, 0, 0), (1, 128, 4, 1, 128, 0, 0), (256, 7168, 256, 8, 2048, 0, 0),
    (4096, 4096, 8, 2, 14336, 1280, 0), (100, 256, 8, 2, 384, 16, 0),
    (100, 256, 8, 2, 384, 40, moe.MOE_FLAG_PAD_TO_CAPACITY)])
def test_fp8_workspace_layout(T, d, E, k, F, C, flags, kind):
    s = moe.shape(T, d, E, k, F, C, flags=flags)
    size, lay = moe.fp8_workspace_size(s, kind), moe.fp8_workspace_layout(s, kind)
    R, per = moe.max_rows(s), (4, 1)[kind]
    offs = list(lay.values()) + [size]
    assert all(o % 256 == 0 for o in offs) and offs == sorted(offs)
    room = {n: b - a for n, a, b in zip(lay, offs, offs[1:])}

    def rows(n, width):
        return (n * width + 255) // 256 * 256 + n * (width // 128) * per

    # the quantized token rows, or packed rows, whichever are more, and the hidden rows
    assert room["x_perm"] >= rows(max(T, R), d) and room["h"] >= rows(R, F)
    assert room["y_perm"] >= R * d * 2 and room["src_token"] >= 4 * R
    # partial sums of at most 256 pieces of 256 x 256 outputs
    assert room["down_acc"] <= 256 * 256 * 256 * 4
    # the table: the count, then (expert, first row) of each row tile
    assert room["sched"] >= 4 * (1 + 2 * tiles(R, E))


# ------------------------------------------------------------------- the binding's own checks
def test_binding_refuses_host_tensors_and_wrong_types(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    g = moe.group_shape(4, 2, 128, 128)
    t = lambda *s, d=torch.uint8: torch.zeros(s, dtype=d)  # noqa: E731
    off = torch.zeros(3, dtype=torch.int32)
    good = dict(xq=t(4, 128), x_scale=t(4, 1, d=torch.float32), wq=t(2, 128, 128),
                w_scale=t(2, 1, 1, d=torch.float32), y=t(4, 128, d=torch.bfloat16))

    def call(**kw):
        a = {**good, **kw}
        moe.grouped_gemm_fp8(g, a["xq"], a["x_scale"], off, a["wq"], a["w_scale"], None, a["y"])

    for kw in (dict(), dict(wq=t(2, 128, 256)), dict(wq=t(2, 128, 128, d=torch.float16)),
               dict(w_scale=t(2, 1, 1)), dict(wq=t(2, 128, 128).transpose(1, 2))):
        with pytest.raises(ValueError):  # dict(): everything fits but is on the host
            call(**kw)


def test_binding_names_what_is_missing(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    x, q = torch.zeros((2, 128, 128)), torch.zeros((2, 128, 128), dtype=torch.uint8)
    scale = torch.zeros((2, 1, 1))
    for args in ((None, 1, 0, q, scale), (x, 128, 0, None, scale), (x, 128, 0, q, None)):
        with pytest.raises(ValueError):
            moe.quantize(*args)
    w = (q, scale)
    s = moe.shape(4, 128, 2, 1, 128)
    a = torch.zeros((4, 128), dtype=torch.bfloat16)
    # (the first weight to be looked at is refused, before anything on the host is)
    for ws in ((None, w, w), ((q,), w, w), (q, w, w), ((None, scale), w, w)):
        with pytest.raises(ValueError, match="w_gate|w_up|w_down"):
            moe.expert_ffn_fp8(s, 0, a, None, torch.zeros(3, dtype=torch.int32), *ws, None, a)
        with pytest.raises(ValueError, match="w_gate|w_up|w_down"):
            moe.layer_fp8(s, 0, a, a[:2], None, *ws, None, a)


# --------------------------------------------------------------- the tests' own plain forms
def test_plain_quantizer_is_the_least_scale_and_the_nearest_value():
    g = torch.Generator().manual_seed(0)
    x = (torch.randn((64, 256), generator=g) * torch.exp(4 * torch.randn((64, 1), generator=g)))
    grid = torch.arange(256, dtype=torch.uint8)
    grid = grid[(grid & 127) != 127].view(torch.float8_e4m3fn).double()
    for dtype in (torch.float32, torch.bfloat16):
        v = x.to(dtype)
        q, e = ref.quantize(v, 1)
        s = ref.power(e)
        amax = v.double().abs().view(64, 2, 128).amax(2)
        assert bool((amax <= 448 * s).all()) and bool((amax > 224 * s).all())
        scaled = v.double() / s.repeat_interleave(128, 1)
        near = (scaled[..., None] - grid).abs().amin(-1)
        assert torch.equal((scaled - q.double()).abs(), near)
