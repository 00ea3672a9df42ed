"""The 8-bit operators against their 64-bit forms: quantizer, grouped product, experts' network
and layer."""
import numpy as np
import pytest
import torch

import moe_inputs as mi
import routing_expert_ffn_router_amd as moe
import _fp8 as ref
from _util import log

pytestmark = pytest.mark.gpu

HALF_BF16 = 2.0 ** -8  # a rounding to bf16, relative to the value


def _bits(q):
    return q.cpu().view(torch.uint8)


# ------------------------------------------------------------------------------- quantizer
def _quantize(x, block, kind):
    rows, K = x.shape
    q = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty((rows // block, K // 128), device="cuda",
                    dtype=torch.float32 if kind == "f32" else torch.uint8)
    moe.quantize(x.cuda(), block, ref.SCALES[kind], q, s)
    return q, s


def _expected_scale(e, kind):
    return ref.power(e).float() if kind == "f32" else (e + 127).to(torch.uint8)


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,K,block", [
    (1, 128, 1), (3, 256, 1), (17, 1152, 1), (1000, 384, 1), (4099, 640, 1),
    (128, 128, 128), (256, 640, 128), (1152, 2048, 128)])
def test_quantize_equals_definition(rows, K, block, dtype, kind):
    g = torch.Generator().manual_seed(rows * 7 + K)
    x = torch.randn((rows, K), generator=g) * torch.exp(2 * torch.randn(K, generator=g))
    x = x.to(dtype)
    x[0, :128] = 0  # (part of) a block of zeros
    q, s = _quantize(x, block, kind)
    want_q, e = ref.quantize(x, block)
    assert torch.equal(_bits(q), want_q.view(torch.uint8))
    assert torch.equal(s.cpu(), _expected_scale(e, kind))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["f32", "e8m0"])
def test_quantize_borders(dtype, kind):
    # one block per row: the border of a power of two, its neighbours, the ends of the range,
    # values far below the block's largest, ties between e4m3 values, zeros of both signs
    big = float(torch.finfo(dtype).max)
    eps = float(torch.finfo(dtype).eps)
    tops = [448.0, 448.0 * (1 + 2 * eps), 447.0, 449.0, 3.5, 3.5 * (1 + 2 * eps), 1.0, 224.0,
            2.0 ** -120, 2.0 ** -126, 2.0 ** -130, 2.0 ** 100, big, 448 * 2.0 ** -126,
            450 * 2.0 ** -126, 0.0, -0.0]
    x = torch.zeros((len(tops), 128), dtype=dtype)
    for i, t in enumerate(tops):
        x[i] = torch.linspace(-1, 1, 128).mul(t).to(dtype) if np.isfinite(t * 2) else t
        x[i, 5] = t
        x[i, 7] = -0.0
        x[i, 9] = t * 17 / 256   # halfway between two e4m3 values for t a power of two
        x[i, 11] = t * 2.0 ** -18  # below half the least e4m3 step
    q, s = _quantize(x, 1, kind)
    want_q, e = ref.quantize(x, 1)
    assert torch.equal(_bits(q), want_q.view(torch.uint8))
    assert torch.equal(s.cpu(), _expected_scale(e, kind))


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_quantize_non_finite_block_is_all_nan(bad, block, kind):
    x = torch.randn((256, 384), generator=torch.Generator().manual_seed(3))
    x[130, 200] = bad
    q, s = _quantize(x, block, kind)
    want_q, e = ref.quantize(torch.where(torch.isfinite(x), x, torch.zeros_like(x)), block)
    want_q = want_q.view(torch.uint8).clone()
    r0, r1 = (130, 131) if block == 1 else (128, 256)
    want_q[r0:r1, 128:256] = 0x7F
    assert torch.equal(_bits(q), want_q)
    s = s.cpu()
    at = (130 // block, 1)
    assert torch.isnan(ref.scale_values(s)[at])
    want_s = _expected_scale(e, kind)
    s[at] = want_s[at]
    assert torch.equal(s, want_s)


def test_quantize_refuses_other_layouts():
    x = torch.zeros((128, 256), device="cuda")
    q = torch.empty((128, 256), dtype=torch.uint8, device="cuda")
    s = torch.empty((128, 2), device="cuda")
    with pytest.raises(ValueError):  # not contiguous
        moe.quantize(torch.zeros((256, 128), device="cuda").t(), 1, moe.MOE_SCALE_F32, q, s)
    with pytest.raises(ValueError):  # scale of another shape
        moe.quantize(x, 128, moe.MOE_SCALE_F32, q, s)
    with pytest.raises(ValueError):  # scale of another type
        moe.quantize(x, 1, moe.MOE_SCALE_E8M0, q, s)
    with pytest.raises(ValueError):  # on the host
        moe.quantize(x.cpu(), 1, moe.MOE_SCALE_F32, q, s)
    with pytest.raises(ValueError):
        moe.quantize(x.half(), 1, moe.MOE_SCALE_F32, q, s)


# ------------------------------------------------------------------------- grouped product
def _product_case(counts, N, K, kind, seed, slack=0, first=0):
    g = torch.Generator().manual_seed(seed)
    E, R = len(counts), first + sum(counts) + slack
    return {
        "xq": ref.random_e4m3((R, K), g), "xs": ref.random_scales((R, K // 128), g, kind, 1 / 112),
        "wq": ref.random_e4m3((E, N, K), g),
        "ws": ref.random_scales((E, N // 128, K // 128), g, kind, 1 / (112 * K ** 0.5)),
        "offsets": ref.offsets_of(counts, first), "R": R, "E": E, "N": N, "K": K, "kind": kind}


SENTINEL = 12345.0


def _run_product(c, offsets="given", workspace=None, y=None):
    gs = moe.group_shape(c["R"], c["E"], c["N"], c["K"], moe.MOE_BF16, ref.SCALES[c["kind"]])
    if y is None:
        y = torch.full((c["R"], c["N"]), SENTINEL, dtype=torch.bfloat16, device="cuda")
    if workspace is None:
        workspace = torch.empty(moe.group_workspace_size(gs), dtype=torch.uint8, device="cuda")
    off = c["offsets"].cuda() if offsets == "given" else offsets
    moe.grouped_gemm_fp8(gs, c["xq"].cuda(), c["xs"].cuda(), off, c["wq"].cuda(),
                         c["ws"].cuda(), workspace, y)
    return y.cpu()


def _check_product(c, y, skip_rows=()):
    off = c["offsets"].tolist()
    yd = y.double()
    worst = 0.0
    for e, (a, b) in enumerate(zip(off, off[1:])):
        if a == b:
            continue
        x = ref.dequantize(c["xq"][a:b], c["xs"][a:b], 1)
        w = ref.dequantize(c["wq"][e], c["ws"][e], 128)
        want, err = ref.product(x, w)
        tol = HALF_BF16 * (want.abs() + err) + err
        worst = max(worst, float(((yd[a:b] - want).abs() / tol).max()))
    assert worst <= 1.0, worst
    sent = torch.tensor(SENTINEL, dtype=torch.bfloat16)
    assert bool((y[:off[0]] == sent).all()) and bool((y[off[-1]:] == sent).all())


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("counts,N,K", [
    ([1], 128, 128),                       # one row, one block
    ([0, 0, 1, 0], 256, 128),              # experts without rows
    ([3, 16, 17, 0, 33, 48, 49, 64], 128, 384),   # every count of 16-row tiles, edges
    ([100, 1, 0, 2, 5, 7, 3, 1], 384, 1152),      # more than one row tile, odd column tiles
    ([37], 1152, 2048),                    # few blocks: reduction split over waves
    ([5, 1], 128, 640),                    # fewer steps than the split
    ([65, 80], 256, 256),                  # the 128-row tile
    ([127, 128, 1, 0], 384, 512),
    ([129, 255, 256, 257, 0, 511], 640, 384),     # the 256-row tile and its shorter last tiles
    ([513], 128, 4096),
    ([700, 30, 3, 0], 2176, 256),
    ([65, 100, 0, 90], 384, 4224),         # few, long tiles: reductions in pieces
    ([300, 128, 129, 1], 640, 4096),
    ([33] * 3 + [0] * 60 + [50] * 6, 256, 4096),
    ([65, 100, 0, 90], 384, 6272), ([300, 128, 129, 1], 640, 6272),
    ([33] * 3 + [0] * 60 + [50] * 6, 256, 6272),
    ([2, 0, 1, 3] * 16, 256, 256),         # as many experts as lanes, and one more
    ([2, 0, 1, 3] * 16 + [70], 128, 256),
    ([0] * 1000 + [5] * 24, 128, 128),
    ([3], 128, 65536),                     # a long reduction
])
def test_grouped_product(counts, N, K, kind):
    c = _product_case(counts, N, K, kind, seed=sum(counts) + N, slack=3)
    _check_product(c, _run_product(c))


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("counts,N,K", [
    ([256], 1024, 4096), ([80], 2048, 4224), ([1000], 1152, 5120), ([70, 0, 66], 384, 4096),
    ([200, 1, 300], 640, 4224),
    ([4200], 5120, 4096)])  # 340 tiles: a whole round, then pieces
def test_few_tiles_in_pieces(counts, N, K, kind):
    c = _product_case(counts, N, K, kind, seed=N + K, slack=3)
    _check_product(c, _run_product(c))


def test_grouped_product_many_experts():
    g = torch.Generator().manual_seed(11)
    counts = torch.randint(0, 20, (256,), generator=g).tolist()
    c = _product_case(counts, 512, 384, "e8m0", seed=5)
    _check_product(c, _run_product(c))


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("counts,N,K", [
    # more than 256 tiles: blocks go on to a second and third tile, of other heights, experts and
    # columns.  Tiles of 64, 128 and 256 rows, found from the offsets and (65 experts) a table
    ([20, 64, 0, 9, 1], 25728, 256), ([20, 64, 0, 9, 1], 33024, 384),
    ([65, 100, 0, 90], 25728, 384), ([1, 128, 70], 33024, 256),
    ([300, 129, 0, 513], 15488, 384), ([700, 5, 257], 17664, 256),
    ([3, 17, 0, 1, 64] * 13, 2176, 384), ([60, 0, 70, 128, 1] * 13, 2176, 256),
    ([300, 1, 0, 257, 129] * 13, 1152, 256),
    # a round of whole tiles, then a short one in pieces
    ([4200, 0, 9000], 1152, 6272), ([40, 64] * 8, 4224, 6272), ([40, 20] * 8, 4224, 6272),
    ([128, 100, 20] * 9, 2688, 6144),
])
def test_blocks_that_work_through_several_tiles(counts, N, K, kind):
    c = _product_case(counts, N, K, kind, seed=sum(counts) + N, slack=3, first=2)
    y = _run_product(c)
    on_gpu = {k: v.cuda() if torch.is_tensor(v) else v for k, v in c.items()}  # large in 64 bits
    _check_product(on_gpu, y.cuda())


@pytest.mark.parametrize("rows", [1, 40, 300])
def test_dense_product_without_offsets(rows):
    c = _product_case([rows], 256, 384, "f32", seed=rows)
    y = _run_product(c, offsets=None)
    _check_product(c, y)
    assert torch.equal(y, _run_product(c))


def test_rows_before_the_first_expert_are_left():
    c = _product_case([20, 0, 45], 256, 256, "e8m0", seed=4, slack=70, first=9)
    _check_product(c, _run_product(c))


@pytest.mark.parametrize("rows", [24, 200, 600])
@pytest.mark.parametrize("kind", ["f32", "e8m0"])
def test_nan_stays_in_its_row_and_column(rows, kind):
    c = _product_case([rows, rows // 2], 256, 384, kind, seed=rows)
    clean = _run_product(c)
    c["xq"].view(torch.uint8)[3, 130] = 0x7F
    nan_scale = float("nan") if kind == "f32" else 255
    c["xs"][5, 2] = nan_scale
    c["ws"][1, 1, 0] = nan_scale
    y = _run_product(c)
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[3], bad[5], bad[rows:, 128:] = True, True, True
    assert bool(torch.isnan(y[bad]).all())
    assert torch.equal(y[~bad], clean[~bad])


@pytest.mark.parametrize("counts,N,K", [
    ([24, 7], 256, 384),                       # the reduction over a block's waves
    ([20, 32, 9], 16512, 384),                 # tiles of 64, 128 and 256 rows
    ([70, 90], 384, 640), ([200, 300, 65], 256, 512),
    ([65, 100, 90], 384, 6272),                # a reduction in pieces
    # blocks that go on from a tile computed twice to others, 64, 128 and 256 rows high
    ([20, 64, 9], 25728, 384), ([66, 100, 90], 25728, 256), ([300, 129, 400], 16768, 256)])
def test_fp32_scales_whose_product_is_past_the_range(counts, N, K):
    c = _product_case(counts, N, K, "f32", seed=N + K)
    clean = _run_product(c)
    a, b = counts[0], K // 128
    # expert 1, its second block of columns and of the reduction: 2^30 for the weights.  Rows of
    # 2^98 there: zeros, and one value of 2^-9, so that the sums stay below 448 * 2^119; a
    # negative scale that is no power of two.
    c["ws"][1, 1, 1] = 2.0 ** 30
    for row, scale, value in ((a + 1, 2.0 ** 100, 0.0), (a + 2, 2.0 ** 98, 2.0 ** -9),
                              (a + 3, -1.37 * 2.0 ** 97, -2.0 ** -9)):
        c["xs"][row, 1] = scale
        c["xq"][row, 128:256] = 0
        c["xq"][row, 128 + 17] = value
    # a row of small values: products below 2^-126 are rounded at 2^-149, times 2^24.7 at most
    c["xs"][a + 4] = 2.0 ** -120
    y = _run_product(c)
    off = c["offsets"].tolist()
    for e, (r0, r1) in enumerate(zip(off, off[1:])):
        x = ref.dequantize(c["xq"][r0:r1], c["xs"][r0:r1], 1)
        w = ref.dequantize(c["wq"][e], c["ws"][e], 128)
        want, err = ref.product(x, w)
        err = err + b * 2.0 ** -125
        tol = HALF_BF16 * (want.abs() + err) + err
        assert bool(((y[r0:r1].double() - want).abs() <= tol).all()), e
    # what has other scales is the same bit for bit
    rows = torch.ones(c["R"], dtype=torch.bool)
    rows[a:off[2]] = False
    assert torch.equal(y[rows], clean[rows])
    rows[a:off[2]] = True
    rows[a + 1:a + 5] = False
    assert torch.equal(y[rows][:, :128], clean[rows][:, :128])
    assert torch.equal(y[rows][:, 256:], clean[rows][:, 256:])


@pytest.mark.parametrize("T,E", [(20, 4), (300, 4), (600, 2)])
def test_experts_rows_of_zeros_under_scales_past_the_range(T, E):
    # rows whose one value meets weights of zero: the same as rows of zeros, though the scales'
    # product is 2^130 and more
    c = _ffn_case(T, E, 1, 256, 256, "f32", seed=T)
    rows = [3, T - 1]
    c["x"][rows] = 0
    for n in ("wg", "wu"):
        c[n][0][:, :, 5] = 0
        c[n][1][:, :, 0] = 2.0 ** 40
    want, _ = _run_ffn(c)
    c["x"][rows, 5] = 1.5 * 2.0 ** 99
    got, _ = _run_ffn(c)
    assert bool(torch.isfinite(want.float()).all())
    assert torch.equal(got, want)


def test_product_of_zero_rows():
    gs = moe.group_shape(0, 4, 128, 128)
    ws = torch.empty(moe.group_workspace_size(gs), dtype=torch.uint8, device="cuda")
    e = lambda *s, d=torch.uint8: torch.empty(s, dtype=d, device="cuda")  # noqa: E731
    moe.grouped_gemm_fp8(gs, e(0, 128), e(0, 1, d=torch.float32),
                         torch.zeros(5, dtype=torch.int32, device="cuda"), e(4, 128, 128),
                         e(4, 1, 1, d=torch.float32), ws, e(0, 128, d=torch.bfloat16))


def test_product_is_deterministic_and_replays_in_a_graph():
    c = _product_case([37, 300, 0, 5], 384, 1152, "e8m0", seed=9)
    want = _run_product(c)
    gs = moe.group_shape(c["R"], c["E"], c["N"], c["K"], moe.MOE_BF16, moe.MOE_SCALE_E8M0)
    ws = torch.empty(moe.group_workspace_size(gs), dtype=torch.uint8, device="cuda")
    dev = {k: c[k].cuda() for k in ("xq", "xs", "wq", "ws", "offsets")}
    y = torch.full((c["R"], c["N"]), SENTINEL, dtype=torch.bfloat16, device="cuda")
    call = lambda: moe.grouped_gemm_fp8(  # noqa: E731
        gs, dev["xq"], dev["xs"], dev["offsets"], dev["wq"], dev["ws"], ws, y)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        y.fill_(SENTINEL)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.cpu(), want)
    # other offsets in the same buffer: the graph reads them on the device
    other = dict(c, offsets=ref.offsets_of([1, 40, 290, 11]))
    dev["offsets"].copy_(other["offsets"])
    y.fill_(SENTINEL)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y.cpu(), _run_product(other))


def test_two_products_at_once_on_two_streams():
    cases = [_product_case([40, 200], 512, 1024, "f32", seed=1),
             _product_case([9, 3, 0, 1], 1024, 512, "e8m0", seed=2)]
    want = [_run_product(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    made = []
    for c in cases:
        gs = moe.group_shape(c["R"], c["E"], c["N"], c["K"], moe.MOE_BF16,
                             ref.SCALES[c["kind"]])
        made.append((gs, [c[k].cuda() for k in ("xq", "xs", "offsets", "wq", "ws")],
                     torch.empty(moe.group_workspace_size(gs), dtype=torch.uint8, device="cuda"),
                     torch.full((c["R"], c["N"]), SENTINEL, dtype=torch.bfloat16,
                                device="cuda")))
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (gs, t, ws, y) in zip(streams, made):
            moe.grouped_gemm_fp8(gs, t[0], t[1], t[2], t[3], t[4], ws, y, stream=s)
    torch.cuda.synchronize()
    for (gs, t, ws, y), w in zip(made, want):
        assert torch.equal(y.cpu(), w)


# ----------------------------------------------------------------------- experts' network
def _region(workspace, layout, name, dtype, shape, skip=0):
    n = int(np.prod(shape)) * torch.tensor([], dtype=dtype).element_size()
    at = layout[name] + skip
    return workspace[at:at + n].view(dtype).view(shape).cpu()


def _align(n):
    return (n + 255) // 256 * 256


def _ffn_case(T, E, k, d, F, kind, seed, gathered=True, counts=None):
    g = torch.Generator().manual_seed(seed)
    chosen = torch.rand((T, E), generator=g).topk(k, dim=1).indices.reshape(-1)
    order = torch.argsort(chosen, stable=True)
    if counts is None:
        counts = torch.bincount(chosen, minlength=E).tolist()
    x = torch.randn((T, d), generator=g).to(torch.bfloat16)
    src = (order // k).to(torch.int32)
    c = {"x": x if gathered else x[src.long()].contiguous(), "src": src if gathered else None,
         "rows": x[src.long()], "offsets": ref.offsets_of(counts), "kind": kind,
         "shape": moe.shape(T, d, E, k, F)}
    for n, o, i in (("wg", F, d), ("wu", F, d), ("wd", d, F)):
        c[n] = (ref.random_e4m3((E, o, i), g),
                ref.random_scales((E, o // 128, i // 128), g, kind, 1 / (112 * i ** 0.5)))
    return c


def _run_ffn(c, workspace=None):
    s, kind = c["shape"], ref.SCALES[c["kind"]]
    R = moe.max_rows(s)
    if workspace is None:
        workspace = torch.empty(moe.fp8_workspace_size(s, kind), dtype=torch.uint8,
                                device="cuda")
    y = torch.full((R, s.d), SENTINEL, dtype=torch.bfloat16, device="cuda")
    cuda = lambda p: tuple(t.cuda() for t in p)  # noqa: E731
    moe.expert_ffn_fp8(s, kind, c["x"].cuda(), None if c["src"] is None else c["src"].cuda(),
                       c["offsets"].cuda(), cuda(c["wg"]), cuda(c["wu"]), cuda(c["wd"]),
                       workspace, y)
    torch.cuda.synchronize()
    return y.cpu(), workspace


def _check_ffn(c):
    """Each step from what the one before it left: the quantized rows and h are read from the
    workspace, so that a rounding to 8 bits near a tie does not blur the next step's check."""
    s, kind = c["shape"], ref.SCALES[c["kind"]]
    y, ws = _run_ffn(c)
    lay = moe.fp8_workspace_layout(s, kind)
    R, d, F = moe.max_rows(s), s.d, s.F
    sdt = torch.float32 if c["kind"] == "f32" else torch.uint8
    nx = c["x"].shape[0]
    xq = _region(ws, lay, "x_perm", torch.float8_e4m3fn, (nx, d))
    xs = _region(ws, lay, "x_perm", sdt, (nx, d // 128), _align(max(s.T, R) * d))
    want_q, e = ref.quantize(c["x"], 1)
    assert torch.equal(xq.view(torch.uint8), want_q.view(torch.uint8))
    assert torch.equal(xs, _expected_scale(e, c["kind"]))
    hq = _region(ws, lay, "h", torch.float8_e4m3fn, (R, F))
    hs = _region(ws, lay, "h", sdt, (R, F // 128), _align(R * F))
    off = c["offsets"].tolist()
    xd = ref.dequantize(xq, xs, 1)
    if c["src"] is not None:
        xd = xd[c["src"].long()]
    worst_h = worst_y = 0.0
    for ex, (a, b) in enumerate(zip(off, off[1:])):
        if a == b:
            continue
        gate, eg = ref.product(xd[a:b], ref.dequantize(c["wg"][0][ex], c["wg"][1][ex], 128))
        up, eu = ref.product(xd[a:b], ref.dequantize(c["wu"][0][ex], c["wu"][1][ex], 128))
        silu = gate * torch.sigmoid(gate)
        h = silu * up
        # silu' is at most 1.1; exp, the reciprocal and three products within 2^-20 of the value
        # (the exponential's argument, up to 90, is rounded to 2^-24 of itself)
        err = 1.1 * eg * (up.abs() + eu) + silu.abs() * eu + 2.0 ** -16 * h.abs()
        got = ref.dequantize(hq[a:b], hs[a:b], 1)
        step = ref.scale_values(hs[a:b]).repeat_interleave(128, 1)
        # a value is at most 448 steps of its scale, and the scale the least such power of two
        amax = h.abs().view(b - a, F // 128, 128).amax(2)
        emax = err.view(b - a, F // 128, 128).amax(2)
        sv = ref.scale_values(hs[a:b])
        assert bool((amax - emax <= 448 * sv).all())
        assert bool((amax + emax > 224 * sv).all() or bool((sv == 2.0 ** -126).any()))
        tol = 2.0 ** -4 * (h.abs() + err) + err + 2.0 ** -10 * step
        worst_h = max(worst_h, float(((got - h).abs() / tol).max()))
        want, ey = ref.product(got, ref.dequantize(c["wd"][0][ex], c["wd"][1][ex], 128))
        tol = HALF_BF16 * (want.abs() + ey) + ey
        worst_y = max(worst_y, float(((y[a:b].double() - want).abs() / tol).max()))
    assert worst_h <= 1.0 and worst_y <= 1.0, (worst_h, worst_y)
    assert bool((y[off[-1]:] == SENTINEL).all()) or off[-1] == R
    return y


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("T,E,k,d,F", [
    (1, 4, 1, 128, 128), (1, 8, 8, 256, 384), (37, 8, 2, 384, 640), (64, 8, 2, 128, 256),
    (100, 4, 2, 512, 384), (333, 3, 2, 256, 896), (700, 2, 1, 640, 256), (130, 64, 6, 256, 128)])
def test_expert_ffn_fp8(T, E, k, d, F, kind):
    _check_ffn(_ffn_case(T, E, k, d, F, kind, seed=T + F))


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("gathered", [True, False])
@pytest.mark.parametrize("T,E,k,d,F", [
    # gate and up in more than 256 tiles of 64, 128 and 256 rows: the next tile's sources and
    # weights are asked for during the epilogue.  (F / 128 column tiles for each row tile)
    (40, 4, 2, 128, 11392), (230, 5, 1, 256, 9600), (700, 2, 1, 128, 8576),
    (330, 66, 2, 128, 640)])
def test_experts_that_work_through_several_tiles(T, E, k, d, F, kind, gathered):
    _check_ffn(_ffn_case(T, E, k, d, F, kind, seed=T + F, gathered=gathered))


@pytest.mark.parametrize("T", [20, 400])
def test_expert_ffn_fp8_on_packed_rows_equals_gathered(T):
    a = _ffn_case(T, 4, 2, 256, 384, "e8m0", seed=8)
    b = _ffn_case(T, 4, 2, 256, 384, "e8m0", seed=8, gathered=False)
    assert torch.equal(_check_ffn(a), _check_ffn(b))


def test_expert_ffn_fp8_leaves_rows_behind_the_last():
    # capacity drops: the offsets end before the row slots do
    c = _ffn_case(50, 4, 2, 256, 128, "f32", seed=2, counts=[10, 0, 33, 5])
    y = _check_ffn(c)
    assert bool((y[48:] == SENTINEL).all())


def test_expert_ffn_fp8_reads_a_row_for_an_empty_slot():
    # sources outside [0, T) stay in bounds and do not touch other rows
    c = _ffn_case(40, 4, 2, 256, 128, "e8m0", seed=6)
    want, _ = _run_ffn(c)
    c["src"][7], c["src"][30] = -1, 2 ** 31 - 1
    y, _ = _run_ffn(c)
    keep = torch.ones(80, dtype=torch.bool)
    keep[7] = keep[30] = False
    assert torch.equal(y[keep], want[keep])


# ---------------------------------------------------------------------------------- layer
def _layer_case(w, flags=0, kind="e8m0", n_groups=0, topk_groups=0):
    C = moe.capacity(w.T, w.k, w.E, w.capacity_factor)
    s = moe.shape(w.T, w.d, w.E, w.k, w.F, C, moe.MOE_BF16, flags, n_groups, topk_groups)
    dev = {n: mi.device_tensor(w, n) for n in ("x", "w_router", "w_gate", "w_up", "w_down")}
    b = mi.router_bias(w)
    dev["b"] = None if b is None else torch.from_numpy(b).cuda()
    lay = moe.MoELayerFp8(s, ref.SCALES[kind])
    q = [lay.quantize_weights(dev[n]) for n in ("w_gate", "w_up", "w_down")]
    return s, dev, lay, q


def _composed(s, dev, q, kind):
    """The layer as its public steps: route, dispatch, the experts, combine."""
    T, E, k, d = s.T, s.E, s.k, s.d
    R = moe.max_rows(s)
    i32 = dict(dtype=torch.int32, device="cuda")
    logits = torch.empty((T, E), device="cuda")
    idx, gates = torch.empty((T, k), **i32), torch.empty((T, k), device="cuda")
    moe.route(s, dev["x"], dev["w_router"], dev["b"], logits, idx, gates)
    routed, kept, off = torch.empty(E, **i32), torch.empty(E, **i32), torch.empty(E + 1, **i32)
    src, dest, drops = torch.empty(R, **i32), torch.empty((T, k), **i32), torch.empty(k + 2, **i32)
    moe.dispatch_no_workspace(s, idx, None, routed, kept, off, src, dest, drops, None)
    ws = torch.empty(moe.fp8_workspace_size(s, kind), dtype=torch.uint8, device="cuda")
    y = torch.empty((R, d), dtype=torch.bfloat16, device="cuda")
    moe.expert_ffn_fp8(s, kind, dev["x"], src, off, q[0], q[1], q[2], ws, y)
    out = torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
    moe.combine(s, y, dest, gates, out)
    return out, drops, kept


LAYERS = {
    "decode": (mi.Workload("fp8_decode", 40, 256, 16, 4, 384, None, "bf16"), 0),
    "capacity": (mi.Workload("fp8_cap", 200, 256, 8, 2, 384, 1.0, "bf16", 0.5), 0),
    "padded": (mi.Workload("fp8_pad", 100, 256, 8, 2, 256, 1.25, "bf16", 0.5),
               moe.MOE_FLAG_PAD_TO_CAPACITY),
    "slot major": (mi.Workload("fp8_slot", 300, 128, 4, 2, 256, 1.0, "bf16", 0.5),
                   moe.MOE_FLAG_SLOT_MAJOR),
    "one token": (mi.Workload("fp8_one", 1, 128, 4, 1, 128, None, "bf16"), 0),
    "grouped": (mi.Workload("fp8_grp", 90, 128, 80, 4, 128, None, "bf16", 0.5),
                moe.MOE_FLAG_BIAS_SELECTION_ONLY),
    "tall": (mi.Workload("fp8_tall", 1500, 256, 4, 2, 384, 1.25, "bf16"), 0),
}


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("name", list(LAYERS))
def test_layer_fp8_equals_its_steps(name, kind):
    w, flags = LAYERS[name]
    groups = (4, 2) if name == "grouped" else (0, 0)
    s, dev, lay, q = _layer_case(w, flags, kind, *groups)
    out = lay(dev["x"], dev["w_router"], dev["b"], *q).clone()
    want, drops, kept = _composed(s, dev, q, ref.SCALES[kind])
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert torch.equal(lay.drops, drops) and torch.equal(lay.tokens_per_expert, kept)
    # and near the bf16 layer on the same routing: e4m3 weights, activations and hidden rows
    # each carry at most 2^-4 of a value, which over sums of random signs is some 7 % of the norm
    bf = moe.MoELayer(s)
    ref_out = bf(dev["x"], dev["w_router"], dev["b"], dev["w_gate"], dev["w_up"], dev["w_down"])
    rel = float((out.float() - ref_out.float()).norm() / ref_out.float().norm())
    log(f"layer_fp8 {name} {kind}: {rel:.3f} of the bf16 layer's norm")
    assert rel < 0.125


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("E,T,k,d,F", [(4, 64, 2, 4096, 2048), (8, 100, 2, 2048, 2304),
                                       (1, 37, 1, 7168, 4096), (64, 20, 2, 256, 2048),
                                       (65, 20, 2, 256, 2048)])
def test_layer_fp8_adds_in_its_steps_order(E, T, k, d, F, kind):
    # few tokens and reductions of 16 to 32 steps, which the down product spreads over the waves
    # of a block: the layer and its steps have to choose the same kernel.  Block scales far apart
    # (and no powers of two, where the type has others) make sums that fp32 has to round, so that
    # another order shows, in a few of the many values.
    w = mi.Workload(f"fp8_few{E}", T, d, E, k, F, None, "bf16")
    s, dev, lay, q = _layer_case(w, 0, kind)
    g = torch.Generator().manual_seed(E)
    if kind == "f32":
        q[2][1].mul_(torch.exp(torch.randn(q[2][1].shape, generator=g)).cuda())
    else:
        q[2][1].add_(torch.randint(-6, 7, q[2][1].shape, generator=g).to(torch.int8).cuda())
    out = lay(dev["x"], dev["w_router"], dev["b"], *q).clone()
    want, _, _ = _composed(s, dev, q, ref.SCALES[kind])
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_two_layers_at_once_on_two_streams():
    cases = [_layer_case(LAYERS[n][0], LAYERS[n][1]) for n in ("decode", "tall")]
    want = [lay(dev["x"], dev["w_router"], dev["b"], *q).clone() for _, dev, lay, q in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(4):
        for st, (_, dev, lay, q) in zip(streams, cases):
            lay(dev["x"], dev["w_router"], dev["b"], *q, stream=st)
    torch.cuda.synchronize()
    for (_, _, lay, _), o in zip(cases, want):
        assert torch.equal(lay.out, o)


def test_layer_fp8_of_no_tokens():
    w = mi.Workload("fp8_none", 1, 128, 4, 2, 128, None, "bf16")
    s, dev, lay, q = _layer_case(w)
    empty = moe.MoELayerFp8(moe.shape(0, 128, 4, 2, 128), moe.MOE_SCALE_E8M0)
    empty.drops.fill_(7)
    empty(dev["x"][:0], dev["w_router"], None, *q)
    torch.cuda.synchronize()
    assert empty.drops.tolist() == [0] * 4


def test_layer_fp8_replays_in_a_graph():
    w, flags = LAYERS["capacity"]
    s, dev, lay, q = _layer_case(w, flags)
    want = lay(dev["x"], dev["w_router"], dev["b"], *q).clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lay(dev["x"], dev["w_router"], dev["b"], *q)
    for i in range(3):
        lay.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(lay.out, want), i
        dev["x"] += 0  # the program's own eager work between replays
    x2 = dev["x"].flip(0).contiguous()
    dev["x"].copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    got = lay.out.clone()
    assert torch.equal(got, lay(x2, dev["w_router"], dev["b"], *q))
