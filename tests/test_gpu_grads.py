"""Gradients of the products grouped by expert against their 64-bit forms, differences and, as a
whole network, autograd."""
import pytest
import torch

import routing_expert_ffn_router_amd as moe
from _fp8 import offsets_of

pytestmark = pytest.mark.gpu

SENTINEL = 777.0
DTYPES = {"bf16": (torch.bfloat16, moe.MOE_BF16, 2.0 ** -8),
          "f32": (torch.float32, moe.MOE_F32, 2.0 ** -24)}


def _case(counts, N, K, dtype, seed, slack=0, first=0):
    g = torch.Generator().manual_seed(seed)
    dt = DTYPES[dtype][0]
    E, R = len(counts), first + sum(counts) + slack
    c = {"dy": torch.randn((R, N), generator=g).to(dt), "x": torch.randn((R, K), generator=g).to(dt),
         "w": (torch.randn((E, N, K), generator=g) / N ** 0.5).to(dt),
         "offsets": offsets_of(counts, first), "R": R, "E": E, "N": N, "K": K, "dtype": dtype}
    # rows that belong to no expert hold anything at all
    for n in ("dy", "x"):
        c[n][:first] = float("nan")
        c[n][first + sum(counts):] = float("inf")
    return c


def _shape(c):
    gs = moe.group_shape(c["R"], c["E"], c["N"], c["K"], DTYPES[c["dtype"]][1])
    return gs, torch.empty(moe.group_workspace_size(gs), dtype=torch.uint8, device="cuda")


def _dgrad(c, offsets="given"):
    gs, ws = _shape(c)
    dx = torch.full((c["R"], c["K"]), SENTINEL, dtype=DTYPES[c["dtype"]][0], device="cuda")
    off = c["offsets"].cuda() if isinstance(offsets, str) else offsets
    moe.grouped_dgrad(gs, c["dy"].cuda(), off, c["w"].cuda(), ws, dx)
    return dx.cpu()


def _wgrad(c, offsets="given"):
    gs, ws = _shape(c)
    dw = torch.full((c["E"], c["N"], c["K"]), float("nan"), dtype=DTYPES[c["dtype"]][0],
                    device="cuda")
    off = c["offsets"].cuda() if isinstance(offsets, str) else offsets
    moe.grouped_wgrad(gs, c["dy"].cuda(), c["x"].cuda(), off, ws, dw)
    return dw.cpu()


def _within(got, a, b, half):
    """got against a @ b: one rounding of the value, and one of 2^-24 for each of the terms'
    products and additions."""
    want = a @ b
    err = (a.shape[1] + 1) * 2.0 ** -24 * (a.abs() @ b.abs())
    return float(((got.double() - want).abs() - half * (want.abs() + err) - err).max()) <= 0


CASES = [
    ([1], 128, 128), ([0, 1, 0], 128, 256), ([2, 0, 31, 32, 33], 384, 128),
    ([63, 64, 65, 0], 128, 384), ([127, 128, 129], 256, 256), ([300, 5, 0, 257], 384, 640),
    ([700], 640, 384), ([1, 2, 3, 0, 0, 0, 4, 190], 256, 1152),
    ([300, 0, 129, 5], 2176, 384), ([20, 31, 1] + [0] * 62 + [40], 2048, 128),
    ([1, 0, 2, 3] * 16, 128, 128), ([2, 0, 7, 1], 6272, 384), ([300, 0, 129, 5], 6272, 384),
    ([20, 31, 1] + [0] * 62 + [40], 6272, 128), ([0] * 1000 + [2] * 24, 128, 128),
    ([5], 32768, 128), ([40], 128, 32768)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("counts,N,K", CASES)
def test_dgrad(counts, N, K, dtype):
    c = _case(counts, N, K, dtype, seed=N + sum(counts), slack=3, first=2)
    dx = _dgrad(c)
    off = c["offsets"].tolist()
    for e, (a, b) in enumerate(zip(off, off[1:])):
        if b > a:
            assert _within(dx[a:b], c["dy"][a:b].double(), c["w"][e].double(),
                           DTYPES[dtype][2]), e
    assert bool((dx[:off[0]] == SENTINEL).all()) and bool((dx[off[-1]:] == SENTINEL).all())


@pytest.mark.parametrize("counts,N,K", [
    ([256], 4096, 2048), ([9], 2048, 1152), ([257], 2176, 384), ([1000], 2048, 5120),
    ([60, 0, 9], 2048, 512), ([0, 300, 1, 20], 4224, 640),
    ([4200], 2048, 5120)])  # 340 tiles: a whole round, then pieces
def test_dgrad_of_few_tiles_in_pieces(counts, N, K):
    c = _case(counts, N, K, "bf16", seed=N + K + len(counts), slack=3, first=2)
    dx = _dgrad(c)
    off = c["offsets"].tolist()
    for e, (a, b) in enumerate(zip(off, off[1:])):
        if b > a:
            assert _within(dx[a:b].cuda(), c["dy"][a:b].cuda().double(),
                           c["w"][e].cuda().double(), 2.0 ** -8), e
    assert bool((dx[:off[0]] == SENTINEL).all()) and bool((dx[off[-1]:] == SENTINEL).all())


@pytest.mark.parametrize("dtype,counts,N,K", [
    # more than 256 tiles: blocks go on to a second and third one (tiles of 256 and, with few
    # rows, 128 rows; fp32 128), found from the offsets and (65 experts) a table
    ("bf16", [20, 300, 0, 5], 128, 16768), ("bf16", [300, 129, 70], 384, 16896),
    ("bf16", [9, 0, 16, 1, 3], 128, 22912), ("bf16", [1, 300, 0, 257, 20] * 13, 256, 1152),
    ("f32", [20, 300, 0, 5], 128, 8576), ("f32", [130, 1, 70], 384, 11392),
    ("f32", [1, 130, 0, 17, 20] * 13, 128, 1152),
    # a round of whole tiles, then a short one in pieces
    ("bf16", [4200, 0, 9000], 6272, 1152), ("bf16", [1, 12, 3, 16] * 8, 6144, 2432)])
def test_dgrad_blocks_that_work_through_several_tiles(dtype, counts, N, K):
    c = _case(counts, N, K, dtype, seed=N + sum(counts), slack=3, first=2)
    dx = _dgrad(c)
    off = c["offsets"].tolist()
    for e, (a, b) in enumerate(zip(off, off[1:])):
        if b > a:
            assert _within(dx[a:b].cuda(), c["dy"][a:b].cuda().double(),
                           c["w"][e].cuda().double(), DTYPES[dtype][2]), e
    assert bool((dx[:off[0]] == SENTINEL).all()) and bool((dx[off[-1]:] == SENTINEL).all())


@pytest.mark.parametrize("dtype,counts,N,K", [
    # 256 blocks at once (fp32: 512): tiles with rows follow each other, and empty experts between
    ("bf16", [70, 1, 0, 129], 2176, 2944), ("bf16", [300, 64, 65], 2432, 2688),
    ("bf16", [33, 0, 200, 7, 64] * 13, 640, 640),
    ("f32", [70, 1, 0, 129], 1664, 1792), ("f32", [31, 33, 200], 2048, 1920),
    ("f32", [33, 0, 200, 7, 64] * 13, 384, 384)])
def test_wgrad_blocks_that_work_through_several_tiles(dtype, counts, N, K):
    c = _case(counts, N, K, dtype, seed=K + sum(counts), slack=5, first=1)
    dw = _wgrad(c)
    off = c["offsets"].tolist()
    for e, (a, b) in enumerate(zip(off, off[1:])):
        if b == a:
            assert bool((dw[e] == 0).all()), e
        else:
            assert _within(dw[e].cuda(), c["dy"][a:b].cuda().double().t(),
                           c["x"][a:b].cuda().double(), DTYPES[dtype][2]), e


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("counts,N,K", CASES)
def test_wgrad(counts, N, K, dtype):
    c = _case(counts, N, K, dtype, seed=K + sum(counts), slack=5, first=1)
    dw = _wgrad(c)
    off = c["offsets"].tolist()
    for e, (a, b) in enumerate(zip(off, off[1:])):
        if b == a:
            assert bool((dw[e] == 0).all()), e
        else:
            assert _within(dw[e], c["dy"][a:b].double().t(), c["x"][a:b].double(),
                           DTYPES[dtype][2]), e


def test_wgrad_of_no_rows_is_zero():
    gs = moe.group_shape(0, 3, 128, 256, moe.MOE_BF16)
    ws = torch.empty(moe.group_workspace_size(gs), dtype=torch.uint8, device="cuda")
    dw = torch.full((3, 128, 256), SENTINEL, dtype=torch.bfloat16, device="cuda")
    none = torch.empty((0, 128), dtype=torch.bfloat16, device="cuda")
    moe.grouped_wgrad(gs, none, torch.empty((0, 256), dtype=torch.bfloat16, device="cuda"),
                      torch.zeros(4, dtype=torch.int32, device="cuda"), ws, dw)
    assert bool((dw == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dense_gradients_without_offsets(dtype):
    c = _case([150], 256, 384, dtype, seed=1)
    assert torch.equal(_dgrad(c, None), _dgrad(c))
    assert torch.equal(_wgrad(c, None), _wgrad(c))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_values_that_are_not_finite_stay_where_the_formula_has_them(dtype):
    # an infinity of one expert's rows reaches neither its neighbours nor other columns
    c = _case([40, 33, 50], 256, 256, dtype, seed=2)
    dw0, dx0 = _wgrad(c), _dgrad(c)
    c["x"][39, 7] = float("inf")   # the last row of expert 0
    c["dy"][73, 100] = float("nan")  # the first row of expert 2
    dw, dx = _wgrad(c), _dgrad(c)
    bad = torch.zeros_like(dw, dtype=torch.bool)
    bad[0, :, 7], bad[2, 100, :] = True, True
    assert not bool(torch.isfinite(dw[bad]).any())
    assert torch.equal(dw[~bad], dw0[~bad])
    rows = torch.arange(c["R"]) != 73
    assert torch.equal(dx[rows], dx0[rows]) and bool(torch.isnan(dx[73]).all())


def test_gradients_match_differences_of_the_forward_product():
    # y = moe_expert_down(h): the loss sum(c * y) is linear in h and in w, so a difference over
    # any step is its derivative up to roundings
    counts, d, F = [30, 0, 70, 28], 256, 384
    E, R = len(counts), sum(counts)
    c = _case(counts, d, F, "f32", seed=4)
    s = moe.shape(R, d, E, 1, F, 0, moe.MOE_F32)
    ws = torch.empty(moe.workspace_size(s), dtype=torch.uint8, device="cuda")

    def forward(h, w):
        y = torch.zeros((R, d), device="cuda")
        moe.expert_down(s, h.cuda(), c["offsets"].cuda(), w.cuda(), ws, y)
        return y.cpu().double()

    dx, dw = _dgrad(c).double(), _wgrad(c).double()
    g = torch.Generator().manual_seed(9)
    vh, vw = torch.randn((R, F), generator=g), torch.randn((E, d, F), generator=g)
    up = c["dy"].double()
    for grad, diff, terms in (
            (dx * vh.double(), forward(c["x"] + vh, c["w"]) - forward(c["x"] - vh, c["w"]), F),
            (dw * vw.double(), forward(c["x"], c["w"] + vw) - forward(c["x"], c["w"] - vw), F)):
        a, b = float(grad.sum()), float((up * diff).sum()) / 2
        # forward errors: (F + 2) roundings of 2^-24 of sums of magnitudes (|x| + |v|)(|w| + |v|),
        # each about 1: F of them per output, weighted by |dy|
        tol = 2 * (terms + 2) * 2.0 ** -24 * float(up.abs().sum()) * terms * 2
        assert abs(a - b) <= tol, (a, b, tol)


def test_gradients_equal_exact_differences_of_the_forward_product():
    # The loss sum(dy * h W^T) is linear in h and in W, so a difference over any step is its
    # derivative.  Whole numbers of at most 3 keep every product and sum a whole number below 2^24
    # (130 rows or 384 columns of at most 9, steps twice that), which fp32 holds exactly: nothing is
    # rounded on either side, and each row's and each expert's derivative has to be equal.
    counts, d, F = [30, 0, 130, 28], 256, 384
    E, R = len(counts), sum(counts)
    g = torch.Generator().manual_seed(12)
    whole = lambda *s: torch.randint(-3, 4, s, generator=g).float()  # noqa: E731
    c = {"dy": whole(R, d), "x": whole(R, F), "w": whole(E, d, F), "offsets": offsets_of(counts),
         "R": R, "E": E, "N": d, "K": F, "dtype": "f32"}
    vh, vw = whole(R, F), whole(E, d, F)
    s = moe.shape(R, d, E, 1, F, 0, moe.MOE_F32)
    ws = torch.empty(moe.workspace_size(s), dtype=torch.uint8, device="cuda")

    def forward(h, w):
        y = torch.zeros((R, d), device="cuda")
        moe.expert_down(s, h.cuda(), c["offsets"].cuda(), w.cuda(), ws, y)
        return y.cpu().double()

    dx, dw, dy = _dgrad(c).double(), _wgrad(c).double(), c["dy"].double()
    by_h = (dy * (forward(c["x"] + vh, c["w"]) - forward(c["x"] - vh, c["w"]))).sum(1) / 2
    by_w = (dy * (forward(c["x"], c["w"] + vw) - forward(c["x"], c["w"] - vw))).sum(1) / 2
    # (hardly any derivative is zero, so that nothing missing can pass)
    assert int((by_h != 0).sum()) > 0.9 * R
    assert torch.equal((dx * vh.double()).sum(1), by_h)
    off = c["offsets"].tolist()
    want = torch.stack([by_w[a:b].sum() for a, b in zip(off, off[1:])])
    assert torch.equal((dw * vw.double()).sum((1, 2)), want)
    assert int((want != 0).sum()) == 3


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_training_step_of_the_experts_network(dtype):
    """Forward through the framework's grouped products, backward through the gradients, as a
    training step strings them together, against autograd in 64 bits."""
    counts, d, F = [70, 0, 129, 33], 256, 384
    E, R = len(counts), sum(counts)
    dt, mdt, half = DTYPES[dtype]
    g = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    x, dy = rnd(R, d).to(dt), rnd(R, d).to(dt)
    wg, wu, wd = ((rnd(E, F, d) / d ** 0.5).to(dt), (rnd(E, F, d) / d ** 0.5).to(dt),
                  (rnd(E, d, F) / F ** 0.5).to(dt))
    off = offsets_of(counts).cuda()
    X, DY, WG, WU, WD = (t.cuda() for t in (x, dy, wg, wu, wd))
    new = lambda *s: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731

    def forward(a, w, n):  # a W[e]^T: moe_expert_down
        s = moe.shape(R, n, E, 1, a.shape[1], 0, mdt)
        ws = torch.empty(moe.workspace_size(s), dtype=torch.uint8, device="cuda")
        y = new(R, n)
        moe.expert_down(s, a, off, w, ws, y)
        return y

    gate, up = forward(X, WG, F), forward(X, WU, F)
    sg = torch.sigmoid(gate.float())
    h = (gate.float() * sg * up.float()).to(dt)
    y = forward(h, WD, d)
    up_shape, down_shape = moe.group_shape(R, E, F, d, mdt), moe.group_shape(R, E, d, F, mdt)
    ws = torch.empty(max(moe.group_workspace_size(up_shape),
                         moe.group_workspace_size(down_shape)), dtype=torch.uint8, device="cuda")
    dh, dwd = new(R, F), new(E, d, F)
    moe.grouped_dgrad(down_shape, DY, off, WD, ws, dh)
    moe.grouped_wgrad(down_shape, DY, h, off, ws, dwd)
    dhf = dh.float()
    dgate = (dhf * up.float() * sg * (1 + gate.float() * (1 - sg))).to(dt)
    dup = (dhf * gate.float() * sg).to(dt)
    dwg, dwu, dxa, dxb = new(E, F, d), new(E, F, d), new(R, d), new(R, d)
    moe.grouped_wgrad(up_shape, dgate, X, off, ws, dwg)
    moe.grouped_wgrad(up_shape, dup, X, off, ws, dwu)
    moe.grouped_dgrad(up_shape, dgate, off, WG, ws, dxa)
    moe.grouped_dgrad(up_shape, dup, off, WU, ws, dxb)
    torch.cuda.synchronize()

    leaves = [t.double().requires_grad_() for t in (x, wg, wu, wd)]
    lx, lg, lu, ld = leaves
    o = offsets_of(counts).tolist()
    ys = []
    for e, (a, b) in enumerate(zip(o, o[1:])):
        gt = lx[a:b] @ lg[e].t()
        ys.append((gt * torch.sigmoid(gt) * (lx[a:b] @ lu[e].t())) @ ld[e].t())
    ref_y = torch.cat(ys)
    ref_y.backward(dy.double())
    # in the norm: at most six roundings in a row of each value's factors (gate, up, h or dh,
    # dgate / dup, the product), each of at most `half`, and twice that for the factors' slopes;
    # fp32 adds its sums' roundings, at most sqrt(2 F) 2^-24 of the norm each for random signs
    tol = 12 * half if dtype == "bf16" else 12 * half + 6 * (2 * F) ** 0.5 * 2.0 ** -24
    for name, got, want in (("y", y, ref_y.detach()), ("dx", dxa.double() + dxb.double(), lx.grad),
                            ("dwg", dwg, lg.grad), ("dwu", dwu, lu.grad), ("dwd", dwd, ld.grad)):
        rel = float((got.cpu().double() - want).norm() / want.norm())
        assert rel <= tol, (name, rel, tol)
    assert bool((dwg[1] == 0).all()) and bool((dwd[1] == 0).all())


def test_gradients_replay_in_a_graph():
    c = _case([37, 300, 0, 5], 384, 512, "bf16", seed=9)
    gs, ws = _shape(c)
    ws2 = torch.empty_like(ws)
    dev = {k: c[k].cuda() for k in ("dy", "x", "w", "offsets")}
    dx = torch.full((c["R"], c["K"]), SENTINEL, dtype=torch.bfloat16, device="cuda")
    dw = torch.empty((c["E"], c["N"], c["K"]), dtype=torch.bfloat16, device="cuda")

    def both():
        moe.grouped_dgrad(gs, dev["dy"], dev["offsets"], dev["w"], ws, dx)
        moe.grouped_wgrad(gs, dev["dy"], dev["x"], dev["offsets"], ws2, dw)

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    want = _dgrad(c), _wgrad(c)
    for _ in range(3):
        dx.fill_(SENTINEL)
        dw.fill_(SENTINEL)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dx.cpu(), want[0]) and torch.equal(dw.cpu(), want[1])
    other = dict(c, offsets=offsets_of([100, 2, 240, 0]))
    dev["offsets"].copy_(other["offsets"])
    dx.fill_(SENTINEL)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dx.cpu(), _dgrad(other)) and torch.equal(dw.cpu(), _wgrad(other))


def test_offsets_that_decrease_stay_within_the_buffers():
    # two experts that claim all rows: more row tiles than the workspace's slots are laid out for.
    # What such rows get is not defined, but nothing past dx and the workspace is written, the
    # weights' gradients follow the clamped ranges, and a good call after it is right.
    c = _case([1024] * 4, 8192, 256, "bf16", 41)
    bad = torch.tensor([0, 4096, 0, 4096, 0], dtype=torch.int32)
    gs = moe.group_shape(c["R"], c["E"], c["N"], c["K"], moe.MOE_BF16)
    size = moe.group_workspace_size(gs)
    guard = 64 << 20  # as far as 256 slots of 256 KB reach
    ws = torch.full((size + guard,), 0x5A, dtype=torch.uint8, device="cuda")
    dx = torch.full((2 * c["R"], c["K"]), SENTINEL, dtype=torch.bfloat16, device="cuda")
    dy, w = c["dy"].cuda(), c["w"].cuda()
    moe.grouped_dgrad(gs, dy, bad.cuda(), w, ws[:size], dx[:c["R"]])
    assert bool((ws[size:] == 0x5A).all()) and bool((dx[c["R"]:] == SENTINEL).all())
    moe.grouped_dgrad(gs, dy, c["offsets"].cuda(), w, ws[:size], dx[:c["R"]])
    got = dx[:c["R"]].cpu()
    for e in range(4):
        r = slice(1024 * e, 1024 * (e + 1))
        assert _within(got[r], c["dy"][r].double(), c["w"][e].double(), 2.0 ** -8)
    dw = torch.full((c["E"], c["N"], c["K"]), float("nan"), dtype=torch.bfloat16, device="cuda")
    moe.grouped_wgrad(gs, dy, c["x"].cuda(), bad.cuda(), ws[:size], dw)
    dw = dw.cpu()
    for e in range(4):
        if e % 2:
            assert not bool(dw[e].any())
        else:
            assert _within(dw[e], c["dy"].double().T, c["x"].double(), 2.0 ** -8)
