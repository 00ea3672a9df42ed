"""The layer for a few tokens against its 64-bit form."""
import pytest
import torch

import _few as ref
import routing_expert_ffn_router_amd as moe
from _fp8 import SCALES, dequantize, random_e4m3, random_scales

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "f32", "e4m3-f32", "e4m3-e8m0"]


def _case(T, E, k, d, F, kind, seed, bias=True):
    g = torch.Generator().manual_seed(seed)
    dt = torch.float32 if kind == "f32" else torch.bfloat16
    c = {"T": T, "E": E, "k": k, "d": d, "F": F, "kind": kind, "dt": dt,
         "x": torch.randn((T, d), generator=g).to(dt),
         "w_router": (torch.randn((E, d), generator=g) / d ** 0.5).to(dt),
         "b": torch.randn(E, generator=g) * 0.3 if bias else None, "w": [], "exact": []}
    for n, kk in ((F, d), (F, d), (d, F)):
        if kind.startswith("e4m3"):
            q = random_e4m3((E, n, kk), g)
            s = random_scales((E, n // 128, kk // 128), g, kind[5:], 1 / (112 * kk ** 0.5))
            c["w"].append((q, s))
            c["exact"].append(torch.stack([dequantize(q[e], s[e], 128) for e in range(E)]))
        else:
            w = (torch.randn((E, n, kk), generator=g) / kk ** 0.5).to(dt)
            c["w"].append(w)
            c["exact"].append(w.double())
    return c


def _cuda(w):
    return tuple(v.cuda() for v in w) if isinstance(w, tuple) else w.cuda()


def _setup(c, capacity=0, flags=0, groups=(0, 0), ws_byte=255):
    dt = moe.MOE_F32 if c["kind"] == "f32" else moe.MOE_BF16
    s = moe.shape(c["T"], c["d"], c["E"], c["k"], c["F"], capacity, dt, flags, *groups)
    ws = torch.empty(moe.few_workspace_size(s), dtype=torch.uint8, device="cuda").fill_(ws_byte)
    return s, ws, torch.full((c["T"], c["d"]), 777.0, dtype=c["dt"], device="cuda")


def _ints(c):
    return [torch.full((n,), -9, dtype=torch.int32, device="cuda")
            for n in (c["E"], c["E"], c["k"] + 2, 1)]


def _call(c, s, ws, out, ints, args=None, stream=None):
    x, wr, b, w = args or _args(c)
    if c["kind"].startswith("e4m3"):
        moe.layer_few_fp8(s, SCALES[c["kind"][5:]], x, wr, b, *w, ws, out, *ints, stream=stream)
    else:
        moe.layer_few(s, x, wr, b, *w, ws, out, *ints, stream=stream)


def _args(c):
    return (c["x"].cuda(), c["w_router"].cuda(), None if c["b"] is None else c["b"].cuda(),
            [_cuda(w) for w in c["w"]])


def _run(c, capacity=0, flags=0, groups=(0, 0), ws_byte=255):
    s, ws, out = _setup(c, capacity, flags, groups, ws_byte)
    ints = _ints(c)
    _call(c, s, ws, out, ints)
    return out.cpu(), [v.cpu() for v in ints]


def _check(c, got, ints, capacity=0, flags=0, groups=(1, 1)):
    idx, gates, finite, largest = ref.route(c["x"], c["w_router"], c["b"], c["k"],
                                            bool(flags & moe.MOE_FLAG_BIAS_SELECTION_ONLY), groups)
    keep = ref.keep_of(idx, c["E"], capacity, bool(flags & moe.MOE_FLAG_SLOT_MAJOR))
    routed, kept, drops = ref.counts(idx, keep, c["E"])
    assert torch.equal(ints[0], routed) and torch.equal(ints[1], kept)
    assert torch.equal(ints[2], drops) and int(ints[3]) == int((~finite).sum())
    half = 2.0 ** -24 if c["kind"] == "f32" else 2.0 ** -8
    want, bound = ref.experts(c["x"], c["exact"], idx, gates, keep, half, largest)
    over = (got.double() - want).abs() - bound
    assert float(over.max()) <= 0, float(((got.double() - want).abs() / bound).max())
    # and closer than a bound shows: bf16's roundings of h and of the output, at random
    size = float(want.norm())
    if size:
        assert float((got.double() - want).norm()) <= (4e-3 if half > 1e-6 else 4e-6) * size


SHAPES = [(1, 1, 1, 128, 128), (1, 8, 2, 256, 384), (2, 5, 3, 384, 128), (3, 4, 2, 256, 512),
          (5, 16, 4, 640, 256), (8, 7, 7, 128, 640), (9, 3, 1, 384, 384), (13, 64, 6, 256, 128),
          (16, 4, 2, 1152, 256), (16, 8, 8, 128, 128), (7, 130, 8, 128, 128), (11, 6, 2, 256, 1152)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,E,k,d,F", SHAPES)
def test_layer(T, E, k, d, F, kind):
    c = _case(T, E, k, d, F, kind, seed=T * 1000 + E)
    _check(c, *_run(c))


@pytest.mark.parametrize("kind", ["bf16", "e4m3-e8m0"])
@pytest.mark.parametrize("T", [4, 16])
@pytest.mark.parametrize("capacity,flags,groups", [
    (1, 0, (0, 0)), (2, moe.MOE_FLAG_SLOT_MAJOR, (0, 0)), (3, moe.MOE_FLAG_PAD_TO_CAPACITY, (0, 0)),
    (0, moe.MOE_FLAG_BIAS_SELECTION_ONLY, (0, 0)), (0, 0, (4, 2)), (2, 0, (8, 3)),
    (1, moe.MOE_FLAG_SLOT_MAJOR | moe.MOE_FLAG_BIAS_SELECTION_ONLY, (2, 1)), (0, 0, (4, 4))])
def test_routing_variants(T, capacity, flags, groups, kind):
    c = _case(T, 16, 3, 128, 256, kind, seed=capacity + 10 * flags + T)
    c["b"] = c["b"] * 5
    got = _run(c, capacity, flags, groups)
    want = groups if groups[0] > 1 and groups[1] < groups[0] else (1, 1)
    _check(c, *got, capacity, flags, want)


def test_every_token_dropped_but_one():
    c = _case(16, 3, 1, 128, 128, "bf16", seed=3)
    c["b"] = torch.tensor([9.0, 0.0, 0.0]) * 10
    out, ints = _run(c, 1)
    _check(c, out, ints, 1)
    assert int(ints[2][0]) == 15 and bool((out[1:] == 0).all()) and bool((out[0] != 0).any())


@pytest.mark.parametrize("T,E,k", [(16, 1024, 32), (8, 1024, 64), (1, 1000, 64), (16, 300, 3)])
def test_many_experts(T, E, k):
    c = _case(T, E, k, 128, 128, "bf16", seed=E + k)
    got = _run(c)
    idx, gates, _, largest = ref.route(c["x"], c["w_router"], c["b"], k)
    keep = ref.keep_of(idx, E, 0)
    assert torch.equal(got[1][0], ref.counts(idx, keep, E)[0])
    want, bound = ref.experts(c["x"], c["exact"], idx, gates, keep, 2.0 ** -8, largest)
    assert float(((got[0].double() - want).abs() - bound).max()) <= 0


@pytest.mark.parametrize("T,E,k,d,F,kind", [
    (1, 8, 2, 4096, 1792, "bf16"), (5, 12, 3, 7168, 2048, "e4m3-e8m0"), (16, 3, 2, 2048, 7168, "bf16"),
    (2, 2, 1, 16384, 128, "f32"), (12, 2, 2, 128, 16384, "e4m3-f32"), (6, 9, 4, 2944, 1408, "bf16")])
def test_longer_reductions(T, E, k, d, F, kind):
    c = _case(T, E, k, d, F, kind, seed=d + F)
    _check(c, *_run(c))


def test_no_tokens():
    c = _case(0, 8, 2, 128, 128, "bf16", seed=1)
    out, ints = _run(c)
    assert all(bool((v == 0).all()) for v in ints)


def test_outputs_are_optional_and_repeat():
    c = _case(9, 12, 3, 256, 384, "bf16", seed=5)
    want = _run(c)[0]
    args = _args(c)
    for byte in (0, 127, 255):
        s, ws, out = _setup(c, ws_byte=byte)
        for _ in range(3):
            out.fill_(5)
            _call(c, s, ws, out, [None] * 4, args)
            assert torch.equal(out.cpu(), want)


def test_ties_go_to_the_lowest_index():
    c = _case(4, 12, 3, 128, 128, "bf16", seed=6, bias=False)
    c["w_router"][7] = c["w_router"][2]
    c["w_router"][9] = c["w_router"][2]
    c["w_router"][11] = c["w_router"][0]
    out, ints = _run(c)
    _check(c, out, ints)
    c["w_router"].zero_()
    out, ints = _run(c)
    _check(c, out, ints)
    assert ints[0].tolist() == [4, 4, 4] + [0] * 9


def test_close_logits_are_told_apart():
    """Logits that differ in their last fp32 bits, where a sum in 32 bits would swap them."""
    c = _case(16, 8, 1, 4096, 128, "f32", seed=8, bias=False)
    base = torch.randn(4096, generator=torch.Generator().manual_seed(9))
    c["w_router"] = base.repeat(8, 1)
    c["w_router"][:, -1] += torch.arange(8) * 2.0 ** -18
    out, ints = _run(c)
    _check(c, out, ints)


@pytest.mark.parametrize("kind", ["bf16", "e4m3-f32"])
def test_what_no_token_chose_is_not_read_into_anything(kind):
    c = _case(6, 8, 2, 256, 256, kind, seed=12)
    c["b"] = torch.tensor([0.0, 0, 0, -90, 0, 0, 0, -90])  # nobody chooses two of them
    clean = _run(c)
    idx = ref.route(c["x"], c["w_router"], c["b"], 2)[0]
    unused = [e for e in range(8) if not bool((idx == e).any())]
    for w in c["w"]:
        if kind == "bf16":
            w[unused] = float("nan")
        else:
            w[1][unused] = float("inf")
    got = _run(c)
    assert torch.equal(got[0], clean[0])
    # an expert's infinities reach its own tokens alone
    e = next(e for e in range(8) if 0 < int((idx == e).sum()) < 6)
    for w in c["w"]:
        if kind == "bf16":
            w[e] = float("inf")
        else:
            w[1][e] = float("nan")
    got = _run(c)
    mine = (idx == e).any(1)
    assert torch.equal(got[0][~mine], clean[0][~mine])
    assert not bool(got[0][mine].isfinite().any())


def test_tokens_with_numbers_that_are_none():
    c = _case(5, 8, 2, 256, 256, "bf16", seed=13)
    clean = _run(c)[0]
    c["x"][2, 100] = float("nan")
    c["x"][4, 3] = float("inf")
    out, ints = _run(c)
    assert int(ints[3]) == 2
    assert torch.equal(out[[0, 1, 3]], clean[[0, 1, 3]])


@pytest.mark.parametrize("kind", ["e4m3-f32", "e4m3-e8m0"])
def test_every_e4m3_value(kind):
    c = _case(4, 2, 1, 128, 256, kind, seed=14)
    codes = torch.arange(256).to(torch.uint8)
    codes[127], codes[255] = 0, 128  # the two NaN
    w = codes.repeat(128).view(256, 128)
    for i in (0, 1):
        q = w.view(torch.float8_e4m3fn).expand(2, 256, 128).contiguous()
        s = c["w"][i][1]
        s = torch.full_like(s, 120) if s.dtype == torch.uint8 else torch.full_like(s, 2.0 ** -7 * 1.3)
        c["w"][i] = (q, s)
        c["exact"][i] = torch.stack([dequantize(q[e], s[e], 128) for e in range(2)])
    _check(c, *_run(c))
    q = c["w"][0][0].clone().view(torch.uint8)
    q[:, 3, 5] = 0x7f
    c["w"][0] = (q.view(torch.float8_e4m3fn), c["w"][0][1])
    assert not bool(_run(c)[0].isfinite().any())


def test_extreme_scales():
    c = _case(3, 2, 1, 256, 128, "e4m3-e8m0", seed=15)
    for i, v in ((0, 0), (1, 254)):  # 2^-127 and 2^127
        q, s = c["w"][i]
        s = torch.full_like(s, v)
        c["w"][i] = (q, s)
    c["x"] = (c["x"].float() * 2.0 ** -60).to(torch.bfloat16)
    c["w_router"] = (c["w_router"].float() * 2.0 ** 60).to(torch.bfloat16)
    out = _run(c)[0]
    # gate about 2^-180: silu(gate) * up vanishes or stays tiny; nothing is infinite or NaN
    assert bool(out.isfinite().all())
    c["w"][0] = (c["w"][0][0], torch.full_like(c["w"][0][1], 255))
    assert not bool(_run(c)[0].isfinite().any())


def test_as_the_layer_for_many_tokens():
    c = _case(16, 8, 2, 512, 1024, "bf16", seed=16)
    s, ws, out = _setup(c)
    args = _args(c)
    _call(c, s, ws, out, [None] * 4, args)
    layer = moe.MoELayer(s)
    want = layer(args[0], args[1], args[2], *args[3])
    # two roundings of an expert's outputs to bf16 apart
    assert float((out.double() - want.double()).norm() / want.double().norm()) <= 8e-3


def test_captured_and_replayed():
    c = _case(5, 8, 2, 256, 384, "bf16", seed=17)
    s, ws, out = _setup(c)
    ints, args = _ints(c), _args(c)
    _call(c, s, ws, out, ints, args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _call(c, s, ws, out, ints, args)
    for seed in range(4):
        n = _case(5, 8, 2, 256, 384, "bf16", seed=20 + seed)
        args[0].copy_(n["x"])
        ws.random_(0, 255)  # whatever other work left there
        out.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        n.update(w=c["w"], exact=c["exact"], w_router=c["w_router"], b=c["b"])
        _check(n, out.cpu(), [v.cpu() for v in ints])


def test_two_at_once_on_two_streams():
    cases = [_case(3, 8, 2, 512, 1024, "bf16", seed=30), _case(16, 4, 2, 256, 512, "e4m3-f32", seed=31)]
    want = [_run(c)[0] for c in cases]
    runs = [(c, *_setup(c), _args(c), torch.cuda.Stream()) for c in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s, ws, out, args, stream in runs:
            _call(c, s, ws, out, [None] * 4, args, stream=stream)
    torch.cuda.synchronize()
    for (c, s, ws, out, args, stream), w in zip(runs, want):
        assert torch.equal(out.cpu(), w)


def test_refusals():
    c = _case(4, 8, 2, 128, 256, "bf16", seed=40)
    s, ws, out = _setup(c)
    x, wr, b, w = _args(c)
    good = dict(x=x, w_router=wr, b_router=b, w_gate=w[0], w_up=w[1], w_down=w[2], workspace=ws,
                out=out)
    for bad in (dict(x=x[:3]), dict(x=x.float()), dict(w_router=wr[:7]), dict(b_router=b.double()),
                dict(w_gate=w[2]), dict(w_up=None), dict(w_down=w[2].cpu()), dict(out=out[:, :64]),
                dict(routed_counts=torch.zeros(8, device="cuda")),
                dict(drops=torch.zeros(3, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            moe.layer_few(s, **{**good, **bad})
    with pytest.raises(moe.MoeError):
        moe.layer_few(s, **{**good, "workspace": ws[:-1]})
    with pytest.raises(moe.MoeError):
        moe.layer_few(s, **{**good, "workspace": None})
    assert moe.few_workspace_size(moe.shape(17, 128, 8, 2, 256)) == 0
