"""The operators as a training and serving program uses them: a step of the experts' network through
linear layers, their backward pass, the products' gradients and clipping, and the trained weights
served for a few tokens.  Eager, captured, on two streams, and at sizes past 2^31 values."""
import pytest
import torch

import _few as ref
import routing_expert_ffn_router_amd as moe
from _fp8 import offsets_of

pytestmark = pytest.mark.gpu

E, D, F = 5, 256, 384
COUNTS = [70, 0, 9, 130, 31]


class Step:
    """y = x + (silu(x Wg^T + bg) * (x Wu^T + bu)) Wd^T + bd for rows grouped by expert, fp32."""

    def __init__(self, seed, stream=None):
        g = torch.Generator().manual_seed(seed)
        self.R = sum(COUNTS)
        self.x = torch.randn((self.R, D), generator=g).cuda()
        self.dy = torch.randn((self.R, D), generator=g).cuda()
        self.off = offsets_of(COUNTS).cuda()
        self.w = {n: (torch.randn(s, generator=g) / s[2] ** 0.5).cuda()
                  for n, s in (("g", (E, F, D)), ("u", (E, F, D)), ("d", (E, D, F)))}
        self.b = {n: (torch.randn((E, s), generator=g) * 0.3).cuda()
                  for n, s in (("g", F), ("u", F), ("d", D))}
        wide, back = moe.group_shape(self.R, E, F, D, moe.MOE_F32), moe.group_shape(self.R, E, D, F,
                                                                                 moe.MOE_F32)
        self.shapes = {"g": wide, "u": wide, "d": back}
        most = max(f(s) for s in (wide, back) for f in (moe.linear_workspace_size,
                                                       moe.group_workspace_size))
        self.ws = torch.empty(most, dtype=torch.uint8, device="cuda")
        self.buf = {n: torch.empty((self.R, F), device="cuda")
                    for n in ("zg", "hg", "hu", "dh", "dzg", "dzu")}
        self.y = torch.empty((self.R, D), device="cuda")
        self.dx = {n: torch.empty((self.R, D), device="cuda") for n in "gu"}
        self.dw = {n: torch.empty_like(v) for n, v in self.w.items()}
        self.db = {n: torch.empty_like(v) for n, v in self.b.items()}
        self.grads = [*self.dw.values(), *self.db.values()]
        self.out = [torch.empty_like(v) for v in self.grads]
        self.norm_ws = torch.empty(moe.grad_workspace_size(len(self.grads)), dtype=torch.uint8,
                                   device="cuda")
        self.norm = torch.empty(1, device="cuda")
        self.stream = stream

    def run(self, max_norm=1.0):
        v, s, st = self.buf, self.shapes, self.stream
        moe.grouped_linear(s["g"], moe.MOE_ACT_SILU, self.x, self.off, self.w["g"], self.b["g"], None,
                           self.ws, v["hg"], v["zg"], stream=st)
        moe.grouped_linear(s["u"], moe.MOE_ACT_NONE, self.x, self.off, self.w["u"], self.b["u"], None,
                           self.ws, v["hu"], stream=st)
        with torch.cuda.stream(st or torch.cuda.current_stream()):
            h = v["hg"] * v["hu"]
        moe.grouped_linear(s["d"], moe.MOE_ACT_NONE, h, self.off, self.w["d"], self.b["d"], self.x,
                           self.ws, self.y, stream=st)
        moe.grouped_linear_grad(s["d"], moe.MOE_ACT_NONE, self.dy, None, self.off, self.ws, None,
                                self.db["d"], stream=st)
        moe.grouped_wgrad(s["d"], self.dy, h, self.off, self.ws, self.dw["d"], stream=st)
        moe.grouped_dgrad(s["d"], self.dy, self.off, self.w["d"], self.ws, v["dh"], stream=st)
        with torch.cuda.stream(st or torch.cuda.current_stream()):
            dg, du = v["dh"] * v["hu"], v["dh"] * v["hg"]
        moe.grouped_linear_grad(s["g"], moe.MOE_ACT_SILU, dg, v["zg"], self.off, self.ws, v["dzg"],
                                self.db["g"], stream=st)
        moe.grouped_linear_grad(s["u"], moe.MOE_ACT_NONE, du, None, self.off, self.ws, v["dzu"],
                                self.db["u"], stream=st)
        for n, dz in (("g", v["dzg"]), ("u", v["dzu"])):
            moe.grouped_wgrad(s[n], dz, self.x, self.off, self.ws, self.dw[n], stream=st)
            moe.grouped_dgrad(s[n], dz, self.off, self.w[n], self.ws, self.dx[n], stream=st)
        moe.clip_grad_norm(self.grads, max_norm, self.norm_ws, self.norm, self.out, stream=st)

    def results(self):
        return [self.y, self.norm, *self.dx.values(), *self.grads, *self.out]

    def reference(self, max_norm=1.0):
        """The same by autograd in 64 bits on the CPU."""
        x = self.x.cpu().double().requires_grad_()
        w = {n: v.cpu().double().requires_grad_() for n, v in self.w.items()}
        b = {n: v.cpu().double().requires_grad_() for n, v in self.b.items()}
        rows, at = [], 0
        for e, n in enumerate(COUNTS):
            r = x[at:at + n]
            h = torch.nn.functional.silu(r @ w["g"][e].t() + b["g"][e]) * (r @ w["u"][e].t() + b["u"][e])
            rows.append(r + h @ w["d"][e].t() + b["d"][e])
            at += n
        y = torch.cat(rows)
        y.backward(self.dy.cpu().double())
        grads = [v.grad for v in (*w.values(), *b.values())]
        norm = torch.stack([(g ** 2).sum() for g in grads]).sum().sqrt()
        scale = min(1.0, max_norm / float(norm))
        return y.detach(), norm, x.grad, grads, [g * scale for g in grads]


def _close(got, want):
    # Four fp32 products follow each other at most, each within (K + 2) 2^-24 of its terms'
    # magnitudes, which for normal data are 0.64 sqrt(K) of the sums: 3e-4 with K = 384
    assert float((got.double().cpu() - want).norm() / want.norm()) <= 1.3e-3


def test_step_against_autograd():
    s = Step(1)
    s.run()
    y, norm, dx, grads, clipped = s.reference()
    _close(s.y, y)
    _close(s.norm, norm.view(1))
    _close(s.dx["g"] + s.dx["u"] + s.dy, dx)  # dy: the residual's
    for got, want in zip(s.grads, grads):
        _close(got, want)
    for got, want in zip(s.out, clipped):
        _close(got, want)
    assert all(bool((v[1] == 0).all()) for v in s.grads)  # the expert without rows


def test_trained_weights_served_for_a_few_tokens():
    s = Step(2)
    s.run(max_norm=3.0)
    w = [v - 0.1 * g for v, g in zip(s.w.values(), s.out)]
    g = torch.Generator().manual_seed(3)
    x, wr = torch.randn((6, D), generator=g), torch.randn((E, D), generator=g) / D ** 0.5
    shape = moe.shape(6, D, E, 2, F, 0, moe.MOE_F32)
    ws = torch.empty(moe.few_workspace_size(shape), dtype=torch.uint8, device="cuda")
    out = torch.empty((6, D), device="cuda")
    moe.layer_few(shape, x.cuda(), wr.cuda(), None, *w, ws, out)
    idx, gates, _, largest = ref.route(x, wr, None, 2)
    want, bound = ref.experts(x, [v.cpu().double() for v in w], idx, gates, ref.keep_of(idx, E, 0),
                              2.0 ** -24, largest)
    assert float(((out.cpu().double() - want).abs() - bound).max()) <= 0
    quantized = moe.MoELayerFp8(moe.shape(6, D, E, 2, F), moe.MOE_SCALE_F32)
    w8 = [quantized.quantize_weights(v) for v in w]
    s8 = moe.shape(6, D, E, 2, F)
    out8 = torch.empty((6, D), dtype=torch.bfloat16, device="cuda")
    moe.layer_few_fp8(s8, moe.MOE_SCALE_F32, x.cuda().bfloat16(), wr.cuda().bfloat16(), None, *w8, ws,
                      out8)
    # e4m3 keeps a weight to 2^-4 of itself; three of them in a product, at random signs
    assert float((out8.double().cpu() - want).norm() / want.norm()) <= 3 * 2.0 ** -4


def test_captured_step_replays():
    s = Step(4)
    s.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for seed in range(3):
        n = Step(10 + seed)
        n.run()
        s.x.copy_(n.x)
        s.dy.copy_(n.dy)
        for k in s.w:
            s.w[k].copy_(n.w[k])
            s.b[k].copy_(n.b[k])
        s.ws.random_(0, 255)
        s.norm_ws.random_(0, 255)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(s.results(), n.results()):
            assert torch.equal(a, b)


def test_steps_on_two_streams():
    alone = [Step(20), Step(21)]
    for s in alone:
        s.run()
    torch.cuda.synchronize()
    both = [Step(20, torch.cuda.Stream()), Step(21, torch.cuda.Stream())]
    torch.cuda.synchronize()
    for _ in range(5):
        for s in both:
            s.run()
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        for u, v in zip(a.results(), b.results()):
            assert torch.equal(u, v)


def test_more_than_2_to_the_31_values():
    R, K, N, experts = 70000, 128, 32768, 2
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((R, K), generator=g, device="cuda", dtype=torch.bfloat16)
    w = torch.randn((experts, N, K), generator=g, device="cuda", dtype=torch.bfloat16) / 8
    b = torch.randn((experts, N), generator=g, device="cuda")
    off = torch.tensor([0, 3, R], dtype=torch.int32, device="cuda")
    shape = moe.group_shape(R, experts, N, K, moe.MOE_BF16)
    ws = torch.empty(moe.linear_workspace_size(shape), dtype=torch.uint8, device="cuda")
    y, z = (torch.empty((R, N), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    moe.grouped_linear(shape, moe.MOE_ACT_RELU, x, off, w, b, None, ws, y, z)
    for a, c, e in ((0, 3, 0), (3, 10, 1), (65530, 65545, 1), (R - 9, R, 1)):
        want = x[a:c].double() @ w[e].double().t() + b[e].double()
        err = (K + 3) * 2.0 ** -24 * (x[a:c].double().abs() @ w[e].double().abs().t() + b[e].abs())
        assert float(((z[a:c].double() - want).abs() - 2.0 ** -8 * (want.abs() + err) - err).max()) <= 0
        assert torch.equal(y[a:c], z[a:c].relu())
    dz, db = torch.empty_like(y), torch.empty((experts, N), device="cuda")
    moe.grouped_linear_grad(shape, moe.MOE_ACT_RELU, y, z, off, ws, dz, db)
    assert torch.equal(dz, y)
    for e, (a, c) in enumerate(((0, 3), (3, R))):
        want = y[a:c].double().sum(0)
        # sixteen rows a wave, four waves, row tiles in sixteen runs: 16 + 4 + R / 1024 + 16 additions
        assert float(((db[e].double() - want).abs() - (36 + R / 1024) * 2.0 ** -24 * want).max()) <= 0
