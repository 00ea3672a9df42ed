"""Cases of the layer for a few tokens, the experts' linear layers and gradient clipping.

Each case is one operator at one size.  `run` computes it either in plain torch operations in
32 bits (`own` false) or through the framework's entry points (`own` true).

Operators ("op" of a case):
  few     a whole mixture-of-experts layer of at most 16 tokens: router logits (64-bit sums rounded
          to 32 bits), the k largest of each token (ties to the lowest index), softmax over them,
          the chosen experts' SwiGLU networks (h rounded to x's type, as the layer defines it) and
          the gate-weighted sum.  Weights are x's type, or e4m3 with a scale per 128 x 128 block
          ("scale" of the case) beside bf16 x
  linear  y[r] = act(z[r]) + residual[r], z[r] = x[r] W[e]^T + b[e] for the rows r of expert e;
          z is an output too where the case keeps it for the backward pass
  linear_grad  dz = dy * act'(z), db[e] = sum of dz over the rows of expert e
  clip    the 2-norm over many gradients, and the gradients times max_norm / norm where the norm is
          larger than max_norm
"""
import math

import torch

own = False

F32, E8M0 = "f32", "e8m0"
BLOCK = 128
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def listed():
    return [
        # a gradient check's or a unit test's layer, 32 bits: latency alone
        {"name": "few tiny fp32", "op": "few", "T": 3, "E": 4, "k": 2, "d": 256, "F": 512,
         "dtype": "f32", "scale": "", "capacity": 0},
        # one token of a chat with eight large experts: two of them are read
        {"name": "few one token", "op": "few", "T": 1, "E": 8, "k": 2, "d": 4096, "F": 14336,
         "dtype": "bf16", "scale": "", "capacity": 0},
        # five drafted tokens at once over 256 small experts in 8 bits
        {"name": "few drafted tokens e4m3", "op": "few", "T": 5, "E": 256, "k": 8, "d": 7168,
         "F": 2048, "dtype": "bf16", "scale": E8M0, "capacity": 0},
        # the largest step: sixteen requests, every expert read, a capacity that drops some
        {"name": "few sixteen tokens", "op": "few", "T": 16, "E": 8, "k": 2, "d": 6144, "F": 16384,
         "dtype": "bf16", "scale": "", "capacity": 5},
        # a shared expert's down projection for a few tokens, added to what is there: latency
        {"name": "linear few rows", "op": "linear", "E": 1, "rows": 33, "slack": 0, "K": 2048,
         "N": 7168, "dtype": "bf16", "act": "none", "bias": False, "residual": True, "keep": False},
        # the first layer of eight experts in training: bias and gelu, z kept
        {"name": "linear train", "op": "linear", "E": 8, "rows": 8191, "slack": 0, "K": 4096,
         "N": 14336, "dtype": "bf16", "act": "gelu", "bias": True, "residual": False, "keep": True},
        # ... and the second one: bias and residual
        {"name": "linear second", "op": "linear", "E": 8, "rows": 8192, "slack": 77, "K": 14336,
         "N": 4096, "dtype": "bf16", "act": "none", "bias": True, "residual": True, "keep": False},
        # a check's size in 32 bits: ragged experts
        {"name": "linear ragged fp32", "op": "linear", "E": 8, "rows": 1001, "slack": 23, "K": 512,
         "N": 1024, "dtype": "f32", "act": "silu", "bias": True, "residual": False, "keep": True},
        # the backward pass of the first layer up to its product
        {"name": "linear_grad train", "op": "linear_grad", "E": 8, "rows": 8191, "slack": 0,
         "N": 14336, "dtype": "bf16", "act": "gelu"},
        # ... of 32 small experts, ragged, in 32 bits
        {"name": "linear_grad ragged fp32", "op": "linear_grad", "E": 32, "rows": 1001, "slack": 23,
         "N": 1024, "dtype": "f32", "act": "silu"},
        # the gradients of a small model's layers, each tensor by itself: latency
        {"name": "clip many small", "op": "clip", "tensors": 320, "largest": 1 << 18,
         "dtype": "mixed", "clipped": True},
        # three projections of eight large experts: 1.4 G values
        {"name": "clip experts", "op": "clip", "tensors": 24, "largest": 14336 * 4096,
         "dtype": "bf16", "clipped": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _wide(rng, lo, hi):
    return 128 * max(1, _log(rng, lo / 128, hi / 128))


def draw(rng):
    op = rng.choice(["few", "few", "linear", "linear_grad", "clip"])
    if op == "few":
        dtype, scale = rng.choice([("bf16", ""), ("bf16", ""), ("f32", ""), ("bf16", F32),
                                   ("bf16", E8M0)])
        E = rng.choice([1, 4, 7, 8, 16, 64, 128, 256])
        k = min(E, rng.choice([1, 2, 4, 6, 8]))
        T = rng.choice([1, 1, 2, 3, 4, 5, 6, 8, 11, 13, 16])
        d, F = _wide(rng, 128, 8192), _wide(rng, 128, 16384)
        most = 1.5e9 if dtype == "f32" else 3e9
        while T * k * d * F > most or E * d * F > 1.5 * most:
            if T * k * d * F > most and T > 1:
                T = T // 2
            elif E > 8:
                E = E // 2
                k = min(k, E)
            else:
                F = max(128, F // 256 * 128)
        return {"op": op, "T": T, "E": E, "k": k, "d": d, "F": F, "dtype": dtype, "scale": scale,
                "capacity": rng.choice([0, 0, 1, 2, 3])}
    if op == "clip":
        tensors = _log(rng, 1, 1000)
        largest = _log(rng, 1, 1 << 26)
        largest = min(largest, max(1, (1 << 30) // tensors))
        return {"op": op, "tensors": tensors, "largest": largest,
                "dtype": rng.choice(["bf16", "f32", "mixed"]),
                "clipped": rng.choice([True, True, False])}
    E = rng.choice([1, 3, 8, 16, 32, 64, 128])
    N, K = _wide(rng, 128, 16384), _wide(rng, 128, 16384)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "linear_grad":
        rows = _log(rng, 1, min(65536, (1 << 27) // N))
        return {"op": op, "E": E, "rows": rows, "slack": rng.choice([0, 0, 1, 77]), "N": N,
                "dtype": dtype, "act": rng.choice(ACTS)}
    while E * N * K > 1 << 31 and E > 1:
        E = max(1, E // 2)
    # the matrix units do 32-bit products at a sixteenth of the 16-bit rate
    most = 4e11 if dtype == "bf16" else 4e10
    rows = _log(rng, 1, min(32768, max(2, int(most / (N * K)))))
    return {"op": op, "E": E, "rows": rows, "slack": rng.choice([0, 0, 1, 77]), "K": K, "N": N,
            "dtype": dtype, "act": rng.choice(ACTS), "bias": rng.choice([True, True, False]),
            "residual": rng.choice([True, False]), "keep": rng.choice([True, False])}


# ------------------------------------------------------------------------------------ inputs
def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, g, dtype, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(std)


def _e4m3(shape, g):
    """e4m3 values as a quantizer leaves them: normal, the largest of a block near 448."""
    v = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    return v.mul_(112).clamp_(-448, 448).to(torch.float8_e4m3fn)


def _scales(shape, g, kind, size):
    """Scales about `size`: any fp32 values, or powers of two as exponent bytes (bias 127)."""
    v = torch.rand(shape, generator=g, device="cuda").add_(0.5).mul_(size)
    if kind == F32:
        return v
    return v.log2_().round_().add_(127).to(torch.uint8)


def _groups(rows, E, g):
    """Offsets [E + 1] of `rows` rows dealt to E experts of unequal popularity."""
    p = (0.5 * torch.randn(E, generator=g, device="cuda")).exp_()
    e = torch.multinomial(p, rows, replacement=True, generator=g)
    counts = torch.bincount(e, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    return offsets, int(counts.max())


def _lengths(case):
    """Lengths of the gradients: equal, or where they are many of several sizes, odd ones too."""
    n, most = case["tensors"], case["largest"]
    if n <= 24:
        return [most] * n
    return [max(1, (most >> 2 * (i % 4)) - i % 3) for i in range(n)]


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    op = case["op"]
    if op == "few":
        T, E, d, F = case["T"], case["E"], case["d"], case["F"]
        dt = _type(case["dtype"])
        s["x"] = _normal((T, d), g, dt)
        s["w_router"] = _normal((E, d), g, dt, 1 / math.sqrt(d))
        s["b_router"] = _normal((E,), g, torch.float32, 0.3)
        for name, n, kk in (("w_gate", F, d), ("w_up", F, d), ("w_down", d, F)):
            if case["scale"]:
                s[name] = _e4m3((E, n, kk), g)
                s[name + "_scale"] = _scales((E, n // BLOCK, kk // BLOCK), g, case["scale"],
                                             1 / (112 * math.sqrt(kk)))
            else:
                s[name] = _normal((E, n, kk), g, dt, 1 / math.sqrt(kk))
        return s
    if op == "clip":
        s["grads"] = []
        for i, n in enumerate(_lengths(case)):
            dt = _type(("bf16", "f32")[i % 2] if case["dtype"] == "mixed" else case["dtype"])
            s["grads"].append(_normal((n,), g, dt, 1e-3 * (1 + i % 7)))
        # the optimizer's flat buffers, one for each type, every tensor's part from a whole line on
        s["flat"], s["out"] = {}, [None] * len(s["grads"])
        for dt in {v.dtype for v in s["grads"]}:
            mine = [i for i, v in enumerate(s["grads"]) if v.dtype == dt]
            ends = [0]
            for i in mine:
                ends.append(ends[-1] + (s["grads"][i].numel() + 63) // 64 * 64)
            s["flat"][str(dt)] = torch.zeros(ends[-1], dtype=dt, device="cuda")
            for i, at in zip(mine, ends):
                s["out"][i] = s["flat"][str(dt)][at:at + s["grads"][i].numel()]
        # a tenth of the norm that values of these sizes have, or ten times it
        size = math.sqrt(sum(v.numel() * (1e-3 * (1 + i % 7)) ** 2
                             for i, v in enumerate(s["grads"])))
        s["max_norm"] = size * (0.1 if case["clipped"] else 10.0)
        return s
    E, rows, N = case["E"], case["rows"], case["N"]
    s["R"] = rows + case["slack"]
    s["offsets"], s["most"] = _groups(rows, E, g)
    dt = _type(case["dtype"])
    # what lies behind the last expert's rows is not the operator's to read
    if op == "linear_grad":
        s["dy"] = _normal((s["R"], N), g, dt)
        s["z"] = _normal((s["R"], N), g, dt)
        s["dy"][rows:] = math.nan
        s["z"][rows:] = math.nan
        s["dz"] = torch.zeros((s["R"], N), dtype=dt, device="cuda")
        s["db"] = torch.empty((E, N), dtype=torch.float32, device="cuda")
        return s
    K = case["K"]
    s["x"] = _normal((s["R"], K), g, dt)
    s["x"][rows:] = math.nan
    s["w"] = _normal((E, N, K), g, dt, 1 / math.sqrt(K))
    s["b"] = _normal((E, N), g, torch.float32, 0.5) if case["bias"] else None
    s["res"] = _normal((s["R"], N), g, dt) if case["residual"] else None
    s["y"] = torch.zeros((s["R"], N), dtype=dt, device="cuda")
    s["z"] = torch.zeros((s["R"], N), dtype=dt, device="cuda") if case["keep"] else None
    return s


# ------------------------------------------------------------------------------- plain forms
def _plain_scale(scale):
    if scale.dtype == torch.float32:
        return scale
    return (scale.to(torch.int32) << 23).view(torch.float32)  # 2^(v - 127), 1 <= v <= 254


def _plain_act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))


def _plain_slope(z, act):
    """act'(z)."""
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = torch.sigmoid(z)
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return (0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def _plain_few(s):
    T, E, k = s["T"], s["E"], s["k"]
    x = s["x"].float()
    # the logits' order decides: 64-bit sums
    logits = (s["x"].double() @ s["w_router"].double().t() + s["b_router"].double()).float()
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    idx = order.indices[:, :k].contiguous()
    top = order.values[:, :k]
    gate = torch.exp(top - top[:, :1])
    gate = gate / gate.sum(dim=1, keepdim=True)
    chosen = torch.zeros((T * k, E), dtype=torch.int32, device=x.device)
    chosen.scatter_(1, idx.view(-1, 1), 1)
    routed = chosen.sum(dim=0).to(torch.int32)
    if s["capacity"]:
        before = (chosen.cumsum(0) - chosen).gather(1, idx.view(-1, 1)).view(T, k)
        kept = before < s["capacity"]
    else:
        kept = torch.ones_like(idx, dtype=torch.bool)
    gate = torch.where(kept, gate, torch.zeros_like(gate))

    def weight(name, e):
        w = s[name].view(torch.uint8).index_select(0, e)[0].view(torch.float8_e4m3fn) \
            if s["scale"] else s[name].index_select(0, e)[0]
        w = w.float()
        if s["scale"]:
            n, kk = w.shape
            b = _plain_scale(s[name + "_scale"].index_select(0, e)[0])
            w = (w.view(n // BLOCK, BLOCK, kk // BLOCK, BLOCK) * b[:, None, :, None]).view(n, kk)
        return w

    out = torch.zeros_like(x)
    for t in range(T):
        for j in range(k):
            e = idx[t, j:j + 1]
            a = weight("w_gate", e) @ x[t]
            h = a * torch.sigmoid(a) * (weight("w_up", e) @ x[t])
            h = h.to(s["x"].dtype).float()
            out[t] += gate[t, j] * (weight("w_down", e) @ h)
    kept_by_slot = kept.sum(dim=0)
    drops = torch.cat([(T * k - kept.sum()).view(1), T - kept_by_slot,
                       (~kept.any(dim=1)).sum().view(1)]).to(torch.int32)
    return {"out": out.to(s["x"].dtype), "routed": routed, "drops": drops}


def _pad(x, offsets, most):
    """Rows of x by expert, [E, most, K], zero where an expert has fewer; the places too."""
    i = torch.arange(most, device=x.device)
    place = offsets[:-1, None].long() + i
    live = place < offsets[1:, None]
    rows = x[place.clamp(max=x.shape[0] - 1)].float()
    return torch.where(live[:, :, None], rows, torch.zeros_like(rows)), place[live], live


def _plain(s):
    op = s["op"]
    if op == "few":
        return _plain_few(s)
    if op == "clip":
        total = torch.stack([(v.double() ** 2).sum() for v in s["grads"]]).sum()
        norm = total.sqrt().float()
        scale = torch.where(norm > s["max_norm"], s["max_norm"] / norm, torch.ones_like(norm))
        for v, o in zip(s["grads"], s["out"]):
            o.copy_((v.float() * scale).to(v.dtype))
        return {"norm": norm.view(1), **s["flat"]}
    if op == "linear_grad":
        dy, place, live = _pad(s["dy"], s["offsets"], s["most"])
        z, _, _ = _pad(s["z"], s["offsets"], s["most"])
        dz = dy * _plain_slope(z, s["act"])
        s["dz"][place] = dz[live].to(s["dz"].dtype)
        return {"dz": s["dz"], "db": dz.sum(dim=1)}
    x, place, live = _pad(s["x"], s["offsets"], s["most"])
    z = torch.bmm(x, s["w"].float().transpose(1, 2).contiguous())
    if s["b"] is not None:
        z = z + s["b"][:, None, :]
    out = {}
    if s["z"] is not None:
        s["z"][place] = z[live].to(s["z"].dtype)
        out["z"] = s["z"]
    y = _plain_act(z, s["act"])[live]
    if s["res"] is not None:
        y = y + s["res"][place].float()
    s["y"][place] = y.to(s["y"].dtype)
    out["y"] = s["y"]
    return out


# -------------------------------------------------------------------------- the framework's
def _own(s):
    import routing_expert_ffn_router_amd as moe

    op = s["op"]
    if op == "clip":
        if "workspace" not in s:
            s["workspace"] = torch.empty(moe.grad_workspace_size(len(s["grads"])),
                                         dtype=torch.uint8, device="cuda")
            s["norm"] = torch.empty(1, dtype=torch.float32, device="cuda")
        moe.clip_grad_norm(s["grads"], s["max_norm"], s["workspace"], s["norm"], s["out"])
        return {"norm": s["norm"], **s["flat"]}
    dt = moe.MOE_BF16 if s["dtype"] == "bf16" else moe.MOE_F32
    if op == "few":
        if "shape" not in s:
            s["shape"] = moe.shape(s["T"], s["d"], s["E"], s["k"], s["F"], s["capacity"], dt)
            s["workspace"] = torch.empty(moe.few_workspace_size(s["shape"]), dtype=torch.uint8,
                                         device="cuda")
            s["out"] = torch.empty_like(s["x"])
            for name, n in (("routed", s["E"]), ("drops", s["k"] + 2)):
                s[name] = torch.empty(n, dtype=torch.int32, device="cuda")
        if s["scale"]:
            kind = moe.MOE_SCALE_F32 if s["scale"] == F32 else moe.MOE_SCALE_E8M0
            moe.layer_few_fp8(s["shape"], kind, s["x"], s["w_router"], s["b_router"],
                              (s["w_gate"], s["w_gate_scale"]), (s["w_up"], s["w_up_scale"]),
                              (s["w_down"], s["w_down_scale"]), s["workspace"], s["out"],
                              routed_counts=s["routed"], drops=s["drops"])
        else:
            moe.layer_few(s["shape"], s["x"], s["w_router"], s["b_router"], s["w_gate"], s["w_up"],
                          s["w_down"], s["workspace"], s["out"], routed_counts=s["routed"],
                          drops=s["drops"])
        return {"out": s["out"], "routed": s["routed"], "drops": s["drops"]}
    act = ACTS.index(s["act"])  # MOE_ACT_NONE ... MOE_ACT_GELU_TANH
    if "shape" not in s:
        s["shape"] = moe.group_shape(s["R"], s["E"], s["N"], s.get("K", BLOCK), dt)
        s["workspace"] = torch.empty(moe.linear_workspace_size(s["shape"]), dtype=torch.uint8,
                                     device="cuda")
    if op == "linear_grad":
        moe.grouped_linear_grad(s["shape"], act, s["dy"], s["z"], s["offsets"], s["workspace"],
                                s["dz"], s["db"])
        return {"dz": s["dz"], "db": s["db"]}
    moe.grouped_linear(s["shape"], act, s["x"], s["offsets"], s["w"], s["b"], s["res"],
                       s["workspace"], s["y"], s["z"])
    return {"z": s["z"], "y": s["y"]} if s["z"] is not None else {"y": s["y"]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------ in 64 bits
def _exact_weight(s, name, e):
    w = s[name][e]
    if not s["scale"]:
        return w.double()
    b = s[name + "_scale"][e]
    b = b.double() if b.dtype == torch.float32 else torch.exp2(b.double() - 127)
    return w.to(torch.float32).double() * b.repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)


def _exact_few(s):
    T, E, k, C = s["T"], s["E"], s["k"], s["capacity"]
    x = s["x"].double()
    # logits are 32-bit numbers
    rows = ((x[:, None, :] * s["w_router"].double()[None]).sum(2)
            + s["b_router"].double()).to(torch.float32).tolist()
    out = torch.zeros_like(x)
    count, slot, none = [0] * E, [0] * k, 0
    work = {}
    for t, row in enumerate(rows):
        best = sorted(range(E), key=lambda e: (-row[e], e))[:k]
        part = [math.exp(row[e] - row[best[0]]) for e in best]
        lost = 0
        for j, e in enumerate(best):
            count[e] += 1
            if C and count[e] > C:
                slot[j] += 1
                lost += 1
            else:
                work.setdefault(e, []).append((t, part[j] / sum(part)))
        none += lost == k
    for e, pairs in work.items():
        at = torch.tensor([t for t, _ in pairs], device=x.device)
        share = torch.tensor([p for _, p in pairs], dtype=torch.float64, device=x.device)
        a = x[at] @ _exact_weight(s, "w_gate", e).t()
        h = a / (1 + torch.exp(-a)) * (x[at] @ _exact_weight(s, "w_up", e).t())
        h = h.to(s["x"].dtype).double()
        out[at] += share[:, None] * (h @ _exact_weight(s, "w_down", e).t())
    return {"out": out, "routed": torch.tensor(count, dtype=torch.int32, device=x.device),
            "drops": torch.tensor([sum(slot), *slot, none], dtype=torch.int32, device=x.device)}


def _exact_act(z, act):
    """(act(z), act'(z))"""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return z * p, p + z * p * (1 - p)
    if act == "gelu":
        p = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    u = math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3)
    p = 1 / (1 + torch.exp(-u))  # (1 + tanh(u / 2)) / 2
    return z * p, p + z * p * (1 - p) * math.sqrt(8 / math.pi) * (1 + 3 * 0.044715 * z ** 2)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "few":
        return _exact_few(s)
    if op == "clip":
        norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(v.double())) ** 2
                                   for v in s["grads"]))
        scale = min(1.0, s["max_norm"] / norm)
        flat = {name: torch.zeros(v.shape, dtype=torch.float64, device="cuda")
                for name, v in s["flat"].items()}
        for v, o in zip(s["grads"], s["out"]):
            at = o.storage_offset()
            flat[str(v.dtype)][at:at + v.numel()] = v.double() * scale
        return {"norm": torch.tensor([norm], dtype=torch.float64, device="cuda"), **flat}
    at = s["offsets"].tolist()
    N = case["N"]
    if op == "linear_grad":
        dz = torch.zeros((s["R"], N), dtype=torch.float64, device="cuda")
        db = torch.zeros((case["E"], N), dtype=torch.float64, device="cuda")
        for e, (a, b) in enumerate(zip(at, at[1:])):
            dz[a:b] = s["dy"][a:b].double() * _exact_act(s["z"][a:b].double(), case["act"])[1]
            db[e] = dz[a:b].sum(0)
        return {"dz": dz, "db": db}
    y = torch.zeros((s["R"], N), dtype=torch.float64, device="cuda")
    z = torch.zeros_like(y)
    for e, (a, b) in enumerate(zip(at, at[1:])):
        if b > a:
            z[a:b] = s["x"][a:b].double() @ s["w"][e].double().t()
            if s["b"] is not None:
                z[a:b] += s["b"][e].double()
            y[a:b] = _exact_act(z[a:b], case["act"])[0]
            if s["res"] is not None:
                y[a:b] += s["res"][a:b].double()
    return {"z": z, "y": y} if case["keep"] else {"y": y}


# ------------------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "clip":
        n = _lengths(case)
        per = {"bf16": 2, "f32": 4}
        size = sum(v * (per[("bf16", "f32")[i % 2]] if case["dtype"] == "mixed"
                        else per[case["dtype"]]) for i, v in enumerate(n))
        return {"bytes": 2 * size, "flops": 3 * sum(n)}
    size = 2 if case["dtype"] == "bf16" else 4
    E = case["E"]
    if op == "few":
        T, k, d, F = case["T"], case["k"], case["d"], case["F"]
        live = E * (1 - (1 - k / E) ** T)  # experts that a token chose: the others stay unread
        per = size
        if case["scale"]:
            per = 1 + (4 if case["scale"] == F32 else 1) / BLOCK ** 2
        return {"bytes": 3 * live * d * F * per + (E * d + 2 * T * d) * size,
                "flops": 2 * T * d * (E + 3 * k * F)}
    R, N = case["rows"], case["N"]
    if op == "linear_grad":
        return {"bytes": 3 * R * N * size + 4 * E * N, "flops": 8 * R * N}
    K = case["K"]
    live = E * (1 - (1 - 1 / E) ** R)  # experts that get a row
    outputs = 1 + (1 if case["keep"] else 0) + (1 if case["residual"] else 0)
    return {"bytes": (R * K + live * N * K + outputs * R * N) * size
            + (4 * live * N if case["bias"] else 0), "flops": 2 * R * N * K}
