"""The layer for a few tokens where tokens have fewer finite logits than slots: the slots without one
take expert 0, as moe_layer's do, each of them counted and each taking a place of its own."""
import pytest
import torch

import _few as ref
import routing_expert_ffn_router_amd as moe

pytestmark = pytest.mark.gpu


def _case(T, E, k, seed, d=128, F=256):
    g = torch.Generator().manual_seed(seed)
    bf = torch.bfloat16
    return {"T": T, "E": E, "k": k, "d": d, "F": F, "x": torch.randn((T, d), generator=g).to(bf),
            "w_router": (torch.randn((E, d), generator=g) / d ** 0.5).to(bf),
            "b": torch.randn(E, generator=g) * 0.3,
            "w": [(torch.randn(s, generator=g) / s[2] ** 0.5).to(bf)
                  for s in ((E, F, d), (E, F, d), (E, d, F))]}


def _select(c, groups):
    """(experts [T, k], gates [T, k], tokens with a logit that is not finite)."""
    E, k = c["E"], c["k"]
    logits = (c["x"].double() @ c["w_router"].double().t() + c["b"].double()).float()
    idx = torch.zeros((c["T"], k), dtype=torch.int64)
    for t, row in enumerate(logits.tolist()):
        ok = [e for e in range(E) if abs(row[e]) < float("inf")]
        if groups[0] > 1:
            size = E // groups[0]
            best = {g: max((row[e] for e in ok if e // size == g), default=None)
                    for g in range(groups[0])}
            best = {g: v for g, v in best.items() if v is not None}
            keep = sorted(best, key=lambda g: (-best[g], g))[:groups[1]]
            ok = [e for e in ok if e // size in keep]
        pick = sorted(ok, key=lambda e: (-row[e], e))[:k]
        idx[t] = torch.tensor(pick + [0] * (k - len(pick)))
    return idx, torch.softmax(logits.double().gather(1, idx), 1), ~logits.isfinite().all(1)


def _call(c, capacity, flags, groups):
    s = moe.shape(c["T"], c["d"], c["E"], c["k"], c["F"], capacity, moe.MOE_BF16, flags,
                  *(groups if groups[0] > 1 else (0, 0)))
    args = [c["x"].cuda(), c["w_router"].cuda(), c["b"].cuda(), *(w.cuda() for w in c["w"])]
    ws = torch.empty(moe.few_workspace_size(s), dtype=torch.uint8, device="cuda").fill_(255)
    out = torch.empty_like(args[0])
    ints = [torch.full((n,), -9, dtype=torch.int32, device="cuda")
            for n in (c["E"], c["E"], c["k"] + 2, 1)]
    moe.layer_few(s, *args, ws, out, *ints)
    layer = moe.MoELayer(s)
    layer(*args)
    many = [layer.routed_counts, layer.tokens_per_expert, layer.drops, layer.status]
    return out.cpu(), [v.cpu() for v in ints], layer.out.cpu(), [v.cpu() for v in many]


def _check(c, capacity, flags=0, groups=(1, 1)):
    E, k, T = c["E"], c["k"], c["T"]
    out, ints, many_out, many = _call(c, capacity, flags, groups)
    idx, gates, bad = _select(c, groups)
    # (no limit, or one past T, is a limit of T, which only expert 0 can pass here)
    keep = ref.keep_of(idx, E, min(capacity or T, T), bool(flags & moe.MOE_FLAG_SLOT_MAJOR))
    want = [*ref.counts(idx, keep, E), torch.tensor([int(bad.sum())], dtype=torch.int32)]
    for got, w, m in zip(ints, want, many):
        assert torch.equal(got, w) and torch.equal(got, m)
    assert int(ints[0].sum()) == T * k and int(ints[2][0]) == int((ints[0] - ints[1]).sum())
    # each token whose chosen logits are finite, several slots of one expert as one of their gates' sum
    merged, first = gates * keep, keep.clone()
    for t in range(T):
        for j in range(k):
            if not first[t, j]:
                continue
            for i in range(j + 1, k):
                if first[t, i] and idx[t, i] == idx[t, j]:
                    merged[t, j] += merged[t, i]
                    first[t, i] = False
    ok = gates.isfinite().all(1)
    exact = [w.double() for w in c["w"]]
    good, bound = ref.experts(torch.where(ok[:, None], c["x"], 0 * torch.ones_like(c["x"])), exact,
                              idx, torch.where(ok[:, None], merged, 0 * merged), first,
                              2.0 ** -8, 8.0)
    over = (out.double() - good).abs() - bound
    assert bool((over[ok] <= 0).all())
    # (a token whose kept slots are none gives zeros, whatever its gates are)
    mine = ~ok & keep.any(1)
    assert not bool(out[mine].isfinite().any()) and not bool(many_out[mine].isfinite().any())
    return ok, bad


VARIANTS = [(0, 0), (1, 0), (2, 0), (3, moe.MOE_FLAG_SLOT_MAJOR), (1, moe.MOE_FLAG_SLOT_MAJOR),
            (5, moe.MOE_FLAG_PAD_TO_CAPACITY)]


@pytest.mark.parametrize("capacity,flags", VARIANTS)
@pytest.mark.parametrize("T,E,k", [(5, 8, 2), (16, 6, 3), (9, 70, 8), (16, 300, 5), (4, 4, 4)])
def test_tokens_without_a_finite_logit(T, E, k, capacity, flags):
    c = _case(T, E, k, seed=T + E)
    c["x"][1, 100] = float("nan")
    c["x"][T - 1, 3] = float("inf")
    c["b"][0] += 0.5  # others choose expert 0 too, and compete with them for its places
    ok, bad = _check(c, capacity, flags)
    assert int((~ok).sum()) == 2 == int(bad.sum())


@pytest.mark.parametrize("capacity,flags", VARIANTS)
@pytest.mark.parametrize("lost", [[3, 4], [1, 2, 3, 4], [2, 4]])
def test_fewer_finite_logits_than_slots(lost, capacity, flags):
    """Expert 0's own logit is finite: its gates are, and so is the output."""
    c = _case(11, 5, 4, seed=len(lost))
    c["w_router"][lost] = float("nan")
    ok, bad = _check(c, capacity, flags)
    assert bool(ok.all()) and bool(bad.all())


@pytest.mark.parametrize("capacity,flags", VARIANTS)
def test_expert_0_is_the_one_without_a_logit(capacity, flags):
    c = _case(7, 4, 3, seed=3)
    c["b"][[0, 2]] = float("nan")
    ok, bad = _check(c, capacity, flags)
    assert not bool(ok.any()) and bool(bad.all())


@pytest.mark.parametrize("capacity,flags", [(0, 0), (2, 0), (1, moe.MOE_FLAG_SLOT_MAJOR)])
def test_groups_without_enough_finite_logits(capacity, flags):
    c = _case(8, 8, 4, seed=5)
    c["w_router"][[1, 3, 5, 7]] = float("nan")
    c["x"][6, 0] = float("nan")
    _check(c, capacity, flags, (4, 2))


@pytest.mark.parametrize("capacity,flags", [(0, 0), (1, moe.MOE_FLAG_SLOT_MAJOR)])
@pytest.mark.parametrize("lost", [[1, 2, 3, 4], [0, 1, 2, 3, 4], [1, 3]])
def test_one_token(lost, capacity, flags):
    """One place and several slots of expert 0: the first of them is kept."""
    c = _case(1, 5, 4, seed=21 + len(lost))
    c["w_router"][lost] = float("nan")
    ok, bad = _check(c, capacity, flags)
    assert bool(bad.all()) and bool(ok.all()) == (0 not in lost)


@pytest.mark.parametrize("T", [2, 16])
def test_most_slots_and_experts(T):
    c = _case(T, 1024, 512 // 16, seed=T, F=128)
    c["w_router"][20:] = float("nan")
    c["x"][1, 5] = float("nan")
    for capacity, flags in ((0, 0), (3, 0), (T, moe.MOE_FLAG_SLOT_MAJOR)):
        _check(c, capacity, flags)
