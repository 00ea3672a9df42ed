"""Plain 64-bit form of the layer for a few tokens, with bounds on its fp32 error (CPU)."""
from __future__ import annotations

import torch

EPS = 2.0 ** -24


def route(x, w_router, b, k, sel_only=False, groups=(1, 1)):
    """(experts [T, k], gates [T, k], finite [T]) of the exact logits rounded to fp32."""
    logits = x.double() @ w_router.double().t()
    if b is not None and not sel_only:
        logits = logits + b.double()
    logits = logits.float()
    sel = logits + b if b is not None and sel_only else logits
    T, E = logits.shape
    idx, gates = torch.zeros((T, k), dtype=torch.int64), torch.zeros((T, k), dtype=torch.float64)
    for t in range(T):
        v = sel[t].tolist()
        allowed = range(E)
        if groups[0] > 1:
            size = E // groups[0]
            best = [max(v[g * size:(g + 1) * size]) for g in range(groups[0])]
            keep = sorted(range(groups[0]), key=lambda g: (-best[g], g))[:groups[1]]
            allowed = [e for e in range(E) if e // size in keep]
        pick = sorted(allowed, key=lambda e: (-v[e], e))[:k]
        idx[t] = torch.tensor(pick)
        g = logits[t, pick].double()
        g = torch.exp(g - g.max())
        gates[t] = g / g.sum()
    finite = logits.isfinite().all(1) & sel.isfinite().all(1)
    return idx, gates, finite, float(logits[logits.isfinite()].abs().max()) if T else 0.0


def keep_of(idx, E, capacity, slot_major=False):
    T, k = idx.shape
    keep, seen = torch.ones((T, k), dtype=torch.bool), [0] * E
    order = [(t, j) for j in range(k) for t in range(T)] if slot_major else \
            [(t, j) for t in range(T) for j in range(k)]
    for t, j in order:
        e = int(idx[t, j])
        if capacity and seen[e] >= capacity:
            keep[t, j] = False
        seen[e] += 1
    return keep


def counts(idx, keep, E):
    T, k = idx.shape
    routed = torch.bincount(idx.flatten(), minlength=E)
    kept = torch.bincount(idx[keep], minlength=E)
    drops = [int((~keep).sum())] + [int((~keep[:, j]).sum()) for j in range(k)]
    drops.append(int((~keep).all(1).sum()) if k else 0)
    return routed.int(), kept.int(), torch.tensor(drops, dtype=torch.int32)


def experts(x, weights, idx, gates, keep, half, largest_logit=1.0):
    """(out, bound): weights = (gate, up, down) in 64 bits, stacked; half: half a step of h's and
    the output's type.  Every sum of n terms is within n 2^-24 of its magnitudes."""
    x = x.double()
    T, d = x.shape
    out, mag, err = (torch.zeros((T, d), dtype=torch.float64) for _ in range(3))
    terms = 16
    for e in sorted(set(idx[keep].tolist())):
        at, slot = torch.nonzero((idx == e) & keep, as_tuple=True)
        g, u, w = (m[e] for m in weights)
        a, b = x[at] @ g.t(), x[at] @ u.t()
        n = (d + d // 128 + 4) * EPS
        ea, eb = n * (x[at].abs() @ g.abs().t()), n * (x[at].abs() @ u.abs().t())
        s = a * torch.sigmoid(a)
        es = 1.1 * ea + EPS * (a.abs() + ea + 8) * (s.abs() + ea)  # silu's slope stays below 1.1
        h = s * b
        eh = s.abs() * eb + b.abs() * es + es * eb + EPS * h.abs()
        eh = eh + (half + EPS) * (h.abs() + eh)
        gate = gates[at, slot][:, None]
        out[at] += gate * (h @ w.t())
        err[at] += gate * (eh @ w.abs().t())
        mag[at] += gate * ((h.abs() + eh) @ w.abs().t())
        terms += h.shape[1] + h.shape[1] // 32
    # sums, and the gates: exp of a difference of logits within (2 |L| + 16) 2^-24 of itself
    err = err + (terms + 4 * largest_logit + 32) * EPS * mag
    return out, err + half * (out.abs() + err)


