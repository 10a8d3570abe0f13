"""Plain 64-bit forms of the operators around the experts' products, on the CPU, and the bounds that
the kernels' results are held to.

Bounds: u = 2^-23 for one operation of FP32 (which may cut rather than round the bits below), a sum
of n terms in any order is off by at most n u S, S the sum of the terms' magnitudes; exp and the
division of FP32 by 2 u each, the exponential's argument by u of its size; the result is rounded once
to its type, by half a step, or half of the smallest step near zero."""
import math

import numpy as np
import torch

U = 2.0 ** -23
TINY = 2.0 ** -125  # exponentials below the smallest normal number may be 0


def close(got, ref, slack, name=""):
    """got within `slack` (and the rounding to its type) of ref; NaN where ref has it."""
    t = torch.finfo(got.dtype)
    g = got.detach().double().cpu()
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(g), nan), (name, "NaN", int(torch.isnan(g).sum()), int(nan.sum()))
    g, ref = torch.where(nan, 0.0, g), torch.where(nan, 0.0, ref)
    # rounding to the nearest gives Inf from half a step past the largest number on
    ref = torch.where(ref.abs() >= t.max * (1 + t.eps / 4), ref * math.inf, ref)
    slack = torch.where(nan, 0.0, torch.as_tensor(slack, dtype=torch.float64).expand(ref.shape))
    tol = slack * (1 + t.eps) + ref.abs() * (t.eps / 2) + t.smallest_normal * t.eps / 2
    off = (g - ref).abs()
    bad = ~((off <= tol) | (g == ref))
    assert not bad.any(), (name, int(bad.sum()), float((off / tol).nan_to_num(9e9).max()))


# ---------------------------------------------------------------------------------- router
def route(x, k, valid, norm):
    """dict of the definition's results in float64, with what the bounds need."""
    x = x.detach().double().cpu()
    T, E = x.shape
    on = torch.ones(T, dtype=torch.bool) if valid is None else valid.cpu().clone()
    on &= (x > -math.inf).any(1) | torch.isnan(x).any(1)
    top = torch.where(on, torch.nan_to_num(x, nan=-math.inf, posinf=math.inf, neginf=-math.inf).amax(1), 0.0)
    e = torch.exp(x - top[:, None])
    p = torch.where(on[:, None], e / e.sum(1, keepdim=True), 0.0)
    experts = np.full((T, k), -1, dtype=np.int64)
    xs = x.numpy()
    for t in range(T):
        if on[t]:
            # NaN first, then by size, of equal ones the lowest index
            rank = sorted(range(E), key=lambda i: (not math.isnan(xs[t, i]), -xs[t, i] if not math.isnan(xs[t, i]) else 0.0, i))
            for j, i in enumerate(rank[:k]):
                if not xs[t, i] == -math.inf:
                    experts[t, j] = i
    experts = torch.from_numpy(experts)
    taken = experts >= 0
    gates = torch.where(taken, p.gather(1, experts.clamp_min(0)), 0.0)
    total = gates.sum(1, keepdim=True)
    if norm:
        gates = torch.where(taken, gates / total, 0.0)
    counts = torch.bincount(experts[taken], minlength=E)
    n, all_ = int(on.sum()), int(counts.sum())
    loss = E * (counts.double() / max(all_, 1) * p.sum(0) / max(n, 1)).sum()
    far = torch.where(torch.isfinite(x), top[:, None] - x, 0.0).clamp_min(0)  # exp's argument
    return dict(on=on, p=p, experts=experts, gates=gates, counts=counts, loss=loss, n=n, all=all_,
                far=far, E=E, k=k, norm=norm, total=total)


def check_route(r, gates, experts, counts, loss):
    E, far = r["E"], r["far"]
    assert torch.equal(experts.cpu().long(), r["experts"])
    assert torch.equal(counts.cpu().long(), r["counts"])
    # p: exp's argument, exp, the sum of E of them, the quotient
    rel = U * (E + 8 + 2 * far)
    slack = r["gates"].abs() * rel.gather(1, r["experts"].clamp_min(0))
    if r["norm"]:  # a second quotient, over k of them
        slack = slack + r["gates"].abs() * (U * (r["k"] + 4) + rel.amax(1, keepdim=True))
    close(gates, r["gates"], slack + TINY / r["total"].clamp_min(1e-9) if r["norm"] else slack + TINY, "gates")
    # (terms of one sign: relative bounds add up)
    most = torch.where(torch.isfinite(r["p"]), r["p"] * rel, 0.0).sum(0)
    slack = E * (r["counts"].double() / max(r["all"], 1) * most / max(r["n"], 1)).sum()
    close(loss, r["loss"], slack + r["loss"].abs() * U * (r["on"].numel() + 8), "loss")


def route_grad(r, dgates, dloss):
    """(dx, bound) of the definition's gradient."""
    p, E, taken = r["p"], r["E"], r["experts"] >= 0
    idx = r["experts"].clamp_min(0)
    dg = torch.zeros_like(r["gates"]) if dgates is None else torch.where(taken, dgates.double().cpu(), 0.0)
    unit = 0.0 if dloss is None else float(dloss) * E / max(r["n"], 1) / max(r["all"], 1)
    G = (unit * r["counts"].double()).expand_as(p).clone()
    mag = G.abs()
    rel = U * (2 * E + 24 + 4 * r["far"])
    extra = torch.zeros_like(p)
    slack = torch.zeros_like(p)
    if r["norm"]:
        g = r["gates"]
        extra.scatter_add_(1, idx, torch.where(taken, g * (dg - (dg * g).sum(1, keepdim=True)), 0.0))
        size = torch.where(taken, g * (dg.abs() + (dg.abs() * g).sum(1, keepdim=True)), 0.0)
        slack.scatter_add_(1, idx, size)
        slack *= rel.amax(1, keepdim=True) + U * r["k"]
    else:
        G.scatter_add_(1, idx, dg)
        mag.scatter_add_(1, idx, dg.abs())
    dx = p * (G - (p * G).sum(1, keepdim=True)) + extra
    slack = slack + p * (mag + (p * mag).sum(1, keepdim=True)) * (rel + rel.amax(1, keepdim=True))
    on = r["on"][:, None]
    return torch.where(on, dx, 0.0), torch.where(on, slack, 0.0) + TINY * (1 + mag.amax())


# --------------------------------------------------------------------------------- adapters
def adapters(y, x, a, b, order, offsets, scale, dout=None):
    """[(name, result, bound)] in float64: out, and dx, da, db where dout is given."""
    y, x, a, b = (t.detach().double().cpu() for t in (y, x, a, b))
    E, rank, K = a.shape
    N = b.shape[2]
    s = torch.ones(E, dtype=torch.float64) if scale is None else scale.double().cpu()
    out, dx, da, db = y.clone(), torch.zeros_like(x), torch.zeros_like(a), torch.zeros_like(b)
    mo, mx, ma, mb = (torch.zeros_like(t) for t in (out, x, a, b))
    d = None if dout is None else dout.double().cpu()
    o = offsets.tolist()
    for e in range(E):
        rows = order[o[e]:o[e + 1]].cpu()
        u, mu = s[e] * (x[rows] @ a[e].t()), s[e].abs() * (x[rows].abs() @ a[e].abs().t())
        out[rows] += u @ b[e]
        mo[rows] = mu @ b[e].abs() * (K + rank + 16) * U + y[rows].abs() * U
        if d is None:
            continue
        v, mv = s[e] * (d[rows] @ b[e].t()), s[e].abs() * (d[rows].abs() @ b[e].abs().t())
        dx[rows], mx[rows] = v @ a[e], mv @ a[e].abs() * (N + rank + 16) * U
        da[e], ma[e] = v.t() @ x[rows], mv.t() @ x[rows].abs() * (N + len(rows) + 16) * U
        db[e], mb[e] = u.t() @ d[rows], mu.t() @ d[rows].abs() * (K + len(rows) + 16) * U
    res = [("out", out, mo)]
    return res if d is None else res + [("dx", dx, mx), ("da", da, ma), ("db", db, mb)]


# ------------------------------------------------------------------------------- gated unit
def gated(x, dh, values=None):
    """((h, bound), (dx, bound)); values: gate and up as they are kept, or None for x's."""
    x, dh = x.detach().double().cpu(), dh.double().cpu()
    N = x.shape[1] // 2
    g, u = x[:, :N], x[:, N:]
    h = g * torch.sigmoid(g) * u
    mh = h.abs() * U * (12 + 2 * g.abs()) + (g * u).abs() * TINY
    if values is not None:
        g, u = values[:, :N], values[:, N:]
    s, rest = torch.sigmoid(g), torch.sigmoid(-g)
    dx = torch.cat([dh * u * s * (1 + g * rest), dh * g * s], 1)
    rel = U * (24 + 4 * g.abs())
    m = torch.cat([(dh * u * s).abs() * (1 + (g * rest).abs()) * rel +
                   (dh * u).abs() * (1 + g.abs()) * TINY,
                   (dh * g * s).abs() * rel + (dh * g).abs() * TINY], 1)
    return (h, mh), (dx, m)
