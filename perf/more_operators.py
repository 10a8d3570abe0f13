"""What a layer of experts needs around its products, as it is measured: cases, inputs, a plain
form of each operator in elementary torch operations, the calls that a user makes, and the results
from their definitions in 64 bits.

Operators:
  route     softmax over the experts, the k best of each row, rows of each expert, balance loss;
            as a training step with the gradient of the logits
  group     rows in the order of their experts, where each went, and where each expert's begin
  adapters  y + scale_e (x A_e^T) B_e, an adapter of low rank for each row's request; as a
            training step with the gradients of y, x, A and B
  gated     silu(gate) up with its backward pass from values kept in 8 bits, or from its input
  kept      an expert-grouped product's training step that keeps its rows in 8 bits
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # a decode batch's router (latency): no gradient, gates that add up to one
        dict(name="route_decode", op="route", T=16, E=64, k=4, dtype="f32", norm=True, pad=0.0,
             blocked=False, step=False),
        # a training batch's router: many experts, padding between the sequences
        dict(name="route_step", op="route", T=16384, E=256, k=8, dtype="f32", norm=True, pad=0.1,
             blocked=False, step=True),
        # odd sizes, 16-bit logits, experts that are not to be had for some rows
        dict(name="route_step_odd", op="route", T=999, E=60, k=3, dtype="bf16", norm=False, pad=0.2,
             blocked=True, step=True),
        # the rows of the same decode batch, and of the same training batch, by expert
        dict(name="group_decode", op="group", n=64, E=64, none=0.0),
        dict(name="group_train", op="group", n=131072, E=256, none=0.1),
        # a decode batch of requests with their own adapters beside a square projection
        dict(name="adapters_decode", op="adapters", T=32, E=64, active=24, none=0.1, K=4096, N=4096,
             r=16, dtype="bf16", step=False),
        # prompts of a dozen requests beside a wide one
        dict(name="adapters_prefill", op="adapters", T=4096, E=16, active=12, none=0.1, K=4096,
             N=11008, r=16, dtype="bf16", step=False),
        # a few adapters trained together
        dict(name="adapters_step", op="adapters", T=8192, E=4, active=4, none=0.0, K=4096, N=4096,
             r=32, dtype="bf16", step=True),
        # the hidden values of an expert layer's training batch, kept in 8 bits
        dict(name="gated_step", op="gated", T=16384, N=2048, dtype="bf16", keep=True),
        # odd sizes in FP32, kept as they are
        dict(name="gated_step_odd", op="gated", T=333, N=1285, dtype="f32", keep=False),
        # an expert product's training step whose rows are kept in 8 bits
        dict(name="kept_step", op="kept", T=16384, pad=0, E=32, active=32, K=4096, N=2048,
             dtype="bf16", tw=False),
        # odd sizes, idle experts, rows of no expert at the end
        dict(name="kept_step_odd", op="kept", T=999, pad=25, E=12, active=9, K=321, N=515,
             dtype="f16", tw=True),
    ]


def _size(rng, lo, hi):
    """A size between lo and hi, even over its logarithm; one in three is left odd, the others
    are multiples of 16 where that leaves something."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = min(max(n, lo), hi)
    if rng.random() < 0.34:
        return min(n | 1, hi)
    return n // 16 * 16 if n >= 16 else n


def draw(rng):
    op = rng.choice(["route", "group", "adapters", "gated", "kept"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    if op == "route":
        E = _size(rng, 2, 512)
        return dict(op=op, T=_size(rng, 1, 16384 * 256 // max(E, 256)), E=E, k=rng.randint(1, min(E, 8)), dtype=dtype,
                    norm=rng.random() < 0.5, pad=rng.choice([0.0, 0.3 * rng.random()]),
                    blocked=rng.random() < 0.3, step=rng.random() < 0.7)
    if op == "group":
        return dict(op=op, n=_size(rng, 1, 131072), E=_size(rng, 1, 512),
                    none=rng.choice([0.0, 0.3 * rng.random()]))
    if op == "adapters":
        E = _size(rng, 1, 64)
        active = rng.randint(max(1, E // 4), E)
        step = rng.random() < 0.5
        return dict(op=op, T=max(active, _size(rng, 1, 4096)), E=E, active=active,
                    none=rng.choice([0.0, 0.3 * rng.random()]), K=_size(rng, 64, 4096),
                    N=_size(rng, 64, 8192), r=rng.choice([1, 4, 8, 9, 16, 24, 32, 64, 100, 128]),
                    dtype=dtype, step=step)
    if op == "gated":
        return dict(op=op, T=_size(rng, 1, 8192), N=_size(rng, 64, 4096 if dtype != "f32" else 2048),
                    dtype=dtype, keep=rng.random() < 0.6)
    E = _size(rng, 2, 32)
    active = rng.randint(max(1, E // 4), E)
    T = max(active, _size(rng, 4, 8192 if dtype != "f32" else 2048))
    return dict(op=op, T=T, pad=rng.choice([0, 0, rng.randint(1, 40)]), E=E, active=active,
                K=_size(rng, 64, 4096), N=_size(rng, 64, 2048), dtype=dtype, tw=rng.random() < 0.5)


# ------------------------------------------------------------------------------ inputs
def _activations(gen, rows, cols, dtype):
    """Normal values whose columns differ in size, as activations do."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    x *= torch.exp(0.7 * torch.randn(cols, generator=gen, device="cuda"))
    return x.to(dtype)


def _normal(gen, scale, dtype, *shape):
    return (scale * torch.randn(*shape, generator=gen, device="cuda")).to(dtype)


def _sizes(T, E, active, seed):
    """Rows of each of E groups: `active` of them have at least one, some many more than others."""
    r = np.random.RandomState(seed % (1 << 31))
    share = np.exp(0.8 * r.randn(active))
    sizes = np.zeros(E, dtype=np.int64)
    sizes[np.sort(r.permutation(E)[:active])] = 1 + r.multinomial(T - active, share / share.sum())
    return sizes


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "route":
        T, E = case["T"], case["E"]
        # some experts are liked by all rows, as early in training
        x = 1.5 * torch.randn(T, E, generator=gen, device="cuda")
        x += torch.randn(E, generator=gen, device="cuda")
        if case["blocked"]:
            at = torch.rand(T, E, generator=gen, device="cuda") < torch.rand(T, 1, generator=gen, device="cuda")
            x[at] = -math.inf
            x[torch.rand(T, generator=gen, device="cuda") < 0.05] = -math.inf  # none at all
        s["logits"] = x.to(DTYPES[case["dtype"]]).requires_grad_(case["step"])
        s["valid"] = None
        if case["pad"]:
            s["valid"] = torch.rand(T, generator=gen, device="cuda") >= case["pad"]
        s["dgates"] = 0.01 * torch.randn(T, case["k"], generator=gen, device="cuda")
        s["dloss"] = torch.full((), 0.02, device="cuda")
    elif op == "group":
        r = np.random.RandomState(seed % (1 << 31))
        share = np.exp(0.8 * r.randn(case["E"]))
        e = r.choice(case["E"], size=case["n"], p=share / share.sum()).astype(np.int32)
        e[r.rand(case["n"]) < case["none"]] = -1
        s["experts"] = torch.from_numpy(e).cuda()
    elif op == "adapters":
        T, E, K, N, rank = (case[n] for n in ("T", "E", "K", "N", "r"))
        dt = DTYPES[case["dtype"]]
        used = max(case["active"], T - int(case["none"] * T))
        sizes = _sizes(used, E, case["active"], seed)
        # rows come in the order of the batch; the plan, made once for all of its projections,
        # sorts them by adapter, rows without one last
        order = torch.randperm(T, generator=gen, device="cuda")
        at = [0] + [int(v) for v in np.cumsum(sizes)]
        for lo, hi in zip(at, at[1:] + [T]):
            order[lo:hi] = order[lo:hi].sort().values
        s["sizes"], s["order"] = [int(v) for v in sizes], order
        s["offsets"] = torch.tensor(at, dtype=torch.int32, device="cuda")
        s["scale"] = 0.5 + torch.rand(E, generator=gen, device="cuda")
        s["x"] = _activations(gen, T, K, dt).requires_grad_(case["step"])
        s["y"] = _normal(gen, 1.0, dt, T, N).requires_grad_(case["step"])
        s["a"] = _normal(gen, K ** -0.5, dt, E, rank, K).requires_grad_(case["step"])
        s["b"] = _normal(gen, 0.5 * rank ** -0.5, dt, E, rank, N).requires_grad_(case["step"])
        if case["step"]:
            s["dout"] = _normal(gen, 0.01, dt, T, N)
    elif op == "gated":
        dt = DTYPES[case["dtype"]]
        s["x"] = _activations(gen, case["T"], 2 * case["N"], dt).requires_grad_()
        s["dh"] = _normal(gen, 0.01, dt, case["T"], case["N"])
    else:
        dt = DTYPES[case["dtype"]]
        rows, E, K, N = case["T"] + case["pad"], case["E"], case["K"], case["N"]
        sizes = _sizes(case["T"], E, case["active"], seed)
        s["sizes"] = [int(v) for v in sizes]
        s["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device="cuda")
        s["x"] = _activations(gen, rows, K, dt).requires_grad_()
        s["w"] = _normal(gen, 0.02, dt, *((E, N, K) if case["tw"] else (E, K, N))).requires_grad_()
        s["dy"] = _normal(gen, 0.01, dt, rows, N)
    return s


# ------------------------------------------------------- the plain form, and the user's calls
def _route(x, valid, k, norm, E):
    """(gates, experts, counts, loss, p, share of each expert's rows, counted rows) in 32 bits."""
    x = x.float()
    top = x.max(dim=1, keepdim=True).values
    on = top[:, 0] > -math.inf
    if valid is not None:
        on = on & valid
    p = torch.exp(x - torch.where(on[:, None], top, torch.zeros_like(top)))
    p = torch.where(on[:, None], p / p.sum(1, keepdim=True), torch.zeros_like(p))
    v, i = torch.sort(x, dim=1, descending=True, stable=True)
    v, i = v[:, :k], i[:, :k]
    taken = on[:, None] & (v > -math.inf)
    gates = torch.where(taken, p.gather(1, i), torch.zeros_like(v))
    if norm:
        gates = gates / torch.where(on, gates.sum(1), torch.ones_like(top[:, 0]))[:, None]
    experts = torch.where(taken, i, torch.full_like(i, -1)).int()
    counts = (experts.flatten()[:, None] == torch.arange(E, device=x.device)).sum(0).int()
    rows = on.sum().clamp_min(1).float()
    share = counts.float() / counts.sum().clamp_min(1).float()
    loss = E * (share * (p.sum(0) / rows)).sum()
    return gates, experts, counts, loss, p, share, rows


def _quantized(x):
    """The values that x has in 8 bits (e4m3fn) with one power-of-two scale for each 128 of a row:
    the smallest that brings their largest magnitude to 448 or less."""
    rows, cols = x.shape
    kb = -(-cols // BLOCK)
    p = torch.nn.functional.pad(x.float(), (0, kb * BLOCK - cols)).view(rows, kb, BLOCK)
    m, e = torch.frexp(p.abs().amax(dim=2))
    e = torch.where(m > 0, e - 9 + (m > 0.875).int(), -126).clamp_min(-126)
    s = torch.ldexp(torch.ones_like(m), e)[:, :, None]
    return ((p / s).to(torch.float8_e4m3fn).float() * s).view(rows, kb * BLOCK)[:, :cols]


def _per_group(s):
    at = 0
    for e, n in enumerate(s["sizes"]):
        if n:
            yield e, at, at + n
        at += n


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "route":
        x = s["logits"].detach()
        E, k = c["E"], c["k"]
        gates, experts, counts, loss, p, share, rows = _route(x, s["valid"], k, c["norm"], E)
        if not c["step"]:
            return gates, experts, counts, loss
        i, taken = experts.clamp_min(0).long(), experts >= 0
        dg = torch.where(taken, s["dgates"], torch.zeros_like(gates))
        dp = (s["dloss"] * E / rows * share).expand_as(p)
        dx = torch.zeros_like(p)
        if c["norm"]:
            dx.scatter_add_(1, i, gates * (dg - (dg * gates).sum(1, keepdim=True)))
        else:
            dp = dp.clone().scatter_add_(1, i, dg)
        dx += p * (dp - (p * dp).sum(1, keepdim=True))
        return gates, experts, counts, loss, dx.to(x.dtype)
    if op == "group":
        e, E = s["experts"].long(), c["E"]
        e = torch.where((e < 0) | (e >= E), torch.full_like(e, E), e)
        order = torch.sort(e, stable=True).indices
        place = torch.empty_like(order)
        place[order] = torch.arange(e.numel(), device=e.device)
        ends = torch.searchsorted(e[order], torch.arange(E + 1, device=e.device))
        return order, place, ends.int()
    if op == "adapters":
        x, y, a, b = (s[n].detach() for n in "xyab")
        out = y.clone()
        dx, da, db = (torch.zeros_like(t) for t in (x, a, b)) if c["step"] else (None,) * 3
        for e, lo, hi in _per_group(s):
            at = s["order"][lo:hi]
            ae, be = a[e].float(), b[e].float()
            xe = x[at].float()
            u = (xe @ ae.t()) * s["scale"][e]
            out[at] = (y[at].float() + u @ be).to(y.dtype)
            if c["step"]:
                de = s["dout"][at].float()
                v = (de @ be.t()) * s["scale"][e]
                dx[at] = (v @ ae).to(x.dtype)
                da[e] = (v.t() @ xe).to(x.dtype)
                db[e] = (u.t() @ de).to(x.dtype)
        return (out, s["dout"], dx, da, db) if c["step"] else out
    if op == "gated":
        x = s["x"].detach()
        g, u = x.float().split(c["N"], dim=1)
        h = (g * torch.sigmoid(g) * u).to(x.dtype)
        if c["keep"]:
            g, u = _quantized(x[:, :c["N"]]), _quantized(x[:, c["N"]:])
        dh, sg = s["dh"].float(), torch.sigmoid(g)
        return h, torch.cat([dh * u * sg * (1 + g * (1 - sg)), dh * g * sg], dim=1).to(x.dtype)
    x, w, dy = s["x"].detach(), s["w"].detach(), s["dy"]
    kept = _quantized(x)
    y = torch.zeros(x.shape[0], c["N"], dtype=x.dtype, device=x.device)
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    for e, lo, hi in _per_group(s):
        we, de = w[e].float(), dy[lo:hi].float()
        if c["tw"]:
            we = we.t()
        y[lo:hi] = (x[lo:hi].float() @ we).to(x.dtype)
        dx[lo:hi] = (de @ we.t()).to(x.dtype)
        g = kept[lo:hi].t() @ de
        dw[e] = (g.t() if c["tw"] else g).to(w.dtype)
    return y, dx, dw


def _calls(s):
    import tiled_double_buffered_amd as tdb
    c = s["case"]
    op = c["op"]
    if op == "route":
        gates, experts, counts, loss = tdb.route_experts(s["logits"], c["k"], valid=s["valid"],
                                                         renormalize=c["norm"])
        if not c["step"]:
            return gates, experts, counts, loss
        dx, = torch.autograd.grad((gates, loss), s["logits"], (s["dgates"], s["dloss"]))
        return gates.detach(), experts, counts, loss.detach(), dx
    if op == "group":
        return tdb.group_rows(s["experts"], c["E"])
    if op == "adapters":
        out = tdb.add_adapters(s["y"], s["x"], s["a"], s["b"], s["order"], s["offsets"], scale=s["scale"])
        if not c["step"]:
            return out
        return (out.detach(),) + torch.autograd.grad(out, [s[n] for n in "yxab"], s["dout"])
    if op == "gated":
        h = tdb.gated_silu(s["x"], checkpoint=c["keep"])
        return (h.detach(),) + torch.autograd.grad(h, (s["x"],), s["dh"])
    y = tdb.linear_grouped(s["x"], s["w"], s["offsets"], transpose_w=c["tw"], checkpoint=True)
    return (y.detach(),) + torch.autograd.grad(y, (s["x"], s["w"]), s["dy"])


def run(state):
    return _calls(state) if own else _plain(state)


# ------------------------------------------------------------------- work and exact results
def work(case):
    op = case["op"]
    if op == "route":
        T, E, k, z = case["T"], case["E"], case["k"], SIZE[case["dtype"]]
        n = T * E * z + 8 * T * k + 4 * E + 4 + (T if case["pad"] else 0)
        if case["step"]:
            n += T * E * z + 4 * T * k + 4
        return dict(bytes=n, flops=T * E * (12 if case["step"] else 5))
    if op == "group":
        return dict(bytes=case["n"] * (4 + 8 + 8) + 4 * (case["E"] + 1), flops=0)
    if op == "adapters":
        T, E, K, N, r = (case[n] for n in ("T", "E", "K", "N", "r"))
        z = SIZE[case["dtype"]]
        used = max(case["active"], T - int(case["none"] * T))
        n = z * (used * K + 2 * T * N + case["active"] * r * (K + N)) + 8 * T + 8 * E
        flops = 2 * used * r * (K + N)
        if case["step"]:  # dout is dy; dx, da and db are written whole
            n += z * (used * N + T * K + E * r * (K + N))
            flops *= 3
        return dict(bytes=n, flops=flops)
    if op == "gated":
        T, N, z = case["T"], case["N"], SIZE[case["dtype"]]
        n = z * T * N * (2 + 1 + 1 + 2)  # x, h, dh, dx
        return dict(bytes=n, flops=20 * T * N)
    T, rows, E, a, K, N = case["T"], case["T"] + case["pad"], case["E"], case["active"], case["K"], case["N"]
    z = SIZE[case["dtype"]]
    return dict(bytes=z * (T * K + a * K * N + rows * N + T * N + rows * K + E * K * N), flops=6 * T * N * K)


def _exact_8_bits(x):
    """Definition in 64 bits: the scale 2^p with the smallest p >= -126 for which no magnitude of
    a row's 128 passes 448 * 2^p, and the nearest value of the 8-bit format (4 exponent bits, 3
    mantissa bits, the smallest exponent -6), ties to the even one."""
    rows, cols = x.shape
    out = torch.empty(rows, cols, dtype=torch.float64, device=x.device)
    for j in range(0, cols, BLOCK):
        v = x[:, j:j + BLOCK].double()
        scale = torch.exp2(torch.ceil(torch.log2(v.abs().amax(1, keepdim=True) / 448.0)).clamp_min(-126.0))
        v = v / scale
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
        out[:, j:j + BLOCK] = torch.round(v / step) * step * scale
    return out


def _exact_route(st):
    c = st["case"]
    E, k = c["E"], c["k"]
    x = st["logits"].detach().double()
    dev = x.device
    raw = x.cpu().numpy()
    on = np.isfinite(raw).any(1)
    if st["valid"] is not None:
        on &= st["valid"].cpu().numpy()
    # best first, of equal ones the lowest index: two keys, the second the index itself
    order = np.lexsort((np.broadcast_to(np.arange(E), raw.shape), -raw), axis=1)[:, :k]
    chosen = np.where(on[:, None] & np.isfinite(np.take_along_axis(raw, order, 1)), order, -1)
    counts = np.bincount(chosen[chosen >= 0], minlength=E)
    p = torch.zeros_like(x)
    live = torch.from_numpy(on).to(dev)
    p[live] = torch.softmax(x[live], dim=1)
    pick = torch.from_numpy(np.eye(E + 1)[:, :E][np.where(chosen < 0, E, chosen)]).to(dev)  # T x k x E, 0 or 1
    gates = (pick * p[:, None, :]).sum(2)
    total = gates.sum(1, keepdim=True).clamp_min(1e-300)
    if c["norm"]:
        gates = gates / total
    f = torch.from_numpy(counts / max(counts.sum(), 1)).to(dev)
    rows = max(int(on.sum()), 1)
    loss = E * torch.dot(f, p.sum(0) / rows)
    res = (gates, torch.from_numpy(chosen.astype(np.int32)), torch.from_numpy(counts.astype(np.int32)), loss)
    if not c["step"]:
        return res
    dg = st["dgates"].double()
    if c["norm"]:  # through the division by the sum of the taken ones
        dg = (dg - (dg * gates).sum(1, keepdim=True)) / total
    dp = (pick * dg[:, :, None]).sum(1) + float(st["dloss"]) * E / rows * f
    return res + (p * (dp - (p * dp).sum(1, keepdim=True)),)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(st)
    if op == "group":
        e = st["experts"].cpu().numpy().astype(np.int64)
        e = np.where(e < 0, case["E"], e)
        order = np.argsort(e, kind="stable")
        ends = np.cumsum(np.bincount(e, minlength=case["E"] + 1))[:case["E"]]
        offsets = np.concatenate([[0], ends]).astype(np.int32)
        return torch.from_numpy(order), torch.from_numpy(np.argsort(order, kind="stable")), torch.from_numpy(offsets)
    if op == "gated":
        N = case["N"]
        x, dh = st["x"].detach().double(), st["dh"].double()
        g, u = x[:, :N], x[:, N:]
        h = u * g / (1 + torch.exp(-g))
        if case["keep"]:
            g, u = _exact_8_bits(g), _exact_8_bits(u)
        e = torch.exp(-g)
        dx = torch.empty_like(x)
        dx[:, :N] = dh * u * (1 + e + g * e) / (1 + e) ** 2
        dx[:, N:] = dh * g / (1 + e)
        return h, dx
    at = np.concatenate([[0], np.cumsum(st["sizes"])])
    if op == "adapters":
        x, y, a, b = (st[n].detach().double() for n in "xyab")
        out = y.clone()
        if case["step"]:
            dout = st["dout"].double()
            dx, da, db = torch.zeros_like(x), torch.zeros_like(a), torch.zeros_like(b)
        for e in range(case["E"]):
            rows = st["order"][int(at[e]):int(at[e + 1])]
            if not len(rows):
                continue
            full = float(st["scale"][e]) * (a[e].t() @ b[e])  # K x N, the adapter as one matrix
            out[rows] += x[rows] @ full
            if case["step"]:
                dx[rows] = dout[rows] @ full.t()
                g = float(st["scale"][e]) * (x[rows].t() @ dout[rows])  # its gradient, K x N
                da[e] = (g @ b[e].t()).t()
                db[e] = a[e] @ g
        return (out, dout, dx, da, db) if case["step"] else out
    x, w, dy = st["x"].detach(), st["w"].detach(), st["dy"]
    y = torch.zeros(x.shape[0], case["N"], dtype=torch.float64, device=x.device)
    dx = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    dw = torch.zeros(w.shape, dtype=torch.float64, device=x.device)
    for e in range(case["E"]):
        i, j = int(at[e]), int(at[e + 1])
        if j > i:
            we, de = w[e].double(), dy[i:j].double()
            kept = _exact_8_bits(x[i:j])
            y[i:j] = x[i:j].double() @ (we.t() if case["tw"] else we)
            dx[i:j] = de @ (we if case["tw"] else we.t())
            dw[e] = de.t() @ kept if case["tw"] else kept.t() @ de
    return y, dx, dw
