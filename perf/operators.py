"""The low-precision and grouped matrix products of this library, as they are measured:
cases, inputs, a plain form of each operator in elementary torch operations, the calls that
a user makes, and the results from their definitions in 64 bits.

Operators:
  quantize     values -> 8-bit floating point with one scale for each block of 128
  fp8          C = (A sa) (B sb)^T, 8-bit operands with a scale for each block of 128
  fp8_step     a linear layer's training step on 8-bit operands: y, dx, dw
  fp8_grouped  the fp8 product with one B per expert and ragged row groups
  grouped      y = x_e w_e per expert with ragged row groups, in 16 or 32 bits
  grouped_step its training step: y, dx, dw
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
F8 = torch.float8_e4m3fn


def blocks(n):
    return -(-n // BLOCK)


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # activations of a decode batch, quantized before a layer's product (latency)
        dict(name="quantize_decode", op="quantize", M=16, K=4096, dtype="bf16", block=1, pair=False),
        # activations of a training batch: by rows for y, transposed for the weight gradient
        dict(name="quantize_train", op="quantize", M=8192, K=8192, dtype="bf16", block=1, pair=True),
        # one token against a layer (latency and the rate at which the weights are read)
        dict(name="fp8_decode", op="fp8", M=1, N=11008, K=4096, out="bf16"),
        # odd sizes throughout: rows that are not 16-byte aligned, partial blocks
        dict(name="fp8_ragged", op="fp8", M=513, N=1285, K=2053, out="f32"),
        # a prompt against a layer
        dict(name="fp8_prefill", op="fp8", M=4096, N=11008, K=4096, out="bf16"),
        # a training step of a linear layer, its quantizations included
        dict(name="fp8_step", op="fp8_step", M=8192, N=4096, K=4096, dtype="bf16"),
        # expert products: a decode batch, where most experts have no row
        dict(name="grouped_decode", op="grouped", T=16, pad=0, E=64, active=14, K=4096, N=2048,
             dtype="bf16", tw=False),
        # expert products: a training step
        dict(name="grouped_step", op="grouped_step", T=16384, pad=0, E=32, active=32, K=4096,
             N=2048, dtype="bf16", tw=False),
        # odd sizes, idle experts, rows of no expert at the end
        dict(name="grouped_step_odd", op="grouped_step", T=999, pad=25, E=12, active=9, K=321,
             N=515, dtype="f16", tw=True),
        # the same in FP32, where FP32 master weights are multiplied
        dict(name="grouped_step_f32", op="grouped_step", T=2048, pad=0, E=8, active=8, K=1024,
             N=2048, dtype="f32", tw=False),
        # quantized experts: a prompt, and a decode batch
        dict(name="fp8_grouped_prefill", op="fp8_grouped", T=8192, pad=0, E=16, active=16,
             K=4096, N=2048, out="bf16"),
        dict(name="fp8_grouped_decode", op="fp8_grouped", T=32, pad=0, E=64, active=24, K=4096,
             N=2048, out="bf16"),
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
    op = rng.choice(["quantize", "fp8", "fp8_step", "fp8_grouped", "grouped", "grouped_step"])
    if op == "quantize":
        return dict(op=op, M=_size(rng, 1, 8192), K=_size(rng, 64, 8192),
                    dtype=rng.choice(["bf16", "f16", "f32"]), block=rng.choice([1, 128]),
                    pair=rng.random() < 0.5)
    if op == "fp8":
        return dict(op=op, M=_size(rng, 1, 4096), N=_size(rng, 64, 11008),
                    K=_size(rng, 64, 8192), out=rng.choice(["bf16", "f16", "f32"]))
    if op == "fp8_step":
        return dict(op=op, M=_size(rng, 64, 8192), N=_size(rng, 64, 4096),
                    K=_size(rng, 64, 4096), dtype=rng.choice(["bf16", "f16"]))
    E = _size(rng, 2, 64)
    active = rng.randint(max(1, E // 4), E)
    c = dict(op=op, T=max(active, _size(rng, 4, 8192)), pad=rng.choice([0, 0, rng.randint(1, 40)]),
             E=E, active=active, K=_size(rng, 64, 4096), N=_size(rng, 64, 2048))
    if op == "fp8_grouped":
        c["out"] = rng.choice(["bf16", "f16", "f32"])
    else:
        c["dtype"] = rng.choice(["bf16", "f16", "f32"])
        c["tw"] = rng.random() < 0.5
        if c["dtype"] == "f32":  # the FP32 matrix rate is a fraction of the 16-bit one
            c["T"] = max(active, c["T"] // 4)
    return c


# ------------------------------------------------------------------------------ inputs
def _activations(gen, rows, cols, dtype):
    """Normal values whose columns differ in size, as activations do."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    x *= torch.exp(0.7 * torch.randn(cols, generator=gen, device="cuda"))
    return x.to(dtype)


def _to_fp8(x, block_rows):
    """x (..., rows, cols) as 8-bit values and scales of any size (the largest of each
    block_rows x 128 block becomes 448), the way a checkpoint holds them."""
    *lead, rows, cols = x.shape
    rb, cb = -(-rows // block_rows), blocks(cols)
    p = torch.zeros(*lead, rb * block_rows, cb * BLOCK, device=x.device)
    p[..., :rows, :cols] = x
    s = p.view(*lead, rb, block_rows, cb, BLOCK).abs().amax(dim=(-3, -1)).clamp_min(1e-20) / E4M3_MAX
    q = (p.view(*lead, rb, block_rows, cb, BLOCK) / s[..., :, None, :, None]).to(F8)
    return q.view(*lead, rb * block_rows, cb * BLOCK)[..., :rows, :cols].contiguous(), s


def _sizes(case, seed):
    """Rows of each expert: `active` of them have at least one, some many more than others."""
    r = np.random.RandomState(seed % (1 << 31))
    T, E, a = case["T"], case["E"], case["active"]
    share = np.exp(0.8 * r.randn(a))
    n = 1 + r.multinomial(T - a, share / share.sum())
    sizes = np.zeros(E, dtype=np.int64)
    sizes[np.sort(r.permutation(E)[:a])] = n
    return [int(v) for v in sizes]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "quantize":
        s["x"] = _activations(gen, case["M"], case["K"], DTYPES[case["dtype"]])
    elif op == "fp8":
        s["a"], s["sa"] = _to_fp8(_activations(gen, case["M"], case["K"], torch.float32), 1)
        s["b"], s["sb"] = _to_fp8(0.02 * torch.randn(case["N"], case["K"], generator=gen, device="cuda"), BLOCK)
    elif op == "fp8_step":
        dt = DTYPES[case["dtype"]]
        s["x"] = _activations(gen, case["M"], case["K"], dt).requires_grad_()
        s["w"] = (0.02 * torch.randn(case["N"], case["K"], generator=gen, device="cuda")).to(dt).requires_grad_()
        s["dy"] = (0.01 * torch.randn(case["M"], case["N"], generator=gen, device="cuda")).to(dt)
    else:
        sizes = _sizes(case, seed)
        rows, E, K, N = case["T"] + case["pad"], case["E"], case["K"], case["N"]
        s["sizes"] = sizes
        s["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device="cuda")
        if op == "fp8_grouped":
            s["a"], s["sa"] = _to_fp8(_activations(gen, rows, K, torch.float32), 1)
            s["b"], s["sb"] = _to_fp8(0.02 * torch.randn(E, N, K, generator=gen, device="cuda"), BLOCK)
        else:
            dt = DTYPES[case["dtype"]]
            x = _activations(gen, rows, K, dt)
            w = (0.02 * torch.randn(*((E, N, K) if case["tw"] else (E, K, N)), generator=gen, device="cuda")).to(dt)
            step = op == "grouped_step"
            s["x"], s["w"] = x.requires_grad_(step), w.requires_grad_(step)
            if step:
                s["dy"] = (0.01 * torch.randn(rows, N, generator=gen, device="cuda")).to(dt)
    return s


# ------------------------------------------------------- the plain form, and the user's calls
def _quantize(x, block_rows):
    """(8-bit values, power-of-two scales) of x: each block_rows x 128 block's scale is the
    smallest power of two that brings its largest magnitude to 448 or less."""
    rows, cols = x.shape
    rb, cb = -(-rows // block_rows), blocks(cols)
    p = torch.nn.functional.pad(x.float(), (0, cb * BLOCK - cols, 0, rb * block_rows - rows))
    p = p.view(rb, block_rows, cb, BLOCK)
    m, e = torch.frexp(p.abs().amax(dim=(1, 3)))
    e = torch.where(m > 0, e - 9 + (m > 0.875).int(), -126).clamp_min(-126)
    s = torch.ldexp(torch.ones_like(m), e)
    q = (p / s[:, None, :, None]).view(rb * block_rows, cb * BLOCK)[:rows, :cols]
    return q.to(F8), s


def _values(q, s, block_rows):
    """The values that 8-bit q with scales s stands for, in 32 bits."""
    rows, cols = q.shape[-2:]
    s = s.repeat_interleave(BLOCK, -1)[..., :cols]
    return q.float() * (s if block_rows == 1 else s.repeat_interleave(block_rows, -2)[..., :rows, :])


def _per_expert(sizes, product):
    return [product(e, n) for e, n in enumerate(sizes)]


def _grouped(x, w, sizes, dtype):
    """Each expert's rows of x (32 bits) times its w; zeros for the rows of no expert."""
    parts = x.split(sizes + [x.shape[0] - sum(sizes)])
    y = _per_expert(sizes, lambda e, n: (parts[e] @ w[e].float()).to(dtype))
    return torch.cat(y + [torch.zeros(parts[-1].shape[0], w.shape[2], dtype=dtype, device=x.device)])


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "quantize":
        q, sc = _quantize(s["x"], c["block"])
        if not c["pair"]:
            return q, sc
        if c["block"] == BLOCK:
            return q, sc, q.t().contiguous(), sc.t().contiguous()
        return (q, sc) + _quantize(s["x"].t(), 1)
    if op == "fp8":
        return (_values(s["a"], s["sa"], 1) @ _values(s["b"], s["sb"], BLOCK).t()).to(DTYPES[c["out"]])
    if op == "fp8_step":
        x, w, dy = s["x"].detach(), s["w"].detach(), s["dy"]
        wq = _values(*_quantize(w, BLOCK), BLOCK)
        y = (_values(*_quantize(x, 1), 1) @ wq.t()).to(x.dtype)
        dx = (_values(*_quantize(dy, 1), 1) @ wq).to(x.dtype)
        dw = _values(*_quantize(dy.t(), 1), 1) @ _values(*_quantize(x.t(), 1), 1).t()
        return y, dx, dw.to(w.dtype)
    if op == "fp8_grouped":
        a, sizes, dt = _values(s["a"], s["sa"], 1), s["sizes"], DTYPES[c["out"]]
        parts = a.split(sizes + [c["pad"]])
        y = _per_expert(sizes, lambda e, n: (parts[e] @ _values(s["b"][e], s["sb"][e], BLOCK).t()).to(dt)
                        if n else parts[e].new_zeros(0, c["N"], dtype=dt))
        return torch.cat(y + [torch.zeros(c["pad"], c["N"], dtype=dt, device=a.device)])
    sizes, x, w = s["sizes"], s["x"].detach(), s["w"].detach()
    wkn = w.transpose(1, 2) if c["tw"] else w
    y = _grouped(x.float(), wkn, sizes, x.dtype)
    if op == "grouped":
        return y
    dy = s["dy"].float()
    dx = _grouped(dy, wkn.transpose(1, 2), sizes, x.dtype)
    xs, ds = x.float().split(sizes + [c["pad"]]), dy.split(sizes + [c["pad"]])
    left, right = (ds, xs) if c["tw"] else (xs, ds)
    dw = torch.stack(_per_expert(sizes, lambda e, n: (left[e].t() @ right[e]).to(w.dtype)))
    return y, dx, dw


def _calls(s):
    import tiled_double_buffered_amd as tdb
    c = s["case"]
    op = c["op"]
    if op == "quantize":
        block = (c["block"], BLOCK)
        return tdb.quantize_fp8_pair(s["x"], block=block) if c["pair"] else tdb.quantize_fp8(s["x"], block=block)
    if op == "fp8":
        return tdb.matmul_fp8(s["a"], s["sa"], s["b"], s["sb"], out_dtype=DTYPES[c["out"]])
    if op == "fp8_step":
        y = tdb.linear_fp8(s["x"], s["w"])
        return (y.detach(),) + torch.autograd.grad(y, (s["x"], s["w"]), s["dy"])
    if op == "fp8_grouped":
        return tdb.matmul_fp8_grouped(s["a"], s["sa"], s["b"], s["sb"], s["offsets"], out_dtype=DTYPES[c["out"]])
    if op == "grouped":
        return tdb.matmul_grouped(s["x"], s["w"], s["offsets"], transpose_w=c["tw"])
    y = tdb.linear_grouped(s["x"], s["w"], s["offsets"], transpose_w=c["tw"])
    return (y.detach(),) + torch.autograd.grad(y, (s["x"], s["w"]), s["dy"])


def run(state):
    return _calls(state) if own else _plain(state)


# ------------------------------------------------------------------- work and exact results
def work(case):
    op = case["op"]
    if op == "quantize":
        M, K = case["M"], case["K"]
        out = M * K + 4 * blocks(K) * (M if case["block"] == 1 else blocks(M))
        return dict(bytes=M * K * SIZE[case["dtype"]] + out * (2 if case["pair"] else 1), flops=0)
    if op == "fp8":
        M, N, K = case["M"], case["N"], case["K"]
        return dict(bytes=M * K + N * K + 4 * blocks(K) * (M + blocks(N)) + M * N * SIZE[case["out"]],
                    flops=2 * M * N * K)
    if op == "fp8_step":
        M, N, K = case["M"], case["N"], case["K"]
        return dict(bytes=2 * SIZE[case["dtype"]] * (M * K + N * K + M * N), flops=6 * M * N * K)
    T, rows, E, a, K, N = case["T"], case["T"] + case["pad"], case["E"], case["active"], case["K"], case["N"]
    if op == "fp8_grouped":
        return dict(bytes=T * K + 4 * T * blocks(K) + a * (N * K + 4 * blocks(N) * blocks(K))
                    + rows * N * SIZE[case["out"]], flops=2 * T * N * K)
    z = SIZE[case["dtype"]]
    if op == "grouped":
        return dict(bytes=z * (T * K + a * K * N + rows * N), flops=2 * T * N * K)
    return dict(bytes=z * (T * K + a * K * N + rows * N + T * N + rows * K + E * K * N), flops=6 * T * N * K)


def _exact_fp8(x, block_rows):
    """Definition in 64 bits: the scale 2^p with the smallest p for which no magnitude of the
    block passes 448 * 2^p, and the nearest value of the 8-bit format (4 exponent bits, 3
    mantissa bits, the smallest exponent -6), ties to the even one."""
    x = x.double()
    rows, cols = x.shape
    rb, cb = -(-rows // block_rows), blocks(cols)
    big = x.new_zeros(rb * block_rows, cb * BLOCK)
    big[:rows, :cols] = x
    big = big.reshape(rb, block_rows, cb, BLOCK).permute(0, 2, 1, 3)
    top = big.abs().flatten(2).max(dim=2).values
    p = torch.ceil(torch.log2(top / E4M3_MAX)).clamp_min(-126.0)
    s = torch.exp2(p)
    v = big / s[:, :, None, None]
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    v = torch.round(v / step) * step
    v = v.permute(0, 2, 1, 3).reshape(rb * block_rows, cb * BLOCK)[:rows, :cols]
    s_of = s.repeat_interleave(block_rows, 0).repeat_interleave(BLOCK, 1)[:rows, :cols]
    return v, s, v * s_of


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        v, s, _ = _exact_fp8(st["x"], case["block"])
        if not case["pair"]:
            return v, s
        vt, sct, _ = _exact_fp8(st["x"].t(), case["block"])
        return v, s, vt, sct

    def full(q, s, block_rows):
        rows, cols = q.shape
        r = torch.arange(rows, device=q.device) // block_rows
        k = torch.arange(cols, device=q.device) // BLOCK
        return q.double() * s.double()[r][:, k]

    if op == "fp8":
        return full(st["a"], st["sa"], 1) @ full(st["b"], st["sb"], BLOCK).t()
    if op == "fp8_step":
        x, w, dy = st["x"].detach(), st["w"].detach(), st["dy"]
        w8 = _exact_fp8(w, BLOCK)[2]
        return (_exact_fp8(x, 1)[2] @ w8.t(), _exact_fp8(dy, 1)[2] @ w8,
                _exact_fp8(dy.t(), 1)[2] @ _exact_fp8(x.t(), 1)[2].t())
    at = [0] + [int(v) for v in np.cumsum(st["sizes"])]
    rows, E, K, N = case["T"] + case["pad"], case["E"], case["K"], case["N"]
    dev = st["offsets"].device
    y = torch.zeros(rows, N, dtype=torch.float64, device=dev)
    if op == "fp8_grouped":
        for e in range(E):
            i, j = at[e], at[e + 1]
            if j > i:
                y[i:j] = full(st["a"][i:j], st["sa"][i:j], 1) @ full(st["b"][e], st["sb"][e], BLOCK).t()
        return y
    x, w = st["x"].detach().double(), st["w"].detach()
    step = op == "grouped_step"
    dy = st["dy"].double() if step else None
    dx = torch.zeros(rows, K, dtype=torch.float64, device=dev)
    dw = torch.zeros(w.shape, dtype=torch.float64, device=dev) if step else None
    for e in range(E):
        i, j = at[e], at[e + 1]
        if j > i:
            we = w[e].double().t() if case["tw"] else w[e].double()
            y[i:j] = x[i:j] @ we
            if step:
                dx[i:j] = dy[i:j] @ we.t()
                g = x[i:j].t() @ dy[i:j]
                dw[e] = g.t() if case["tw"] else g
    return (y, dx, dw) if step else y
