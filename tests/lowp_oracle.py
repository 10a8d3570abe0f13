"""Plain 64-bit forms of the low-precision and expert-grouped products, on the CPU, and the
bounds that the kernels' results are held to.

Bounds: a sum of n products held in FP32 in any order is off by at most n u S, S the sum of
the products' magnitudes and u = 2^-23 (the matrix cores may cut rather than round the bits
below); scaling a block's sum and adding it rounds four more times at most; the result is
rounded once to its type, by half a step, or half of the smallest step near zero."""
import torch

BLOCK = 128
F8 = torch.float8_e4m3fn
U = 2.0 ** -23


def blocks(n):
    return -(-n // BLOCK)


def quantize(x, block_rows):
    """(values, scales) from the definition, both float64."""
    x = x.double().cpu()
    rows, cols = x.shape
    rb, cb = -(-rows // block_rows), blocks(cols)
    v = torch.zeros(rows, cols, dtype=torch.float64)
    s = torch.zeros(rb, cb, dtype=torch.float64)
    for i in range(rb):
        for j in range(cb):
            b = x[i * block_rows:(i + 1) * block_rows, j * BLOCK:(j + 1) * BLOCK]
            fin = torch.where(torch.isfinite(b), b, torch.zeros_like(b))
            top = float(fin.abs().max())
            e = -126
            while top > 448.0 * 2.0 ** e:
                e += 1
            s[i, j] = 2.0 ** e
            q = fin / 2.0 ** e
            step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 3)
            q = torch.round(q / step) * step
            q[~torch.isfinite(b)] = float("nan")
            v[i * block_rows:(i + 1) * block_rows, j * BLOCK:(j + 1) * BLOCK] = q
    return v, s


def values(q, s, block_rows):
    """What 8-bit q with scales s stands for, float64."""
    rows, cols = q.shape
    r = torch.arange(rows) // block_rows
    k = torch.arange(cols) // BLOCK
    return q.cpu().double() * s.cpu().double()[r][:, k]


def product(a, b):
    """(a b, |a| |b|) in float64."""
    return a @ b, a.abs() @ b.abs()


def ranges(offsets):
    o = [int(v) for v in offsets]
    return [(o[e], o[e + 1]) for e in range(len(o) - 1)]


def check(got, ref, mag, n, name=""):
    """got against ref, whose sums of n products have magnitudes mag."""
    t = torch.finfo(got.dtype)
    g = got.detach().double().cpu()
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    tol = (n + 8) * U * mag * (1 + t.eps) + ref.abs() * (t.eps / 2) + \
        t.smallest_normal * t.eps / 2
    bad = ~((g - ref).abs() <= tol)
    assert not bad.any(), (name, int(bad.sum()), float(((g - ref).abs() / tol).nan_to_num(9e9).max()))
