"""The low-precision and expert-grouped products on the GPU against plain 64-bit forms
(tests/lowp_oracle.py, which derives the bounds)."""
import sys

import pytest

torch = pytest.importorskip("torch")
import tiled_double_buffered_amd as tdb  # noqa: E402
from tiled_double_buffered_amd import lowp  # noqa: E402
import lowp_oracle as lo  # noqa: E402

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

DEV = torch.device("cuda:0")
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
NAN = float("nan")


def _say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(params=["", "256", "128", "64", "644"], ids=lambda v: f"tile{v or '-auto'}")
def tile(request, monkeypatch):
    """Every tile's kernel, wherever it takes the operands, besides the one that is chosen."""
    if request.param:
        monkeypatch.setenv("GEMM_LP_TILE", request.param)
    return request.param


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g)


# ------------------------------------------------------------------------------ quantization
def _wide(rows, cols, dtype, seed):
    """Values of very different sizes, zero blocks, halves of a step, 448 and just above."""
    g = _gen(seed)
    x = _randn(g, rows, cols) * torch.exp2(torch.randint(-9, 5, (rows, cols), generator=g).float())
    if dtype != torch.float16:
        x *= torch.exp2(torch.randint(-60, 60, (rows, 1), generator=g).float())
    x[rows // 2] = 0.0
    x[0, 0] = 448.0
    x[0, cols - 1] = 449.0
    x[rows - 1, 0] = 1.0625
    return x.to(dtype)


def _same(q, s, v, sc):
    assert q.dtype == lo.F8 and s.dtype == torch.float32
    assert tuple(q.shape) == tuple(v.shape) and tuple(s.shape) == tuple(sc.shape)
    assert torch.equal(s.double().cpu(), sc)
    assert torch.equal(q.float().double().cpu().nan_to_num(9e9), v.nan_to_num(9e9))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("shape", [(1, 1), (1, 128), (3, 129), (16, 512), (130, 257), (257, 136),
                                   (64, 1000)], ids=str)
def test_quantize(shape, block, dtype):
    x = _wide(*shape, TYPES[dtype], 11 + shape[0] + shape[1])
    xd = x.to(DEV)
    _say("[quantize]", shape, block, dtype)
    v, s = lo.quantize(x, block)
    vt, st = lo.quantize(x.t(), block)
    _same(*tdb.quantize_fp8(xd, block=(block, 128)), v, s)
    q, sq, qt, sqt = tdb.quantize_fp8_pair(xd, block=(block, 128))
    _same(q, sq, v, s)
    _same(qt, sqt, vt, st)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("shape", [(1, 1), (3, 129), (130, 257), (257, 136)], ids=str)
def test_quantize_exponents(shape, block, dtype):
    """The exponent bytes are the scales', one for each row; the 8-bit values are the same."""
    rows, cols = shape
    x = _wide(rows, cols, TYPES[dtype], 13 + rows).to(DEV)
    x[rows - 1, cols // 2] = float("inf")
    q, s, qt, st = tdb.quantize_fp8_pair(x, block=(block, 128))
    pair = lowp._quantize_exp(x, block, True, True)
    plain = lowp._quantize_exp(x, block, True, False)
    for (e, ex), (v, sc), (r, c) in ((pair[:2], (q, s), shape), (plain[:2], (q, s), shape),
                                     (pair[2:], (qt, st), (cols, rows))):
        assert torch.equal(e[:, :c].view(torch.uint8), v.contiguous().view(torch.uint8))
        exps = torch.log2(sc).to(torch.int32) + 127
        by_row = exps if block == 1 else exps.repeat_interleave(128, 0)[:r]
        assert torch.equal(ex[:, :r].t().to(torch.int32), by_row)


@pytest.mark.parametrize("block", [1, 128])
def test_quantize_not_finite_and_tiny(block):
    x = _randn(_gen(5), 140, 300)
    x[3, 5] = float("inf")
    x[3, 200] = -float("inf")
    x[139, 299] = NAN
    x[7, :128] = NAN              # a block of nothing else
    x[9] = 2.0 ** -140            # subnormal values: the smallest scale, and zeros
    x[10, :128] = 2.0 ** -126 * 1.75
    x[11, 0] = torch.finfo(torch.float32).max
    v, s = lo.quantize(x, block)
    vt, st = lo.quantize(x.t(), block)
    q, sq, qt, sqt = tdb.quantize_fp8_pair(x.to(DEV), block=(block, 128))
    _same(q, sq, v, s)
    _same(qt, sqt, vt, st)
    _same(*tdb.quantize_fp8(x.to(DEV), block=(block, 128)), v, s)


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_views(dtype):
    """Rows that start at any element and do not fill their stride."""
    big = _randn(_gen(6), 70, 421).to(TYPES[dtype])
    x, xd = big[3:67, 5:398], big.to(DEV)[3:67, 5:398]
    v, s = lo.quantize(x, 1)
    _same(*tdb.quantize_fp8(xd), v, s)
    vt, st = lo.quantize(x.t(), 1)
    _same(*tdb.quantize_fp8_pair(xd)[2:], vt, st)


# ------------------------------------------------------------------------------ 8-bit products
def _scaled(rows, cols, block, seed, lead=()):
    """8-bit values and scales of any size, as a checkpoint holds them."""
    g = _gen(seed)
    q = (_randn(g, *lead, rows, cols) * 60).to(lo.F8)
    s = torch.exp(_randn(g, *lead, -(-rows // block), lo.blocks(cols)))
    return q, s


def _aligned(q):
    """The same values in rows that start at multiples of 16 bytes; the rest of each is NaN."""
    ld = (q.shape[-1] + 15) // 16 * 16
    p = torch.full((*q.shape[:-1], ld), NAN, device=q.device).to(lo.F8)
    p[..., :q.shape[-1]] = q
    return p[..., :q.shape[-1]]


FP8_SHAPES = [(1, 1, 1), (1, 64, 128), (5, 33, 127), (16, 256, 1024), (33, 130, 129),
              (127, 193, 61), (129, 257, 400), (200, 520, 2053), (300, 384, 896), (7, 1000, 4096),
              (512, 512, 640), (260, 264, 1024), (131, 300, 2500)]


@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("b_block", [1, 128])
@pytest.mark.parametrize("shape", FP8_SHAPES, ids=str)
def test_matmul_fp8(shape, b_block, out, tile):
    M, N, K = shape
    a, sa = _scaled(M, K, 1, 21 + M)
    b, sb = _scaled(N, K, b_block, 22 + N)
    ref, mag = lo.product(lo.values(a, sa, 1), lo.values(b, sb, b_block).t())
    if out == "f16":  # into its range
        f = 2.0 ** -12
        sa, ref, mag = sa * f, ref * f, mag * f
    ad, sad, bd, sbd = (t.to(DEV) for t in (a, sa, b, sb))
    for how, (p, r) in dict(plain=(ad, bd), aligned=(_aligned(ad), _aligned(bd)),
                            mixed=(ad, _aligned(bd))).items():
        _say("[matmul_fp8]", shape, b_block, out, how)
        c = tdb.matmul_fp8(p, sad, r, sbd, out_dtype=TYPES[out])
        assert c.dtype == TYPES[out]
        lo.check(c, ref, mag, K, how)


def test_matmul_fp8_no_depth_and_no_rows():
    z = torch.empty(5, 0, device=DEV, dtype=lo.F8)
    s = torch.empty(5, 0, device=DEV)
    c = tdb.matmul_fp8(z, s, z[:3], s[:1])
    assert c.shape == (5, 3) and not c.any()
    a, sa = (t.to(DEV) for t in _scaled(4, 256, 1, 3))
    b, sb = (t.to(DEV) for t in _scaled(4, 256, 128, 3))
    assert tdb.matmul_fp8(a[:0], sa[:0], b, sb).shape == (0, 4)
    assert tdb.matmul_fp8(a, sa, b[:0], sb[:0]).shape == (4, 0)


def _split(sizes, lead, tail):
    """Offsets of groups of these sizes after `lead` rows of no expert; rows with the tail."""
    o = [lead]
    for n in sizes:
        o.append(o[-1] + n)
    return o, o[-1] + tail


# sizes, rows of no expert before and after
GROUPS = [([5], 0, 0), ([1, 0, 3, 0, 0, 7], 0, 0), ([0, 0, 0], 2, 3), ([130, 1, 0, 64], 1, 5),
          ([300, 5, 257], 0, 70), ([0, 17, 33, 0, 1, 1, 1, 128, 16, 0], 0, 1),
          ([1] * 20 + [0] * 50 + [2] * 30, 3, 0)]


@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("groups", GROUPS, ids=lambda g: f"{len(g[0])}e-{sum(g[0])}")
@pytest.mark.parametrize("NK", [(64, 128), (130, 400), (257, 261), (132, 1300)], ids=str)
def test_matmul_fp8_grouped(groups, NK, out, tile):
    N, K = NK
    off, rows = _split(*groups)
    E = len(groups[0])
    a, sa = _scaled(rows, K, 1, 31)
    b, sb = _scaled(N, K, 128, 32, (E,))
    sa *= 2.0 ** -12
    ref = torch.zeros(rows, N, dtype=torch.float64)
    mag = torch.zeros_like(ref)
    av = lo.values(a, sa, 1)
    for e, (i, j) in enumerate(lo.ranges(off)):
        ref[i:j], mag[i:j] = lo.product(av[i:j], lo.values(b[e], sb[e], 128).t())
    a.view(torch.uint8)[:off[0]] = 0x7f  # NaN in the rows of no expert stays out
    a.view(torch.uint8)[off[-1]:] = 0x7f
    offd = torch.tensor(off, dtype=torch.int32, device=DEV)
    ad, sad, bd, sbd = (t.to(DEV) for t in (a, sa, b, sb))
    for how, (p, r) in dict(plain=(ad, bd), aligned=(_aligned(ad), _aligned(bd))).items():
        _say("[matmul_fp8_grouped]", E, rows, NK, out, how)
        lo.check(tdb.matmul_fp8_grouped(p, sad, r, sbd, offd, out_dtype=TYPES[out]), ref, mag, K,
                 how)


# ------------------------------------------------------------------------- expert products
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tw", [False, True])
@pytest.mark.parametrize("groups", GROUPS, ids=lambda g: f"{len(g[0])}e-{sum(g[0])}")
@pytest.mark.parametrize("KN", [(1, 1), (64, 128), (136, 264), (321, 131), (400, 72)], ids=str)
def test_grouped_step(groups, KN, tw, dtype, tile):
    """y, dx and dw of a step, NaN in the rows of no expert (which must not leak)."""
    K, N = KN
    off, rows = _split(*groups)
    E = len(groups[0])
    g = _gen(41 + K)
    x = _randn(g, rows, K).to(TYPES[dtype])
    w = (0.1 * _randn(g, *((E, N, K) if tw else (E, K, N)))).to(TYPES[dtype])
    dy = _randn(g, rows, N).to(TYPES[dtype])
    x64, w64, dy64 = x.double(), w.double(), dy.double()
    ref = [torch.zeros(rows, N).double(), torch.zeros(rows, K).double(), torch.zeros_like(w64)]
    mag = [torch.zeros_like(t) for t in ref]
    for e, (i, j) in enumerate(lo.ranges(off)):
        we = w64[e].t() if tw else w64[e]
        ref[0][i:j], mag[0][i:j] = lo.product(x64[i:j], we)
        ref[1][i:j], mag[1][i:j] = lo.product(dy64[i:j], we.t())
        l, r = (dy64[i:j], x64[i:j]) if tw else (x64[i:j], dy64[i:j])
        ref[2][e], mag[2][e] = lo.product(l.t(), r)
    for t in (x, dy):
        t[:off[0]] = NAN
        t[off[-1]:] = NAN
    _say("[grouped_step]", E, rows, KN, tw, dtype)
    offd = torch.tensor(off, dtype=torch.int32, device=DEV)
    xd, wd = x.to(DEV).requires_grad_(), w.to(DEV).requires_grad_()
    y = tdb.linear_grouped(xd, wd, offd, transpose_w=tw)
    assert y.dtype == x.dtype
    dx, dw = torch.autograd.grad(y, (xd, wd), dy.to(DEV))
    lo.check(y, ref[0], mag[0], K, "y")
    lo.check(dx, ref[1], mag[1], N, "dx")
    lo.check(dw, ref[2], mag[2], max(rows, 1), "dw")
    assert torch.equal(tdb.matmul_grouped(xd.detach(), wd.detach(), offd, transpose_w=tw),
                       y.detach())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tw", [False, True])
def test_grouped_views(dtype, tw, tile):
    """Operands whose rows and experts do not fill their strides."""
    K, N, E = 96, 80, 3
    off, rows = _split([9, 0, 40], 0, 2)
    g = _gen(51)
    bigx = _randn(g, rows, K + 9).to(TYPES[dtype]).to(DEV)
    bigw = _randn(g, E + 2, (N if tw else K) + 3, (K if tw else N) + 5).to(TYPES[dtype]).to(DEV)
    x = bigx[:, 3:3 + K]
    w = bigw[1:1 + E, 2:-1, 3:-2]
    offd = torch.tensor(off, dtype=torch.int32, device=DEV)
    y = tdb.matmul_grouped(x, w, offd, transpose_w=tw)
    ref = torch.zeros(rows, N, dtype=torch.float64)
    mag = torch.zeros_like(ref)
    for e, (i, j) in enumerate(lo.ranges(off)):
        we = w[e].double().cpu()
        ref[i:j], mag[i:j] = lo.product(x[i:j].double().cpu(), we.t() if tw else we)
    lo.check(y, ref, mag, K)


@pytest.mark.parametrize("dtype", TYPES)
def test_inf_and_nan_stay_in_their_rows_and_experts(dtype, tile):
    """An Inf or NaN of one expert's rows reaches that expert's results and no others."""
    K, N, E = 128, 128, 3
    off = [0, 20, 40, 60]
    g = _gen(52)
    x = _randn(g, 60, K).to(TYPES[dtype]).to(DEV)
    w = _randn(g, E, K, N).to(TYPES[dtype]).to(DEV)
    dy = _randn(g, 60, N).to(TYPES[dtype]).to(DEV)
    offd = torch.tensor(off, dtype=torch.int32, device=DEV)
    x[19, 3] = float("inf")
    x[40, 5] = NAN
    dy[20, 0] = NAN
    y = tdb.matmul_grouped(x, w, offd)
    bad = ~torch.isfinite(y).all(1)
    assert bad.nonzero().flatten().tolist() == [19, 40]
    dw = tdb.matmul_grouped_wgrad(x, dy, offd)
    finite = torch.isfinite(dw)
    assert not finite[0, 3].any() and finite[0].sum() == (K - 1) * N
    assert not finite[1, :, 0].any() and finite[1].sum() == K * (N - 1)
    assert not finite[2, 5].any() and finite[2].sum() == (K - 1) * N


def test_wrong_offsets_stay_in_bounds(tile):
    """Offsets past the rows, negative and decreasing ones: the values are undefined, the call
    ends, and what lies around the outputs keeps its values."""
    K, N, E, rows = 64, 64, 4, 50
    g = _gen(53)
    x = _randn(g, rows, K).bfloat16().to(DEV)
    w = _randn(g, E, K, N).bfloat16().to(DEV)
    for off in ([0, 60, 70, 80, 90], [-5, -3, 10, 20, 1 << 30], [50, 40, 30, 20, 10],
                [0, 50, 0, 50, 0], [-(1 << 31), (1 << 31) - 1, 0, 50, -1]):
        offd = torch.tensor(off, dtype=torch.int32, device=DEV)
        _say("[wrong offsets]", off)
        guard = torch.full((rows + 20, N), 7.0, device=DEV).bfloat16()
        rc = tdb.gemm_grouped(rows, N, K, E, offd.data_ptr(), x.data_ptr(), K, w.data_ptr(), N,
                              K * N, 0, guard[10:].data_ptr(), N, 0,
                              torch.cuda.current_stream().cuda_stream)
        assert rc == tdb.OK
        torch.cuda.synchronize()
        assert (guard[:10] == 7).all() and (guard[10 + rows:] == 7).all()
        dw = tdb.matmul_grouped_wgrad(x, x, offd)
        torch.cuda.synchronize()
        assert dw.shape == (E, K, K)


# ------------------------------------------------------------------------------ training steps
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(1, 1, 1), (5, 130, 70), (128, 128, 128), (200, 384, 264),
                                   (257, 129, 513), (1100, 260, 1027)], ids=str)
def test_linear_fp8(shape, dtype, tile):
    M, N, K = shape
    g = _gen(61 + M)
    x = _randn(g, M, K).to(TYPES[dtype])
    w = (0.05 * _randn(g, N, K)).to(TYPES[dtype])
    dy = _randn(g, M, N).to(TYPES[dtype])

    def v(t, b):
        return lo.values(*lo.quantize(t, b), b)

    y64 = lo.product(v(x, 1), v(w, 128).t())
    dx64 = lo.product(v(dy, 1), v(w, 128))
    dw64 = lo.product(v(dy.t(), 1), v(x.t(), 1).t())
    xd, wd = x.to(DEV).requires_grad_(), w.to(DEV).requires_grad_()
    _say("[linear_fp8]", shape, dtype)
    y = tdb.linear_fp8(xd, wd)
    dx, dw = torch.autograd.grad(y, (xd, wd), dy.to(DEV))
    assert y.dtype == dx.dtype == dw.dtype == x.dtype
    lo.check(y, *y64, K, "y")
    lo.check(dx, *dx64, N, "dx")
    lo.check(dw, *dw64, M, "dw")


def test_linear_fp8_leading_axes_and_missing_gradients():
    g = _gen(62)
    x = _randn(g, 3, 5, 64).bfloat16().to(DEV)
    w = _randn(g, 32, 64).bfloat16().to(DEV).requires_grad_()
    y = tdb.linear_fp8(x, w)
    assert y.shape == (3, 5, 32)
    y.sum().backward()  # the gradient of a sum comes as one broadcast value
    assert x.grad is None and w.grad.shape == w.shape
    flat = tdb.linear_fp8(x.view(15, 64), w.detach())
    assert torch.equal(flat.view(3, 5, 32), y.detach()) and not flat.requires_grad
    x.requires_grad_()
    tdb.linear_fp8(x, w.detach()).sum().backward()
    assert x.grad.shape == x.shape


@pytest.mark.parametrize("op", ["fp8", "grouped"])
def test_without_gradients(op):
    """Parameters under no_grad: the same product, nothing to differentiate."""
    x = _randn(_gen(64), 40, 256).bfloat16().to(DEV).requires_grad_()
    w = _randn(_gen(65), 2, 72, 256).bfloat16().to(DEV).requires_grad_()
    off = torch.tensor([0, 11, 40], dtype=torch.int32, device=DEV)

    def f():
        return tdb.linear_fp8(x, w[0]) if op == "fp8" else tdb.linear_grouped(x, w, off, True)

    y = f()
    with torch.no_grad():
        z = f()
    assert y.requires_grad and not z.requires_grad
    assert torch.equal(y.detach(), z)


@pytest.mark.parametrize("op", ["fp8", "grouped"])
def test_gradients_against_differences(op):
    """Both layers are linear wherever the 8-bit values are exact (whole numbers up to 15 are),
    so that differences of the loss are exact too: along any direction of whole numbers,
    loss(x + d) - loss(x) = <dx, d>, and the same in w."""
    g = _gen(63)

    def whole(*shape):
        return torch.randint(-3, 4, shape, generator=g).float().to(DEV)

    x, dy = whole(24, 96), whole(24, 40)
    off = torch.tensor([0, 10, 10, 23], dtype=torch.int32, device=DEV)
    w = whole(40, 96) if op == "fp8" else whole(3, 96, 40)
    f = tdb.linear_fp8 if op == "fp8" else lambda a, b: tdb.linear_grouped(a, b, off)
    xr, wr = x.clone().requires_grad_(), w.clone().requires_grad_()
    dx, dw = torch.autograd.grad(f(xr, wr), (xr, wr), dy)
    loss = lambda a, b: (f(a, b).double() * dy.double()).sum()  # noqa: E731
    for _ in range(3):
        d, v = whole(*x.shape), whole(*w.shape)
        assert loss(x + d, w) - loss(x, w) == (dx.double() * d.double()).sum()
        assert loss(x, w + v) - loss(x, w) == (dw.double() * v.double()).sum()


# -------------------------------------------------------------------- streams and graphs
def test_other_stream():
    x = _randn(_gen(71), 64, 256).bfloat16().to(DEV)
    w = _randn(_gen(72), 128, 256).bfloat16().to(DEV)
    ref = tdb.matmul_fp8(*tdb.quantize_fp8(x), *tdb.quantize_fp8(w, block=(128, 128)))
    torch.cuda.synchronize()
    s = torch.cuda.Stream(DEV)
    q = tdb.quantize_fp8(x, stream=s)
    p = tdb.quantize_fp8(w, block=(128, 128), stream=s)
    c = tdb.matmul_fp8(*q, *p, stream=s)
    s.synchronize()
    assert torch.equal(c, ref)


def test_graph_replays_follow_their_inputs():
    """Captured calls read the offsets and values that the buffers hold at each replay."""
    K, N, E, rows = 192, 160, 4, 90
    x = torch.zeros(rows, K, device=DEV, dtype=torch.bfloat16)
    w = _randn(_gen(73), E, K, N).bfloat16().to(DEV)
    wq, ws = tdb.quantize_fp8(w.view(E * K, N), block=(128, 128))
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    bq = _randn(_gen(75), E, N, K).to(lo.F8).to(DEV)
    bs = torch.ones(E, lo.blocks(N), lo.blocks(K), device=DEV)

    def step():
        q, s, qt, st = tdb.quantize_fp8_pair(x)
        return (tdb.matmul_grouped(x, w, off), tdb.matmul_grouped_wgrad(x, x, off),
                tdb.matmul_fp8_grouped(q, s, bq, bs, off), tdb.matmul_fp8(qt, st, qt, st))

    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed, o in enumerate(([0, 30, 30, 60, 90], [0, 0, 0, 0, 0], [5, 6, 80, 85, 88],
                              [0, 90, 90, 90, 90])):
        x.copy_(_randn(_gen(80 + seed), rows, K).bfloat16())
        off.copy_(torch.tensor(o, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip(held, step()):
            assert torch.equal(got, ref)
    del wq, ws


# --------------------------------------------------------------------------- the layer of experts
def test_expert_layer_trains_and_serves():
    """The products together: the loss falls, and the layer served in 8 bits stays near.  Each
    of the served form's two products in a row has inputs and weights off by at most half a step
    of 2^-4 relative, four roundings that differ from the training form's: 4 * 2^-4."""
    from tiled_double_buffered_amd import expert_layer as el
    layer = el.ExpertLayer(256, 384, 6, DEV)
    losses, x = el.train(layer, 500, 256, 12, DEV)
    assert losses[-1] < 0.8 * losses[0] and all(b == b for b in losses)
    serve = layer.served()
    for n in (500, 33, 1):
        with torch.no_grad():
            ref = layer(x[:n]).float()
        y = serve(x[:n]).float()
        assert y.shape == ref.shape
        assert (y - ref).norm() <= 4 * 2.0 ** -4 * ref.norm()


def test_broadcast_weights_share_their_gradient():
    """One matrix for all experts, as an expanded view: its gradient is the experts' sum."""
    K, N, E = 40, 24, 3
    x = torch.randint(-3, 4, (30, K), generator=_gen(91)).float().to(DEV)
    w = torch.randint(-3, 4, (K, N), generator=_gen(92)).float().to(DEV).requires_grad_()
    off = torch.tensor([0, 4, 4, 30], dtype=torch.int32, device=DEV)
    y = tdb.linear_grouped(x, w.expand(E, K, N), off)
    dy = torch.randint(-3, 4, (30, N), generator=_gen(93)).float().to(DEV)
    (dw,) = torch.autograd.grad(y, w, dy)
    assert torch.equal(y.detach(), x @ w.detach())  # whole numbers: exact
    assert torch.equal(dw, x.t() @ dy)


@pytest.mark.parametrize("op", ["fp8", "grouped"])
def test_only_once_differentiable(op):
    x = _randn(_gen(94), 8, 16).to(DEV).requires_grad_()
    w = _randn(_gen(95), 1, 16, 8).to(DEV)
    off = torch.tensor([0, 8], dtype=torch.int32, device=DEV)
    y = tdb.linear_grouped(x, w, off) if op == "grouped" else tdb.linear_fp8(x, w[0].t().contiguous())
    (dx,) = torch.autograd.grad(y.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        dx.sum().backward()


@pytest.mark.parametrize("spare", [(0, 0), (1, 0), (64, 3), (128, 0), (129, 0), (100, 56), (100, 57)],
                         ids=str)
@pytest.mark.parametrize("kind", ["bf16-256", "f16-256", "f32-256", "f32-64", "f32-644"])
def test_last_round_in_halves(kind, spare, monkeypatch):
    """256 + R whole row tiles of one column, and P groups that end with half a tile or less,
    around the counts at which the last round's tiles are computed in halves (2 R + P <= 256).
    Whole numbers: exact, with one rounding at the end."""
    dtype, tile = kind.split("-")
    monkeypatch.setenv("GEMM_LP_TILE", tile)
    bm = 256 if tile == "256" else 64
    R, P = spare
    E = max(P, 3)
    sizes = [(256 + R) // E * bm] * E
    sizes[-1] += (256 + R) % E * bm
    for e in range(P):
        sizes[e] += 1 + e * 7 % (bm // 2)  # 1 .. half a tile
    if P == 0:
        sizes[0] -= bm // 4  # a whole tile still: more than half of its rows are left
    g = _gen(66)
    rows, K, N = sum(sizes), 72, 40
    off = torch.tensor([0] + sizes, dtype=torch.int64).cumsum(0).int().to(DEV)
    x = torch.randint(-3, 4, (rows, K), generator=g).float().to(DEV)
    w = torch.randint(-3, 4, (E, K, N), generator=g).float().to(DEV)
    expected = torch.cat([a @ b for a, b in zip(x.split(sizes), w)]).to(TYPES[dtype])
    _say("[halves]", kind, spare)
    for tw in (False, True):
        b = (w.transpose(1, 2).contiguous() if tw else w).to(TYPES[dtype])
        y = tdb.matmul_grouped(x.to(TYPES[dtype]), b, off, transpose_w=tw)
        assert torch.equal(y, expected), tw
        one = tdb.matmul_grouped(x.to(TYPES[dtype]), b[:1], off[[0, -1]].contiguous(), transpose_w=tw)
        assert torch.equal(one, (x @ w[0]).to(TYPES[dtype])), tw


# ------------------------------------------------------------------------------- far offsets
def test_rows_and_experts_past_32_bit_offsets():
    """Operands of more than 2^32 bytes: rows and experts at the far end, whole numbers (exact)."""
    if torch.cuda.get_device_properties(0).total_memory < 48 * 2 ** 30:
        pytest.skip("needs 48 GiB")
    rows, K, N = 140000, 32768, 32
    x = torch.zeros(rows, K, dtype=torch.uint8, device=DEV).view(lo.F8)  # 4.6 GB
    far = torch.randint(-3, 4, (5, K), generator=_gen(96)).float().to(DEV)
    x[-5:] = far.to(lo.F8)
    sx = torch.ones(rows, K // 128, device=DEV)
    b = torch.randint(-3, 4, (N, K), generator=_gen(97)).float().to(DEV)
    sb = torch.ones(1, K // 128, device=DEV)
    ref = far.double() @ b.double().t()
    c = tdb.matmul_fp8(x, sx, b.to(lo.F8), sb, out_dtype=torch.float32)
    assert torch.equal(c[-5:].double(), ref) and not c[:-5].any()
    del x, sx, c
    y = torch.zeros(rows, K, dtype=torch.bfloat16, device=DEV)  # 9.2 GB
    y[-5:] = far.bfloat16()
    q, s = tdb.quantize_fp8(y)
    assert torch.equal(q[-5:].float() * s[-5:].repeat_interleave(128, 1), far)
    off = torch.tensor([0, rows - 5, rows], dtype=torch.int32, device=DEV)
    w = torch.stack([torch.zeros_like(b.t()), b.t()]).bfloat16()
    z = tdb.matmul_grouped(y, w, off)
    assert torch.equal(z[-5:], ref.bfloat16()) and not z[:-5].any()
    dw = tdb.matmul_grouped_wgrad(z[:, :8], y, off)
    assert torch.equal(dw[1].float(), (z[-5:, :8].double().t() @ far.double()).bfloat16().float())
    assert not dw[0].any()
    del y, q, s, z, dw
    E = 70
    w = torch.zeros(E, 1024, K, dtype=torch.bfloat16, device=DEV)  # 4.7 GB
    w[-1] = 1.0
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[-1] = 5
    z = tdb.matmul_grouped(far.bfloat16(), w, off, transpose_w=True)
    assert torch.equal(z.float(), far.sum(1, keepdim=True).bfloat16().float().expand(5, 1024))


# -------------------------------------------------------------------- sums of 8-bit values
def _cancelling(M, N, K, seed):
    """(a, b), M x K and N x K whole numbers that 8 bits hold: products of 2^16 and -2^16 cancel,
    anywhere along K, and ones of -1, 0, 1 are what is left of them.  Every partial sum, in any
    order, is a whole number below 2^24, so that FP32 sums are exact."""
    g = _gen(seed)
    a = torch.randint(0, 2, (M, K), generator=g).float()
    b = torch.randint(-1, 2, (N, K), generator=g).float()
    at = torch.randperm(K, generator=g)[:K // 32 * 2]
    plus, minus = at[0::2], at[1::2]
    big = 256.0 * (1 - 2 * torch.randint(0, 2, (M, 1), generator=g).float())
    a[:, plus], a[:, minus] = big, -big
    b[:, at] = 256.0 * (1 - 2 * torch.randint(0, 2, (N, 1), generator=g).float())
    ref, mag = lo.product(a.double(), b.double().t())
    assert mag.max() < 2 ** 24 and ref.abs().max() <= 256  # which every type holds
    assert ref.abs().max() > 0
    return a, b, ref


@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("b_block", [1, 128])
@pytest.mark.parametrize("shape", [(40, 70, 128), (300, 130, 1024), (1, 260, 2053), (130, 300, 3000)],
                         ids=str)
def test_8_bit_sums_hold_32_bits(shape, b_block, out, tile):
    """Small products next to large ones that cancel: what is left of the sum is exact."""
    M, N, K = shape
    a, b, ref = _cancelling(M, N, K, 101 + K)
    g = _gen(102)
    sa = torch.exp2(torch.randint(-2, 3, (M, 1), generator=g).float()).expand(M, lo.blocks(K))
    sb = torch.exp2(torch.randint(-2, 3, (-(-N // b_block), 1), generator=g).float())
    ref = ref * sa[:, :1].double() * sb.double().repeat_interleave(b_block, 0)[:N].t()
    sa, sb = sa.contiguous().to(DEV), sb.expand(-1, lo.blocks(K)).contiguous().to(DEV)
    ad, bd = a.to(lo.F8).to(DEV), b.to(lo.F8).to(DEV)
    for p, r in ((ad, bd), (_aligned(ad), _aligned(bd))):
        _say("[sums]", shape, b_block, out)
        c = tdb.matmul_fp8(p, sa, r, sb, out_dtype=TYPES[out])
        assert torch.equal(c.cpu().double(), ref)


@pytest.mark.parametrize("out", TYPES)
def test_8_bit_sums_of_experts_hold_32_bits(out, tile):
    M, N, K = 70, 130, 1280
    a, b, _ = _cancelling(M, 2 * N, K, 103)
    off, one = [0, 30, 30, M], torch.ones(M, lo.blocks(K), device=DEV)
    w = torch.stack([b[:N], b[:N], b[N:]])
    ref = torch.cat([a[:30].double() @ b[:N].double().t(), a[30:].double() @ b[N:].double().t()])
    c = tdb.matmul_fp8_grouped(a.to(lo.F8).to(DEV), one, w.to(lo.F8).to(DEV),
                               torch.ones(3, lo.blocks(N), lo.blocks(K), device=DEV),
                               torch.tensor(off, dtype=torch.int32, device=DEV), TYPES[out])
    assert torch.equal(c.cpu().double(), ref)


@pytest.mark.parametrize("dtype", TYPES)
def test_8_bit_training_sums_hold_32_bits(dtype, tile):
    """The same along each of the three contractions of a step (256 and 1 are exact in 8 bits
    with any scale that a block of them gets)."""
    for which, (M, N, K) in enumerate(((50, 90, 2048), (50, 2048, 90), (2048, 50, 90))):
        x, w, dy = (torch.zeros(s) for s in ((M, K), (N, K), (M, N)))
        if which == 0:
            x, w, ref = _cancelling(M, N, K, 104)
        elif which == 1:
            dy, wt, ref = _cancelling(M, K, N, 105)
            w = wt.t().contiguous()
        else:
            dyt, xt, ref = _cancelling(N, K, M, 106)
            dy, x = dyt.t().contiguous(), xt.t().contiguous()
        xd, wd = (t.to(TYPES[dtype]).to(DEV).requires_grad_() for t in (x, w))
        _say("[training sums]", dtype, which)
        y = tdb.linear_fp8(xd, wd)
        got = (y.detach(), *torch.autograd.grad(y, (xd, wd), dy.to(TYPES[dtype]).to(DEV)))
        assert torch.equal(got[which].cpu().double(), ref), which


@pytest.mark.parametrize("K", [1024, 8192])
@pytest.mark.parametrize("b_block", [1, 128])
def test_8_bit_sums_are_off_by_little_in_the_mean(K, b_block, tile):
    """n roundings of at most 2^-23 of partial sums that stay under 4 sqrt(n) p (p the products'
    root mean square), with no common sign: together 4 n p 2^-23 in the mean square, and the sum
    of magnitudes is n p / 2 at least for normal values, so 8 * 2^-23 of it."""
    a, sa = _scaled(64, K, 1, 107)
    b, sb = _scaled(96, K, b_block, 108)
    sa = torch.exp2(torch.round(torch.log2(sa[:, :1]))).expand(sa.shape).contiguous()
    sb = torch.ones_like(sb)
    ref, mag = lo.product(lo.values(a, sa, 1), lo.values(b, sb, b_block).t())
    c = tdb.matmul_fp8(*(t.to(DEV) for t in (a, sa, b, sb)), out_dtype=torch.float32)
    off = (c.cpu().double() - ref).square().mean().sqrt()
    assert off <= 8 * 2.0 ** -23 * mag.square().mean().sqrt()


@pytest.mark.parametrize("shape", [(3, 5, 0), (0, 5, 64), (4, 0, 64), (64,), (0,)], ids=str)
def test_linear_fp8_empty_and_leading_axes(shape):
    """No rows, no depth and a single row: the axes that a linear layer gives, and zeros."""
    K = shape[-1]
    x = torch.zeros(shape, device=DEV).requires_grad_()
    w = _randn(_gen(109), 7, K).to(DEV).requires_grad_()
    y = tdb.linear_fp8(x, w)
    assert y.shape == (*shape[:-1], 7) and not y.any()
    dx, dw = torch.autograd.grad(y, (x, w), torch.ones_like(y))
    assert dx.shape == x.shape and dw.shape == w.shape and not dw.any()


@pytest.mark.parametrize("block", [1, 128])
def test_quantize_more_rows_than_an_axis_of_workgroups(block):
    """Past 65535 blocks of rows; a short last one.  Whole numbers up to 15: exact."""
    rows, cols = 65536 * 128 + 40, 8
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    some = torch.randint(-15, 16, (300, cols), generator=_gen(110)).bfloat16().to(DEV)
    x[-300:], x[:300] = some, some.flip(0)
    _say("[tall]", block)
    q, s, qt, st = tdb.quantize_fp8_pair(x, block=(block, 128))
    assert qt.shape == (cols, rows) and st.shape == ((cols, 1)[block == 128], rows // 128 + 1)
    for at in (slice(0, 300), slice(rows - 300, rows)):
        r = torch.arange(rows, device=DEV)[at]
        assert torch.equal(q[at].float() * s[r // block], x[at].float())
        scale = st[:, r // 128] if block == 1 else st[0, r // 128]
        assert torch.equal(qt[:, at].float() * scale, x[at].float().t())
    assert not q[300:-300].view(torch.uint8).any() and not qt[:, 300:-300].float().any()


def test_tall_training_step():
    """linear_fp8 of more rows than that: the weight gradient sums over all of them, exactly."""
    rows = 65536 * 128 + 3
    x = torch.zeros(rows, 8, dtype=torch.bfloat16, device=DEV)
    x[-5:] = torch.randint(-3, 4, (5, 8), generator=_gen(111)).bfloat16().to(DEV)
    x[0] = 1.0
    w = torch.randint(-3, 4, (16, 8), generator=_gen(112)).bfloat16().to(DEV).requires_grad_()
    y = tdb.linear_fp8(x, w)
    assert torch.equal(y[-5:].float(), x[-5:].float() @ w.detach().float().t())
    (dw,) = torch.autograd.grad(y, w, torch.ones_like(y))
    assert torch.equal(dw.float(), x.float().sum(0).expand(16, 8))


@pytest.mark.parametrize("width, hidden", [(200, 300), (129, 40), (384, 256)])
def test_expert_layer_serves_any_width(width, hidden):
    """Widths that blocks of 128 do not divide; within the same 4 * 2^-4 of the training form."""
    from tiled_double_buffered_amd import expert_layer as el
    layer = el.ExpertLayer(width, hidden, 5, DEV)
    x = _randn(_gen(113), 77, width).bfloat16().to(DEV)
    serve = layer.served()
    for n in (77, 1):
        with torch.no_grad():
            ref = layer(x[:n]).float()
        y = serve(x[:n]).float()
        assert (y - ref).norm() <= 4 * 2.0 ** -4 * ref.norm()


def _stream_calls():
    """Every call that takes a stream, as (name, call of tensors, fresh tensors)."""
    x = _randn(_gen(114), 64, 256).bfloat16().to(DEV)
    w = _randn(_gen(115), 2, 256, 128).bfloat16().to(DEV)
    off = torch.tensor([0, 20, 64], dtype=torch.int32, device=DEV)
    a, sa = tdb.quantize_fp8(x)
    b, sb = tdb.quantize_fp8(w[0].t().contiguous(), block=(128, 128))
    bb, sbb = torch.stack([b.view(torch.uint8)] * 2).view(b.dtype), torch.stack([sb] * 2)
    return [("quantize", tdb.quantize_fp8, (x,)), ("pair", tdb.quantize_fp8_pair, (x,)),
            ("fp8", tdb.matmul_fp8, (a, sa, b, sb)),
            ("fp8_grouped", tdb.matmul_fp8_grouped, (a, sa, bb, sbb, off)),
            ("grouped", tdb.matmul_grouped, (x, w, off)),
            ("wgrad", tdb.matmul_grouped_wgrad, (x, x.clone(), off))]


def test_operands_dropped_after_a_call_on_another_stream():
    """While the stream is busy with other work, the memory of operands that the caller dropped
    is not handed out again; and the results are the operands'."""
    side = torch.cuda.Stream(DEV)
    for name, call, tensors in _stream_calls():
        ref = call(*tensors)
        own = [t.clone() for t in tensors]
        torch.cuda.synchronize()
        held = {t.data_ptr() for t in own}
        _say("[dropped]", name)
        with torch.cuda.stream(side):
            torch.cuda._sleep(50_000_000)
        got = call(*own, stream=side)
        sizes = [t.numel() * t.element_size() for t in own]
        del own
        again = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in sizes]
        assert not side.query(), "the other work was over too soon to tell"
        assert not held & {t.data_ptr() for t in again}, name
        side.synchronize()
        for g, r in zip(*((v if isinstance(v, tuple) else (v,)) for v in (got, ref))):
            assert torch.equal(g.float(), r.float()), name


def test_stream_of_another_device_is_refused():
    class Elsewhere:
        device = torch.device("cuda:1")

    for name, call, tensors in _stream_calls():
        with pytest.raises(ValueError, match="stream is on cuda:1"):
            call(*tensors, stream=Elsewhere())


# ------------------------------------------------------------- whole 256x256 tiles, step by step
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tiles", [(16, 16), (11, 35)], ids=["256", "385"])
@pytest.mark.parametrize("steps, short", [(1, 0), (1, 3), (2, 0), (2, 5), (3, 1), (4, 0), (9, 7)])
def test_whole_tiles_of_any_depth(steps, short, tiles, dtype, monkeypatch):
    """As many 256x256 tiles as are never computed in halves (256, or more than 128 past that), of
    one group and of ragged ones, from a single K step to the loop's steady state.  Whole numbers:
    exact, with one rounding at the end."""
    monkeypatch.setenv("GEMM_LP_TILE", "256")
    tm, tn = tiles
    K = steps * (32 if dtype == "f32" else 64) - short
    sizes = [(tm - 9) * 256, 4 * 256 - 50, 0, 5 * 256]  # (the second ends with more than half a tile)
    rows, N = sum(sizes), tn * 256 - 6
    g = _gen(116)
    x = torch.randint(-3, 4, (rows, K), generator=g).float().to(DEV)
    w = torch.randint(-3, 4, (4, K, N), generator=g).float().to(DEV)
    off = torch.tensor([0] + sizes).cumsum(0).int().to(DEV)
    each = torch.cat([a @ b for a, b in zip(x.split(sizes), w)]).to(TYPES[dtype])
    one = (x @ w[0]).to(TYPES[dtype])
    _say("[whole tiles]", steps, short, tiles, dtype)
    for tw in (False, True):
        b = (w.transpose(1, 2).contiguous() if tw else w).to(TYPES[dtype])
        xd = x.to(TYPES[dtype])
        if K % 4:  # rows that start at multiples of four bytes, NaN between them
            xd = torch.nn.functional.pad(xd, (0, 4 - K % 4), value=NAN)[:, :K]
            if tw:
                b = torch.nn.functional.pad(b, (0, 4 - K % 4), value=NAN)[..., :K]
        assert torch.equal(tdb.matmul_grouped(xd, b, off, transpose_w=tw), each), tw
        ends = off[[0, -1]].contiguous()
        assert torch.equal(tdb.matmul_grouped(xd, b[:1], ends, transpose_w=tw), one), tw


@pytest.mark.parametrize("dtype", TYPES)
def test_whole_weight_gradient_tiles_of_any_depth(dtype, monkeypatch):
    """Experts of no row, one row, and one to nine K steps, whole and not."""
    monkeypatch.setenv("GEMM_LP_TILE", "256")
    ks = 32 if dtype == "f32" else 64
    sizes = [0, 1, ks, ks + 1, 2 * ks, 3 * ks - 5, 4 * ks, 9 * ks - 1]
    g = _gen(117)
    x = torch.randint(-3, 4, (sum(sizes), 512), generator=g).float().to(DEV)
    dy = torch.randint(-3, 4, (sum(sizes), 768), generator=g).float().to(DEV)
    off = torch.tensor([0] + sizes).cumsum(0).int().to(DEV)
    dw = tdb.matmul_grouped_wgrad(x.to(TYPES[dtype]), dy.to(TYPES[dtype]), off)
    for e, (a, b) in enumerate(zip(x.split(sizes), dy.split(sizes))):
        assert torch.equal(dw[e], (a.t() @ b).to(TYPES[dtype])), e


@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("groups", GROUPS, ids=lambda g: f"{len(g[0])}e-{sum(g[0])}")
@pytest.mark.parametrize("NK", [(64, 128), (130, 400), (257, 261), (132, 1300)], ids=str)
def test_matmul_fp8_grouped_with_a_scale_for_each_row(groups, NK, out, tile):
    N, K = NK
    off, rows = _split(*groups)
    E = len(groups[0])
    a, sa = _scaled(rows, K, 1, 118)
    b, sb = _scaled(N, K, 1, 119, (E,))
    sa *= 2.0 ** -12
    ref = torch.zeros(rows, N, dtype=torch.float64)
    mag = torch.zeros_like(ref)
    av = lo.values(a, sa, 1)
    for e, (i, j) in enumerate(lo.ranges(off)):
        ref[i:j], mag[i:j] = lo.product(av[i:j], lo.values(b[e], sb[e], 1).t())
    offd = torch.tensor(off, dtype=torch.int32, device=DEV)
    ad, sad, bd, sbd = (t.to(DEV) for t in (a, sa, b, sb))
    for how, (p, r) in dict(plain=(ad, bd), aligned=(_aligned(ad), _aligned(bd))).items():
        _say("[fp8_grouped rows]", E, rows, NK, out, how)
        lo.check(tdb.matmul_fp8_grouped(p, sad, r, sbd, offd, out_dtype=TYPES[out]), ref, mag, K,
                 how)


# ------------------------------------------------------------------------------ ends of ranges
@pytest.mark.parametrize("b_block", [1, 128])
def test_scales_at_the_ends_of_their_range(b_block, tile):
    """Scales whose product is 0, subnormal, or near the largest number: whole numbers, so that
    each result is exact wherever float32 holds it (down to 2^-149)."""
    K, N = 256, 3 * b_block
    g = _gen(120)
    a = torch.randint(-3, 4, (5, K), generator=g).float()
    b = torch.randint(-3, 4, (N, K), generator=g).float()
    sa = torch.tensor([2.0 ** -126, 2.0 ** -100, 0.0, 1.0, 2.0 ** 100])[:, None].expand(5, 2)
    sb = torch.tensor([2.0 ** -23, 1.0, 2.0 ** 15])[:, None].expand(3, 2)
    ref = lo.values(a.to(lo.F8), sa, 1) @ lo.values(b.to(lo.F8), sb, b_block).t()
    assert (ref == 0).sum() < ref.numel() / 2 and ref.abs().max() < 2.0 ** 127
    c = tdb.matmul_fp8(*(t.contiguous().to(DEV) for t in (a.to(lo.F8), sa, b.to(lo.F8), sb)),
                       out_dtype=torch.float32)
    assert torch.equal(c.cpu().double(), ref)


@pytest.mark.parametrize("dtype", TYPES)
def test_no_experts_and_no_rows(dtype, tile):
    """Without experts every row is no expert's; without rows every expert's gradient is zeros."""
    dt = TYPES[dtype]
    x = torch.full((70, 96), NAN, dtype=dt, device=DEV)
    for at in (0, 30, 70):
        none = torch.tensor([at], dtype=torch.int32, device=DEV)
        y = tdb.matmul_grouped(x, torch.empty(0, 96, 40, dtype=dt, device=DEV), none)
        assert y.shape == (70, 40) and not y.any()
        assert tdb.matmul_grouped_wgrad(x, x, none).shape == (0, 96, 96)
    q, s = x.to(lo.F8), torch.full((70, 1), NAN, device=DEV)
    b, sb = torch.empty(0, 40, 96, device=DEV).to(lo.F8), torch.empty(0, 1, 1, device=DEV)
    c = tdb.matmul_fp8_grouped(q, s, b, sb, none, out_dtype=dt)
    assert c.shape == (70, 40) and not c.any()
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    w = torch.full((3, 96, 40), NAN, dtype=dt, device=DEV).requires_grad_()
    e = x[:0].clone().requires_grad_()
    y = tdb.linear_grouped(e, w, off)
    assert y.shape == (0, 40)
    dx, dw = torch.autograd.grad(y, (e, w), torch.ones_like(y))
    assert dx.shape == (0, 96) and dw.shape == w.shape and not dw.any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tw", [False, True])
def test_expert_sums_hold_32_bits(dtype, tw, tile):
    """What large products leave when they cancel, along each contraction of a grouped step (an
    expert without rows in between); exact in every type."""
    dt, off = TYPES[dtype], [0, 300, 300, 340]
    a, b, ref = _cancelling(340, 130, 1100, 121)   # rows, one side, the contraction
    offd = torch.tensor(off, dtype=torch.int32, device=DEV)
    for side, call in (("y", tw), ("dx", not tw)):  # dx is the product with the other transposition
        w = (b if call else b.t().contiguous()).expand(3, *(b.shape if call else b.t().shape))
        w = w.to(dt).to(DEV).contiguous()
        if side == "y":
            got = tdb.matmul_grouped(a.to(dt).to(DEV), w, offd, transpose_w=call)
        else:
            x = torch.zeros(340, 130, dtype=dt, device=DEV).requires_grad_()
            y = tdb.linear_grouped(x, w, offd, transpose_w=not call)
            (got,) = torch.autograd.grad(y, x, a.to(dt).to(DEV))
        _say("[expert sums]", dtype, tw, side)
        assert torch.equal(got.cpu().double(), ref), side
    p, q, ref = _cancelling(260, 90, 1500, 122)    # dw: the rows are the contraction
    rows = torch.cat([p.t(), p.t()[:7]]).contiguous(), torch.cat([q.t(), q.t()[:7]]).contiguous()
    offd = torch.tensor([0, 0, 1500, 1507], dtype=torch.int32, device=DEV)
    dw = tdb.matmul_grouped_wgrad(*(t.to(dt).to(DEV) for t in rows), offd).cpu().double()
    assert not dw[0].any() and torch.equal(dw[1], ref)
    if not tw:
        return
    lin = rows[1].to(dt).to(DEV), torch.zeros(3, 260, 90, dtype=dt, device=DEV).requires_grad_()
    y = tdb.linear_grouped(*lin, offd, transpose_w=True)
    (dw,) = torch.autograd.grad(y, lin[1], rows[0].to(dt).to(DEV))
    assert torch.equal(dw[1].cpu().double(), ref)


@pytest.mark.parametrize("dtype", TYPES)
def test_expert_sums_are_off_by_little_in_the_mean(dtype, tile):
    """As for 8-bit values: 8 * 2^-23 of the sum of magnitudes in the mean square, and the result's
    rounding, half a step at most of each."""
    K, N, off = 4096, 96, [0, 50, 64]
    g = _gen(123)
    x, w = _randn(g, 64, K).to(TYPES[dtype]), _randn(g, 2, K, N).to(TYPES[dtype])
    got = tdb.matmul_grouped(x.to(DEV), w.to(DEV), torch.tensor(off, dtype=torch.int32, device=DEV))
    ref, mag = zip(*(lo.product(x[i:j].double(), w[e].double())
                     for e, (i, j) in enumerate(lo.ranges(off))))
    ref, mag = torch.cat(ref), torch.cat(mag)
    half = torch.finfo(got.dtype).eps / 2
    err = ((got.cpu().double() - ref).abs() - half * ref.abs()).clamp_min(0)
    assert err.square().mean().sqrt() <= 8 * 2.0 ** -23 * mag.square().mean().sqrt()
