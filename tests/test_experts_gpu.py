"""The operators around the experts' products on the GPU, against plain 64-bit forms
(experts_oracle.py): sizes and masks where they can go wrong, gradients against formulas and against
differences, views, streams, captured graphs, and all of them together."""
import math
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import tiled_double_buffered_amd as tdb  # noqa: E402
sys.path.insert(0, os.path.dirname(__file__))
import experts_oracle as xo  # noqa: E402
import lowp_oracle as lo  # noqa: E402

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

DEV = torch.device("cuda:0")
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def _gen(seed):
    return torch.Generator(device="cpu").manual_seed(seed)


def _randn(g, *shape, scale=1.0, dtype=torch.float32):
    return (scale * torch.randn(*shape, generator=g)).to(dtype).to(DEV)


# ---------------------------------------------------------------------------------- router
def _logits(T, E, dtype, seed, holes=0.0):
    g = _gen(seed)
    x = 2.0 * torch.randn(T, E, generator=g)
    if holes:
        x[torch.rand(T, E, generator=g) < holes] = -math.inf
        x[::7] = -math.inf
    return x.to(dtype).to(DEV)


def _check_step(x, k, valid, norm, seed=3):
    """One training step of the router against the definition."""
    x = x.detach().requires_grad_()
    gates, experts, counts, loss = tdb.route_experts(x, k, valid=valid, renormalize=norm)
    assert experts.dtype == torch.int32 and counts.dtype == torch.int32
    r = xo.route(x, k, valid, norm)
    xo.check_route(r, gates, experts, counts, loss)
    g = _gen(seed)
    dgates, dloss = _randn(g, x.shape[0], k), torch.tensor(0.7, device=DEV)
    for dg, dl in ((dgates, dloss), (dgates, None), (None, dloss)):
        outs = [o for o, d in ((gates, dg), (loss, dl)) if d is not None]
        dx, = torch.autograd.grad(outs, x, [d for d in (dg, dl) if d is not None], retain_graph=True)
        assert dx.dtype == x.dtype
        ref, slack = xo.route_grad(r, dg, dl)
        xo.close(dx, ref, slack, "dx")
    with torch.no_grad():  # the same without a gradient
        for a, b in zip((gates, experts, counts, loss), tdb.route_experts(x, k, valid, norm)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("size", [(1, 1, 1), (1, 2, 2), (5, 16, 16), (3, 17, 3), (16, 64, 4),
                                  (17, 65, 8), (33, 60, 5), (200, 256, 8), (130, 257, 2),
                                  (7, 1000, 16), (20, 1024, 6), (2049, 8, 2)], ids=str)
def test_route(size, norm, dtype):
    T, E, k = size
    valid = None if T < 3 else (torch.rand(T, generator=_gen(T)) < 0.8).to(DEV)
    _check_step(_logits(T, E, dtype, 10 * T + E), k, valid, norm)


@pytest.mark.parametrize("norm", [False, True])
def test_route_many_rows_for_each_workgroup(norm):
    """More rows than all workgroups take at once, so that each goes round several times."""
    _check_step(_logits(40000, 12, torch.bfloat16, 5), 3, None, norm)


@pytest.mark.parametrize("T, E, k", [(70000, 12, 2), (17000, 300, 3)])
def test_route_gradient_of_more_rows_than_its_workgroups(T, E, k):
    """More rows than the gradient's workgroups take at once (65536 of up to 256 experts, 16384 of
    more), so that each goes round twice."""
    _check_step(_logits(T, E, torch.float32, 6), k, (torch.arange(T) % 9 != 4).to(DEV), k == 3)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("size", [(29, 6, 6), (50, 40, 8), (30, 300, 16)], ids=str)
def test_route_masked_experts(size, norm, dtype):
    """Logits of -Inf: never taken, rows with fewer than k left, rows with none."""
    T, E, k = size
    x = _logits(T, E, dtype, 7, holes=0.9)
    _check_step(x, k, None, norm)
    _check_step(x, k, (torch.arange(T) % 3 != 0).to(DEV), norm)


def test_route_masks_of_the_lowest_value():
    """The type's lowest value is a logit like another: its probability is 0, and it is taken
    where nothing better is left."""
    for dtype in TYPES:
        x = _logits(9, 20, dtype, 8)
        x[:, 3:] = torch.finfo(dtype).min
        _check_step(x, 5, None, False)
        _check_step(x, 5, None, True)
        _, experts, _, _ = tdb.route_experts(x, 5)
        assert torch.equal(experts[:, 3:].cpu(), torch.tensor([[3, 4]], dtype=torch.int32).expand(9, 2))


def test_route_nothing_counts():
    for x, valid in ((torch.full((5, 8), -math.inf, device=DEV), None),
                     (torch.zeros(5, 8, device=DEV), torch.zeros(5, dtype=torch.bool, device=DEV)),
                     (torch.zeros(0, 8, device=DEV), None)):
        x.requires_grad_()
        gates, experts, counts, loss = tdb.route_experts(x, 2, valid=valid, renormalize=True)
        assert (gates == 0).all() and (experts == -1).all() and (counts == 0).all() and loss == 0
        dx, = torch.autograd.grad((gates, loss), x, (torch.ones_like(gates), torch.ones_like(loss)))
        assert dx.shape == x.shape and (dx == 0).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_route_ties_go_to_the_lowest_index(dtype):
    x = torch.randint(0, 3, (100, 90), generator=_gen(1)).to(dtype).to(DEV)
    x[0] = 0.0
    x[1, ::2] = -0.0  # equal to 0
    x[1, 1::2] = 0.0
    _, experts, _, _ = tdb.route_experts(x, 16)
    ref = torch.sort(x.float().cpu(), dim=1, descending=True, stable=True).indices[:, :16]
    assert torch.equal(experts.cpu().long(), ref)


@pytest.mark.parametrize("norm", [False, True])
def test_route_nan_and_inf_stay_in_their_rows(norm):
    x = _logits(12, 40, torch.float32, 2)
    x[3, 7], x[5, 1], x[5, 30] = math.nan, math.inf, -math.inf
    x[8] = math.nan
    x.requires_grad_()
    gates, experts, counts, loss = tdb.route_experts(x, 4, renormalize=norm)
    r = xo.route(x, 4, None, norm)
    assert torch.equal(experts.cpu().long(), r["experts"]) and torch.equal(counts.cpu().long(), r["counts"])
    bad = torch.zeros(12, dtype=torch.bool)
    bad[[3, 5, 8]] = True
    assert torch.isnan(gates.cpu()[bad]).all() and not torch.isnan(gates.cpu()[~bad]).any()
    assert torch.isnan(loss)
    dx, = torch.autograd.grad(gates, x, torch.ones_like(gates))
    assert not torch.isnan(dx.cpu()[~bad]).any() and torch.isnan(dx.cpu()[bad]).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_route_views(dtype):
    """Rows at odd strides and starts, a valid mask with a stride, a transposed matrix."""
    big = _logits(60, 91, dtype, 4)
    _check_step(big[1:, 3:70], 4, (torch.arange(118, device=DEV) % 5 != 0)[::2], True)
    _check_step(big.t()[:40], 4, None, False)


def test_route_gradient_against_differences():
    """The step in FP32 against central differences of the definition in 64 bits: quadratic terms
    of h = 2^-10 are 2^-20 of a function whose third derivatives are below 8."""
    x = _logits(6, 10, torch.float32, 9).requires_grad_()
    w = _randn(_gen(2), 6, 3)
    for norm in (False, True):
        gates, experts, counts, loss = tdb.route_experts(x, 3, renormalize=norm)
        dx, = torch.autograd.grad((gates, loss), x, (w, torch.tensor(1.5, device=DEV)))
        h, base = 2.0 ** -10, x.detach().double().cpu()

        def value(z):
            p = torch.softmax(z, 1)
            g = p.gather(1, experts.cpu().long())
            if norm:
                g = g / g.sum(1, keepdim=True)
            f = counts.cpu().double() / counts.cpu().sum()
            return (g * w.double().cpu()).sum() + 1.5 * 10 * (f * p.mean(0)).sum()
        for t, e in ((0, 0), (1, 9), (2, 4), (5, 7), (3, int(experts[3, 0]))):
            d = torch.zeros_like(base)
            d[t, e] = h
            diff = (value(base + d) - value(base - d)) / (2 * h)
            assert abs(float(dx[t, e]) - float(diff)) <= 8 * h * h / 6 + 1e-5 * (1 + abs(float(diff)))


def test_route_only_once_differentiable_and_constants():
    x = _logits(4, 8, torch.float32, 1).requires_grad_()
    gates, experts, counts, loss = tdb.route_experts(x, 2)
    assert not experts.requires_grad and not counts.requires_grad and gates.requires_grad
    dx, = torch.autograd.grad(loss, x, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(dx.sum(), x)


def test_route_bounds_on_the_gpu():
    x = torch.zeros(4, 1025, device=DEV)
    for call in (lambda: tdb.route_experts(x, 2), lambda: tdb.route_experts(x[:, :0], 1),
                 lambda: tdb.route_experts(x[:, :8], 9), lambda: tdb.route_experts(x[:, :8], 0),
                 lambda: tdb.route_experts(x[:, :64], 17),
                 lambda: tdb.route_experts(x[:, :8], 2, valid=torch.ones(4, dtype=torch.bool))):
        with pytest.raises(ValueError):
            call()


# --------------------------------------------------------------------------------- grouping
def _group_ref(ids, count):
    e = ids.cpu().numpy().reshape(-1).astype(np.int64)
    e = np.where((e < 0) | (e >= count), count, e)
    order = np.argsort(e, kind="stable")
    place = np.empty_like(order)
    place[order] = np.arange(len(e))
    return order, place, np.concatenate([[0], np.cumsum(np.bincount(e, minlength=count + 1))])[:count + 1]


def _check_group(ids, count):
    order, place, offsets = tdb.group_rows(ids, count)
    assert order.dtype == place.dtype == torch.int64 and offsets.dtype == torch.int32
    assert place.shape == ids.shape
    ref = _group_ref(ids, count)
    for name, got, want in zip(("order", "place", "offsets"), (order, place.reshape(-1), offsets), ref):
        assert np.array_equal(got.cpu().numpy(), want), name


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("count", [0, 1, 2, 64, 255, 1024, 1025, 4096])
@pytest.mark.parametrize("n", [0, 1, 63, 64, 65, 512, 1000, 2048, 2049, 8192, 8193, 40001])
def test_group_rows(n, count, dtype):
    ids = torch.randint(-1, count + 2, (n,), generator=_gen(n + count), dtype=dtype).to(DEV)
    _check_group(ids, count)


def test_group_rows_many_and_uneven():
    g = _gen(4)
    n = 700001
    e = (torch.rand(n, generator=g) ** 4 * 70).to(torch.int32)
    _check_group(e.to(DEV), 64)
    _check_group(torch.full((20000,), 3, dtype=torch.int32, device=DEV), 8)  # all the same
    _check_group(torch.arange(20000, 0, -1, dtype=torch.int32, device=DEV), 4096)


def test_group_rows_shapes_and_far_numbers():
    ids = torch.randint(0, 9, (300, 6), generator=_gen(2)).to(DEV)
    _check_group(ids, 9)
    _check_group(ids[:, :2], 9)  # a view
    _check_group(ids.t(), 9)
    far = ids.clone()
    far[::3] += 1 << 40          # past 32 bits: of no expert
    far[1::3] -= 1 << 33
    _check_group(far, 9)
    _check_group(torch.tensor(4, device=DEV), 9)  # no axis: one element


# --------------------------------------------------------------------------------- adapters
def _groups(sizes, T, seed):
    """(order, offsets): places of the adapters, rows shuffled, rows of no adapter last."""
    ids = torch.full((T,), -1, dtype=torch.int64)
    rows = torch.randperm(T, generator=_gen(seed))
    at = 0
    for e, n in enumerate(sizes):
        ids[rows[at:at + n]] = e
        at += n
    order, _, offsets = tdb.group_rows(ids.to(DEV), len(sizes))
    return order, offsets


def _adapter_inputs(T, E, r, K, N, dtype, seed):
    g = _gen(seed)
    return (_randn(g, T, N, dtype=dtype), _randn(g, T, K, dtype=dtype),
            _randn(g, E, r, K, scale=max(K, 1) ** -0.5, dtype=dtype),
            _randn(g, E, r, N, scale=r ** -0.5, dtype=dtype), _randn(g, T, N, dtype=dtype),
            torch.rand(E, generator=g).to(DEV) + 0.5)


def _check_adapters(y, x, a, b, order, offsets, scale, dout):
    leaves = [t.detach().requires_grad_() for t in (y, x, a, b)]
    out = tdb.add_adapters(*leaves, order, offsets, scale=scale)
    grads = torch.autograd.grad(out, leaves, dout)
    assert torch.equal(grads[0], dout)
    got = dict(zip(("out", "dx", "da", "db"), (out, *grads[1:])))
    for name, ref, slack in xo.adapters(y, x, a, b, order, offsets, scale, dout):
        assert got[name].dtype == x.dtype
        xo.close(got[name], ref, slack, name)
    with torch.no_grad():
        assert torch.equal(tdb.add_adapters(y, x, a, b, order, offsets, scale=scale), out)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("r", [1, 3, 8, 16, 17, 32, 50, 64, 65, 128])
def test_adapters_ranks(r, dtype):
    sizes, T, K, N = (5, 0, 17, 40, 1), 70, 328, 264
    y, x, a, b, d, s = _adapter_inputs(T, 5, r, K, N, dtype, r)
    _check_adapters(y, x, a, b, *_groups(sizes, T, r), s, d)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("size", [(1, (1,), 1, 1), (1, (0, 1), 64, 128), (2, (1, 1), 130, 7),
                                  (16, (16,), 512, 512), (33, (0, 0, 33, 0), 65, 129),
                                  (40, (3,) * 13, 1000, 515), (300, (280, 4), 4096, 640),
                                  (500, (500,), 96, 2048)], ids=lambda s: f"{s[0]}x{s[2]}x{s[3]}")
def test_adapters_sizes(size, dtype):
    T, sizes, K, N = size
    y, x, a, b, d, s = _adapter_inputs(T, len(sizes), 12, K, N, dtype, T + K)
    _check_adapters(y, x, a, b, *_groups(sizes, T, K), s if T % 2 else None, d)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("r", [8, 30, 64, 120])
@pytest.mark.parametrize("T, sizes, K, N", [(8300, (3000, 0, 5200), 72, 136), (3500, (900, 1500, 1000), 264, 80),
                                            (1100, (1000, 40), 520, 1032), (2500, (900, 0, 1500), 1100, 72)],
                         ids=str)
def test_adapters_many_rows(T, sizes, K, N, r, dtype):
    """Every way of sharing the rows out: tiles of 64 places whose waves share a step, and partial sums
    that are joined."""
    y, x, a, b, d, s = _adapter_inputs(T, len(sizes), r, K, N, dtype, T + r)
    _check_adapters(y, x, a, b, *_groups(sizes, T, r), s, d)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [8, 9, 63, 64, 65, 127, 128, 511, 1023])
def test_adapters_every_end_of_the_wide_axis(K, dtype):
    """The steps' ends, in both directions (K in, K out)."""
    for T, sizes in ((20, (11, 9)), (8200, (4100, 4000))):
        y, x, a, b, d, s = _adapter_inputs(T, 2, 20, K, K, dtype, K)
        _check_adapters(y, x, a, b, *_groups(sizes, T, K), s, d)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("r, K", [(r, K) for r in (9, 20) for K in (8, 9, 63, 64, 65, 127, 128, 511, 1023)] +
                         [(r, K) for r in (50, 100) for K in (9, 65, 511)])
def test_adapters_every_end_of_the_wide_axis_in_tiles_of_64(K, r, dtype):
    """So many rows that a workgroup of the contraction takes 64 of them, whatever the columns."""
    T = 10050 if r <= 64 else 5050
    y, x, a, b, d, s = _adapter_inputs(T, 2, r, K, 40, dtype, K)
    _check_adapters(y, x, a, b, *_groups((T // 2 + 17, T // 2 - 60), T, K), s, d)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T, sizes, r, K", [(1030, (400, 0, 600), 30, 2100), (1030, (1, 1000, 2), 50, 1030),
                                            (1030, (65, 63, 64, 800), 100, 513), (5003, (4000, 900), 7, 2050),
                                            (1200, (18,) * 64, 64, 1090)], ids=str)
def test_adapters_few_rows_in_tiles_of_64(T, sizes, r, K, dtype):
    """Columns and ranks whose bytes ask for tiles of 64 with few rows, splits of the columns among them."""
    y, x, a, b, d, s = _adapter_inputs(T, len(sizes), r, K, 40, dtype, r)
    _check_adapters(y, x, a, b, *_groups(sizes, T, r), s, d)


@pytest.mark.parametrize("dtype", TYPES)
def test_adapters_of_a_plan_that_begins_past_the_first_place(dtype):
    """Places before the first adapter's, and x that is y too."""
    T, r, K = 300, 9, 72
    y, x, a, b, d, s = _adapter_inputs(T, 3, r, K, K, dtype, 1)
    order = torch.randperm(T, generator=_gen(2)).to(DEV)
    offsets = torch.tensor([11, 60, 60, 250], dtype=torch.int32, device=DEV)
    _check_adapters(y, x, a, b, order, offsets, s, d)
    assert torch.equal(tdb.add_adapters(y, y, a, b, order, offsets), tdb.add_adapters(y, y.clone(), a, b, order, offsets))


def test_adapters_of_many_requests():
    """More groups than a wave looks at at once, most of them empty."""
    sizes = [0] * 400
    for i in (0, 63, 64, 65, 130, 255, 399):
        sizes[i] = 1 + i % 40
    y, x, a, b, d, s = _adapter_inputs(250, 400, 7, 40, 56, torch.bfloat16, 3)
    _check_adapters(y, x, a, b, *_groups(sizes, 250, 3), s, d)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_adapters_rows_split_for_the_gradient(dtype):
    """One adapter with many rows: its gradients' rows are split over workgroups."""
    assert tdb.gemm_adapters_grad_workspace(3001, 136, 200, 24, 1, 0) > 0
    y, x, a, b, d, s = _adapter_inputs(3001, 1, 24, 136, 200, dtype, 1)
    _check_adapters(y, x, a, b, *_groups((2900,), 3001, 3), s, d)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("r", [9, 40, 70])
def test_adapters_with_many_rows_among_those_with_few(r, dtype):
    """Gradients that several workgroups add up among such that one has whole, more adapters than a
    wave looks at at once: the sums lie one after another, whichever adapters they are of."""
    sizes = [(0, 1, 3)[i % 3] for i in range(150)]
    for i, n in ((0, 300), (1, 129), (5, 128), (62, 700), (63, 257), (64, 1000), (65, 2), (100, 385),
                 (127, 130), (128, 256), (149, 2000)):
        sizes[i] = n
    T, K, N = sum(sizes) + 7, 136, 200
    y, x, a, b, d, s = _adapter_inputs(T, 150, r, K, N, dtype, r)
    _check_adapters(y, x, a, b, *_groups(sizes, T, r), s, d)


@pytest.mark.parametrize("dtype", TYPES)
def test_adapters_views(dtype):
    """Odd strides and starts, broadcast adapters, leading axes, transposed operands."""
    g = _gen(6)
    T, E, r, K, N = 45, 4, 6, 70, 51
    y, x = _randn(g, T + 2, N + 5, dtype=dtype)[1:-1, 3:-2], _randn(g, T, K + 9, dtype=dtype)[:, 1:K + 1]
    a = _randn(g, E, r + 1, K + 3, scale=0.1, dtype=dtype)[:, 1:, 2:K + 2]
    b = _randn(g, E, r, N + 1, dtype=dtype)[:, :, 1:]
    d = _randn(g, T, N + 3, dtype=dtype)[:, 2:-1]
    order, offsets = _groups((10, 0, 20, 9), T, 1)
    _check_adapters(y, x, a, b, order, offsets, None, d)
    _check_adapters(y, x, a[:1].expand(E, r, K), b, order, offsets, None, d)
    _check_adapters(y.t().contiguous().t(), x.t().contiguous().t(), a.transpose(1, 2).contiguous().transpose(1, 2),
                    b.transpose(1, 2).contiguous().transpose(1, 2), order, offsets, None, d.t().contiguous().t())
    lead = tdb.add_adapters(y.reshape(3, 15, N), x.reshape(3, 15, K), a, b, order, offsets)
    assert lead.shape == (3, 15, N)
    assert torch.equal(lead.view(T, N), tdb.add_adapters(y, x, a, b, order, offsets))


def test_adapters_shared_by_all_experts_add_their_gradients():
    """One adapter broadcast to all groups: its gradient is the sum of theirs."""
    g = _gen(8)
    y, x, a, b, d, _ = _adapter_inputs(50, 3, 5, 40, 30, torch.float32, 8)
    order, offsets = _groups((20, 10, 15), 50, 2)
    one = a[0].detach().requires_grad_()
    out = tdb.add_adapters(y, x, one.expand(3, 5, 40), b, order, offsets)
    got, = torch.autograd.grad(out, one, d)
    each = dict((n, (v, s)) for n, v, s in xo.adapters(y, x, one.detach().expand(3, 5, 40), b, order, offsets, None, d))
    ref, slack = each["da"]
    xo.close(got, ref.sum(0), slack.sum(0) + ref.abs().sum(0) * 4 * xo.U, "shared")


@pytest.mark.parametrize("dtype", TYPES)
def test_adapters_rows_of_none_keep_y(dtype):
    """Bit for bit, zeros of either sign, Inf and the smallest numbers among them; every kernel, rows of
    none before the first adapter's and behind the last one's.  Their dx is 0 (not -0)."""
    ends = torch.tensor([0.0, -0.0, math.inf, -math.inf, torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal,
                         -torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps])
    bits = torch.int32 if dtype == torch.float32 else torch.int16
    for T, r, N in ((40, 5, 72), (40, 40, 72), (40, 5, 7), (5000, 12, 264)):
        y, x, a, b, d, s = _adapter_inputs(T, 2, r, 24, N, dtype, r)
        y = ends.repeat(T * N // 7 + 1)[:T * N].view(T, N).to(dtype).to(DEV)
        order = torch.randperm(T, generator=_gen(T)).to(DEV)
        offsets = torch.tensor([7, T // 2, T - 9], dtype=torch.int32, device=DEV)
        x.requires_grad_()
        out = tdb.add_adapters(y, x, a, b, order, offsets)
        none = torch.cat([order[:7], order[T - 9:]])
        assert torch.equal(out[none].view(bits), y[none].view(bits))
        dx, = torch.autograd.grad(out, x, d)
        assert (dx[none].view(bits) == 0).all()


def test_adapters_missing_gradients():
    y, x, a, b, d, s = _adapter_inputs(20, 2, 4, 24, 40, torch.float32, 3)
    order, offsets = _groups((9, 8), 20, 4)
    leaves = [t.detach().requires_grad_() for t in (y, x, a, b)]
    full = torch.autograd.grad(tdb.add_adapters(*leaves, order, offsets, scale=s), leaves, d)
    for i in range(4):
        some = [t.detach().requires_grad_(j == i) for j, t in enumerate((y, x, a, b))]
        got, = torch.autograd.grad(tdb.add_adapters(*some, order, offsets, scale=s), some[i], d)
        assert torch.equal(got, full[i])


def test_adapters_empty():
    for dtype in TYPES:
        for T, E, K, N in ((0, 2, 8, 8), (5, 0, 8, 8), (5, 2, 0, 8), (5, 2, 8, 0)):
            y, x, a, b, d, _ = _adapter_inputs(T, E, 3, K, N, dtype, 1)
            order, offsets = _groups((min(T, 3), 0)[:E], T, 1)
            _check_adapters(y, x, a, b, order, offsets, None, d)


@pytest.mark.parametrize("dtype", TYPES)
def test_adapters_inf_and_nan_stay_in_their_rows(dtype):
    y, x, a, b, d, s = _adapter_inputs(40, 3, 6, 100, 90, dtype, 5)
    order, offsets = _groups((15, 10, 10), 40, 6)
    clean = tdb.add_adapters(y, x, a, b, order, offsets)
    rows = order[offsets[1]:offsets[2]]
    bad = x.clone()
    bad[rows[2]], bad[order[-1]] = math.nan, math.inf  # the last row has no adapter
    got = tdb.add_adapters(y, bad, a, b, order, offsets)
    keep = torch.ones(40, dtype=torch.bool, device=DEV)
    keep[rows[2]] = False
    assert torch.equal(got[keep], clean[keep]) and torch.isnan(got[rows[2]]).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_adapters_inf_in_a_row(dtype):
    """Inf in x: the row's results are what the formula gives, Inf or NaN; the others do not change.
    Inf in an adapter: its rows alone are not finite."""
    y, x, a, b, d, s = _adapter_inputs(24, 2, 5, 72, 40, dtype, 9)
    order, offsets = _groups((12, 12), 24, 3)
    a = a.abs()
    b = torch.where(b.abs() < 0.1, torch.ones_like(b), b)
    clean = tdb.add_adapters(y, x, a, b, order, offsets)
    bad = x.clone()
    bad[4, 3], bad[9, 70] = math.inf, -math.inf
    got = tdb.add_adapters(y, bad, a, b, order, offsets)
    _, ref, slack = xo.adapters(y, bad, a, b, order, offsets, None)[0]
    xo.close(got, ref, torch.nan_to_num(slack, posinf=0.0), "inf in x")
    keep = torch.ones(24, dtype=torch.bool, device=DEV)
    keep[[4, 9]] = False
    assert torch.equal(got[keep], clean[keep]) and not torch.isfinite(got[~keep]).any()
    worse = b.clone()
    worse[1, 2, 7] = math.inf
    got = tdb.add_adapters(y, x, a, worse, order, offsets)
    rows = order[offsets[1]:offsets[2]]
    assert not torch.isfinite(got[rows, 7]).any()
    got[rows, 7] = clean[rows, 7]
    assert torch.equal(got, clean)


def test_adapters_large_and_small_numbers_in_fp16():
    """x A^T beyond fp16's range and below its smallest step, with results inside it."""
    g = _gen(4)
    for up, down in ((200.0, 2.0 ** -14), (2.0 ** -9, 100.0)):
        y = torch.zeros(33, 72, dtype=torch.float16, device=DEV)
        x = _randn(g, 33, 512, scale=up, dtype=torch.float16)
        a = _randn(g, 2, 9, 512, scale=50.0 if up > 1 else 2.0 ** -9, dtype=torch.float16)
        b = _randn(g, 2, 9, 72, scale=down, dtype=torch.float16)
        d = _randn(g, 33, 72, scale=2.0 ** -12 if up > 1 else 1.0, dtype=torch.float16)
        for name, ref, slack in xo.adapters(y, x, a, b, *(p := _groups((20, 13), 33, 1)), None):
            xo.close(tdb.add_adapters(y, x, a, b, *p), ref, slack, name)


@pytest.mark.parametrize("exponent", [-100, -112, -124, -130])
def test_adapters_small_contractions_in_bf16(exponent):
    """x A^T near FP32's smallest normal number and below it, with results of ordinary size: nothing
    is lost but the bits below bf16's smallest step, 2^-133, of each of the contraction's numbers."""
    g = _gen(2)
    T, r, K, N = 40, 6, 64, 72
    half = exponent // 2
    y = torch.zeros(T, N, dtype=torch.bfloat16, device=DEV)
    x = _randn(g, T, K, scale=2.0 ** half, dtype=torch.bfloat16)
    a = _randn(g, 1, r, K, scale=2.0 ** (exponent - half), dtype=torch.bfloat16)
    b = _randn(g, 1, r, N, scale=2.0 ** 100, dtype=torch.bfloat16)
    order, offsets = _groups((T,), T, 1)
    got = tdb.add_adapters(y, x, a, b, order, offsets)
    (_, ref, slack), = xo.adapters(y, x, a, b, order, offsets, None)
    # (of FP32's own steps, 2^-149: one for each product of the contraction)
    lost = (2.0 ** -133 + K * 2.0 ** -149) * b[0].double().cpu().abs().sum(0)
    xo.close(got, ref, slack + lost, "out")


def test_adapters_rows_behind_are_left():
    """Through the C ABI: columns past N and places of no adapter keep what they hold."""
    T, E, r, K, N = 20, 2, 5, 48, 40
    y, x, a, b, d, s = _adapter_inputs(T, E, r, K, N, torch.bfloat16, 2)
    order, offsets = _groups((7, 6), T, 1)
    stream = torch.cuda.current_stream().cuda_stream
    u = torch.full((2, T, 16), 7.0, device=DEV)
    rc = tdb.gemm_adapters_down(T, K, r, E, order.data_ptr(), offsets.data_ptr(), x.data_ptr(), K,
                                a.data_ptr(), K, r * K, s.data_ptr(), u.data_ptr(), 2, 0, 0, stream)
    assert rc == tdb.OK and (u[:, 13:] == 7).all() and (u[:, :13] != 7).all()
    assert (u[:, :13, r:] == 0).all()
    out = torch.full((T + 1, N + 3), 7.0, dtype=torch.bfloat16, device=DEV)
    rc = tdb.gemm_adapters_up(T, N, r, E, order.data_ptr(), offsets.data_ptr(), u.data_ptr(), 2,
                              b.data_ptr(), N, r * N, y.data_ptr(), N, out.data_ptr(), N + 3, 0, stream)
    assert rc == tdb.OK and (out[T] == 7).all() and (out[:, N:] == 7).all()
    for name, ref, slack in xo.adapters(y, x, a, b, order, offsets, s):
        xo.close(out[:T, :N], ref, slack, name)


def test_adapters_wrong_plans_stay_in_bounds():
    """Rows and offsets out of range give some values, and touch nothing else."""
    T, E, r, K, N = 30, 3, 4, 64, 64
    y, x, a, b, d, s = _adapter_inputs(T, E, r, K, N, torch.float32, 2)
    order = torch.arange(T, device=DEV)
    order[3], order[7] = 1 << 40, -5
    for offsets in ([0, 10, 20, 99], [5, 3, 50, 20], [-9, -3, 10, 30]):
        o = torch.tensor(offsets, dtype=torch.int32, device=DEV)
        leaves = [t.detach().requires_grad_() for t in (y, x, a, b)]
        out = tdb.add_adapters(*leaves, order, o)
        assert out.shape == (T, N)
        torch.autograd.grad(out, leaves, d)
    torch.cuda.synchronize()


class _Guarded:
    """Buffers with 64 KiB of a pattern on both sides, which has to be there afterwards."""
    PAD = 1 << 16

    def __init__(self):
        self.all = []

    def __call__(self, *shape, dtype=torch.float32):
        n = math.prod(shape) * torch.empty((), dtype=dtype).element_size()
        raw = torch.full((2 * self.PAD + (n + 255) // 256 * 256,), 0x5A, dtype=torch.uint8, device=DEV)
        self.all.append((raw, n))
        return raw[self.PAD:self.PAD + n].view(dtype).view(shape)

    def check(self):
        torch.cuda.synchronize()
        for raw, n in self.all:
            assert (raw[:self.PAD] == 0x5A).all() and (raw[self.PAD + n:] == 0x5A).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("r", [4, 48])
@pytest.mark.parametrize("T, plans", [
    (30, ([0, 10, 20, 99], [5, 3, 50, 20], [-9, -3, 10, 30], [30, 20, 10, 0])),
    (2000, ([0, 2000, 0, 2000], [0, 5000, -1, 1 << 30], [1999, 0, 2000, 3]))], ids=["few", "many"])
def test_adapters_wrong_plans_leave_the_memory_around(T, plans, r, dtype):
    """Through the C ABI: rows and offsets that are out of range, decrease or overlap write nothing
    outside U, the results, the gradients and the workspace."""
    E, K, N = 3, 200, 136
    y, x, a, b, d, s = _adapter_inputs(T, E, r, K, N, dtype, 2)
    order = torch.arange(T, device=DEV)
    order[3], order[7], order[T - 1] = 1 << 40, -5, T
    code, stream = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}[dtype], torch.cuda.current_stream().cuda_stream
    ldu = (r + 15) // 16 * 16
    for plan in plans:
        g = _Guarded()
        o = torch.tensor(plan, dtype=torch.int32, device=DEV)
        su, sv = tdb.gemm_adapters_splits(T, K, r, E), tdb.gemm_adapters_splits(T, N, r, E)
        u, v, out, dx = g(su, T, ldu), g(sv, T, ldu), g(T, N, dtype=dtype), g(T, K, dtype=dtype)
        da, db = g(E, r, K, dtype=dtype), g(E, r, N, dtype=dtype)
        need = tdb.gemm_adapters_grad_workspace(T, K, N, r, E, code)
        assert (need > 0) == (T == 2000)
        ws = g(max(need, 8), dtype=torch.uint8)
        for w in (u, v):
            w.zero_()
        at = order.data_ptr(), o.data_ptr()
        for rc in (
                tdb.gemm_adapters_down(T, K, r, E, *at, x.data_ptr(), K, a.data_ptr(), K, r * K,
                                       s.data_ptr(), u.data_ptr(), su, 0, code, stream),
                tdb.gemm_adapters_down(T, N, r, E, *at, d.data_ptr(), N, b.data_ptr(), N, r * N,
                                       s.data_ptr(), v.data_ptr(), sv, 1, code, stream),
                tdb.gemm_adapters_up(T, N, r, E, *at, u.data_ptr(), su, b.data_ptr(), N, r * N,
                                     y.data_ptr(), N, out.data_ptr(), N, code, stream),
                tdb.gemm_adapters_up(T, K, r, E, *at, v.data_ptr(), 1, a.data_ptr(), K, r * K, None, 0,
                                     dx.data_ptr(), K, code, stream),
                tdb.gemm_adapters_grad(T, r, E, *at, K, v.data_ptr(), 1, x.data_ptr(), K, da.data_ptr(), K,
                                       r * K, N, u.data_ptr(), su, d.data_ptr(), N, db.data_ptr(), N, r * N,
                                       ws.data_ptr(), need, code, stream)):
            assert rc == tdb.OK
        g.check()


def test_adapter_gradients_against_differences():
    """Central differences in 64 bits of the definition, which is linear in each operand: exact but
    for rounding."""
    y, x, a, b, d, s = _adapter_inputs(12, 2, 3, 10, 14, torch.float32, 7)
    order, offsets = _groups((6, 4), 12, 2)
    leaves = [t.detach().requires_grad_() for t in (y, x, a, b)]
    grads = torch.autograd.grad(tdb.add_adapters(*leaves, order, offsets, scale=s), leaves, d)

    def value(ops):
        return float((xo.adapters(*ops, order, offsets, s)[0][1] * d.double().cpu()).sum())
    base = [t.double().cpu() for t in (y, x, a, b)]
    for i in range(4):
        for at in (0, 7, base[i].numel() - 1):
            ops = [t.clone() for t in base], [t.clone() for t in base]
            ops[0][i].view(-1)[at] += 0.5
            ops[1][i].view(-1)[at] -= 0.5
            diff = value(ops[0]) - value(ops[1])
            got = float(grads[i].reshape(-1)[at])
            assert abs(got - diff) <= 1e-5 * (1 + abs(diff)), (i, at, got, diff)


def test_adapters_refusals_on_the_gpu():
    y, x, a, b, d, s = _adapter_inputs(8, 2, 4, 16, 16, torch.float32, 1)
    order, offsets = _groups((4, 4), 8, 1)
    for call, error in ((lambda: tdb.add_adapters(y, x, a, b, order[:7], offsets), ValueError),
                        (lambda: tdb.add_adapters(y, x, a, b, order.int(), offsets), TypeError),
                        (lambda: tdb.add_adapters(y, x, a, b, order.cpu(), offsets), ValueError),
                        (lambda: tdb.add_adapters(y, x, a, b, order, offsets[:2]), ValueError),
                        (lambda: tdb.add_adapters(y, x, a, b, order, offsets.long()), TypeError),
                        (lambda: tdb.add_adapters(y, x, a, b, order, offsets, scale=s.requires_grad_()), ValueError),
                        (lambda: tdb.add_adapters(y, x.cpu(), a, b, order, offsets), ValueError)):
        with pytest.raises(error):
            call()


# ------------------------------------------------------------------------------- gated unit
def _wide(rows, cols, dtype, seed):
    """Values of many sizes, zeros and whole blocks of zeros among them."""
    g = _gen(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp2(4 * torch.randn(rows, 1, generator=g)).clamp(2e-3, 60)
    x[torch.rand(rows, cols, generator=g) < 0.05] = 0.0
    x[rows // 2, :130] = 0.0
    return x.to(dtype).to(DEV)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("shape", [(1, 1), (1, 128), (3, 129), (16, 512), (130, 257), (5, 1000),
                                   (257, 136)], ids=str)
def test_gated(shape, keep, dtype):
    rows, N = shape
    x, dh = _wide(rows, 2 * N, dtype, rows + N).requires_grad_(), _wide(rows, N, dtype, 5)
    h = tdb.gated_silu(x, checkpoint=keep)
    dx, = torch.autograd.grad(h, x, dh)
    values = None
    if keep:
        values = torch.cat([lo.values(*_quantized(half), 1) for half in x.detach().split(N, 1)], 1)
    (rh, mh), (rx, mx) = xo.gated(x, dh, values)
    xo.close(h, rh, mh, "h")
    xo.close(dx, rx, mx, "dx")
    assert h.dtype == dx.dtype == dtype
    with torch.no_grad():
        assert torch.equal(tdb.gated_silu(x, checkpoint=keep), h)


def _quantized(x):
    """lowp_oracle's 8-bit values over their scales, and the scales."""
    v, s = lo.quantize(x, 1)
    return v.to(torch.float32), s


def test_gated_far_ends():
    """Gates whose exponential leaves FP32's range, Inf and NaN: as the definition has them."""
    g = torch.tensor([0.0, -0.0, 80.0, -80.0, 100.0, -100.0, 1e4, -1e4, 6e4, -6e4, math.inf, math.nan])
    for dtype in TYPES:
        x = torch.cat([g, torch.full_like(g, 3.0)])[None].to(dtype).to(DEV).requires_grad_()
        dh = torch.full((1, 12), 0.5, dtype=dtype, device=DEV)
        h = tdb.gated_silu(x)
        dx, = torch.autograd.grad(h, x, dh)
        (rh, mh), (rx, mx) = xo.gated(x, dh)
        xo.close(h[:, :11], rh[:, :11], mh[:, :11].nan_to_num(), "h")
        xo.close(dx[:, :10], rx[:, :10], mx[:, :10], "dx")
        assert torch.isnan(h[0, 11]) and torch.isnan(dx[0, 11])


@pytest.mark.parametrize("dtype", TYPES)
def test_gated_small_sigmoids(dtype):
    """Gates whose sigmoid is below the smallest normal number of FP32, with an up (for the forward
    pass) or a gradient (for the backward) that makes numbers of the products again: as exact as any
    other, with no allowance for small exponentials."""
    g = torch.tensor([-86.0, -87.5, -90.0, -95.0, -100.0, -104.0, -110.0, -125.0, -150.0, -170.0, -174.0])
    big = 0.9 * torch.finfo(dtype).max
    for up, grad in ((big, 0.5), (-3.0, big), (big, 2.0 ** 9), (1.0, 1.0)):
        x = torch.cat([g, torch.full_like(g, up)])[None].to(dtype).to(DEV).requires_grad_()
        dh = torch.full((1, len(g)), grad, dtype=dtype, device=DEV)
        h = tdb.gated_silu(x)
        dx, = torch.autograd.grad(h, x, dh)
        gd, ud, dd = x.detach()[0, :len(g)].double().cpu(), float(x.detach()[0, -1]), float(dh[0, 0])
        s = torch.sigmoid(gd)
        for name, got, ref in (("h", h[0], gd * s * ud),
                               ("dgate", dx[0, :len(g)], dd * ud * s * (1 + gd * torch.sigmoid(-gd))),
                               ("dup", dx[0, len(g):], dd * gd * s)):
            # (FP32 products that fall below the normal numbers on the way: a few of its smallest steps)
            xo.close(got, ref, ref.abs() * xo.U * (24 + 4 * gd.abs()) + 2.0 ** -148, f"{name} {up} {grad}")


@pytest.mark.parametrize("dtype", TYPES)
def test_gated_kept_values_at_the_ends_of_the_range(dtype):
    """The type's largest and lowest numbers in 8 bits can round to more than the type has: they
    count as its largest then, and the gradients are finite where those of x itself are."""
    most = torch.finfo(dtype).max
    g = torch.tensor([-most, most, 1.0, -2.0, -most, most, 0.0, 0.97 * most])
    u = torch.tensor([1.0, 1.0, -most, most, most, -0.5, -most, 1.0])
    # (a block of its own for each, so that every scale is its value's)
    x = torch.stack([torch.cat([a.view(1), b.view(1)]) for a, b in zip(g, u)]).to(dtype).to(DEV).requires_grad_()
    dh = torch.full((8, 1), 0.5, dtype=dtype, device=DEV)
    h = tdb.gated_silu(x, checkpoint=True)
    dx, = torch.autograd.grad(h, x, dh)
    values = torch.cat([lo.values(*_quantized(half), 1) for half in x.detach().split(1, 1)], 1).clamp(-most, most)
    (_, _), (rx, mx) = xo.gated(x, dh, values)
    xo.close(dx, rx, mx, "dx")
    plain, = torch.autograd.grad(tdb.gated_silu(x), x, dh)
    assert torch.isfinite(plain).all() and torch.isfinite(dx).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_gated_views_and_leading_axes(dtype):
    big = _wide(41, 131, dtype, 3)
    dh = _wide(40, 61, dtype, 4)[:, 1:]
    for keep in (False, True):
        x = big[1:, 5:125].detach().requires_grad_()
        h = tdb.gated_silu(x, checkpoint=keep)
        got = torch.autograd.grad(h, x, dh)[0]
        y = x.detach().clone().requires_grad_()
        ref = tdb.gated_silu(y.view(2, 20, 120), checkpoint=keep)
        assert ref.shape == (2, 20, 60) and torch.equal(ref.view(40, 60), h)
        assert torch.equal(torch.autograd.grad(ref, y, dh.reshape(2, 20, 60))[0], got)
        t = x.detach().t().contiguous().t().requires_grad_()
        assert torch.equal(tdb.gated_silu(t, checkpoint=keep), h)
    one = big[0, :130].detach().requires_grad_()
    assert tdb.gated_silu(one).shape == (65,)


def test_gated_empty():
    for shape in ((0, 8), (4, 0), (0,), (2, 0, 6)):
        for keep in (False, True):
            x = torch.zeros(shape, device=DEV, requires_grad=True)
            h = tdb.gated_silu(x, checkpoint=keep)
            assert h.shape == (*shape[:-1], shape[-1] // 2)
            assert torch.autograd.grad(h, x, torch.ones_like(h))[0].shape == shape


def test_gated_gradient_against_differences():
    """h = 2^-8 and third derivatives below 4: quadratic terms below 2^-16 of them."""
    x = _randn(_gen(1), 3, 20).requires_grad_()
    w = _randn(_gen(2), 3, 10)
    dx, = torch.autograd.grad(tdb.gated_silu(x), x, w)
    h, base = 2.0 ** -8, x.detach().double().cpu()

    def value(z):
        g, u = z[:, :10], z[:, 10:]
        return float((g / (1 + torch.exp(-g)) * u * w.double().cpu()).sum())
    for t, c in ((0, 0), (1, 9), (2, 13), (0, 19)):
        d = torch.zeros_like(base)
        d[t, c] = h
        diff = (value(base + d) - value(base - d)) / (2 * h)
        size = 1 + float(w.abs().max()) * float(x.abs().max())
        assert abs(float(dx[t, c]) - diff) <= 4 * size * h * h / 6 + 1e-5 * size


# --------------------------------------------------------------------------- 8-bit values
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("shape", [(1, 1), (3, 129), (130, 257), (257, 136)], ids=str)
def test_dequantize(shape, block, dtype):
    x = _wide(*shape, torch.float32, 7)
    q, s = tdb.quantize_fp8(x, block=(block, 128))
    got = tdb.dequantize_fp8(q, s, dtype)
    assert torch.equal(got, lo.values(q.float(), s, block).to(dtype).to(DEV))
    odd = torch.rand(s.shape, generator=_gen(1)).to(DEV) - 0.5  # any scales
    ref = lo.values(q.float(), odd, block)
    xo.close(tdb.dequantize_fp8(q, odd, dtype), ref, ref.abs() * xo.U)


@pytest.mark.parametrize("dtype", TYPES)
def test_dequantize_forms_the_product_in_float32(dtype):
    """Scales of 24 bits: the product rounded to FP32, then to the type, to the nearest each time."""
    q, _ = tdb.quantize_fp8(_wide(64, 640, torch.float32, 3))
    s = (torch.rand(64, 5, generator=_gen(4)) + 0.5).to(DEV)
    ref = (q.float() * s.repeat_interleave(128, 1)).to(dtype)
    assert torch.equal(tdb.dequantize_fp8(q, s, dtype), ref)


def test_dequantize_every_value_and_the_ends():
    q = torch.arange(256, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).view(2, 128)
    for s in (1.0, 2.0 ** -126, 256.0, 2.0 ** 100, 2.0 ** 120, 1e38):
        scale = torch.full((2, 1), s, device=DEV)
        exact = q.float().double().cpu() * float(scale[0, 0])
        for dtype in TYPES:
            most = torch.finfo(dtype).max
            xo.close(tdb.dequantize_fp8(q, scale, dtype), exact.clamp(-most, most), exact.abs().clamp(max=most) * xo.U)
    inf = tdb.dequantize_fp8(q, torch.full((2, 1), math.inf, device=DEV), torch.float32)
    assert torch.equal(torch.isinf(inf), (q.float() != 0) & ~torch.isnan(q.float()))


# --------------------------------------------------------- expert products that keep 8 bits
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tw", [False, True])
@pytest.mark.parametrize("sizes, pad, K, N", [((1,), 0, 1, 1), ((0, 5, 0, 40), 3, 130, 72),
                                              ((64, 1, 200), 0, 257, 131), ((0, 0), 4, 64, 64)],
                         ids=lambda v: str(v))
def test_kept_step(sizes, pad, K, N, tw, dtype):
    g = _gen(K)
    rows, E = sum(sizes) + pad, len(sizes)
    x = _wide(rows, K, dtype, 2).requires_grad_()
    w = _randn(g, *((E, N, K) if tw else (E, K, N)), scale=0.1, dtype=dtype).requires_grad_()
    dy = _randn(g, rows, N, dtype=dtype)
    offsets = torch.tensor([0, *np.cumsum(sizes)], dtype=torch.int32, device=DEV)
    y = tdb.linear_grouped(x, w, offsets, transpose_w=tw, checkpoint=True)
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    plain = tdb.linear_grouped(x, w, offsets, transpose_w=tw)
    assert torch.equal(y, plain)
    assert torch.equal(dx, torch.autograd.grad(plain, x, dy)[0])
    kept = lo.values(*_quantized(x.detach()), 1)
    most = torch.finfo(dtype).max
    kept = kept.clamp(-most, most)
    for e, (i, j) in enumerate(lo.ranges(offsets.tolist())):
        left, right = (dy.double().cpu()[i:j], kept[i:j])
        ref, mag = lo.product(*((left.t(), right) if tw else (right.t(), left)))
        lo.check(dw[e], ref, mag, j - i, f"dw {e}")


def test_kept_values_that_round_past_fp16():
    """65504 in blocks of 8 bits is 256 * 2^8 = 65536, which fp16 does not have: its largest."""
    x = torch.full((4, 128), 65504.0, dtype=torch.float16, device=DEV)
    w = torch.zeros(1, 128, 8, dtype=torch.float16, device=DEV, requires_grad=True)
    dy = torch.full((4, 8), 2.0 ** -10, dtype=torch.float16, device=DEV)
    off = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    dw, = torch.autograd.grad(tdb.linear_grouped(x, w, off, checkpoint=True), w, dy)
    assert torch.equal(dw, torch.full_like(dw, 4 * 65504.0 / 1024))


@pytest.mark.parametrize("need", ["x", "w", "none"])
def test_kept_missing_gradients(need):
    g = _gen(3)
    x, w = _randn(g, 20, 40, dtype=torch.bfloat16), _randn(g, 2, 40, 24, dtype=torch.bfloat16)
    off = torch.tensor([0, 12, 18], dtype=torch.int32, device=DEV)
    x.requires_grad_(need == "x"), w.requires_grad_(need == "w")
    y = tdb.linear_grouped(x, w, off, checkpoint=True)
    assert torch.equal(y.detach(), tdb.matmul_grouped(x.detach(), w.detach(), off))
    if need != "none":
        torch.autograd.grad(y, x if need == "x" else w, torch.ones_like(y))


def test_kept_memory():
    """What a step keeps: 8 bits a value and a scale for each 128, not the input."""
    x = torch.randn(4096, 1024, device=DEV).to(torch.bfloat16)
    wide = torch.randn(4096, 2048, device=DEV).to(torch.bfloat16).requires_grad_()
    w = torch.randn(1, 1024, 64, device=DEV).to(torch.bfloat16).requires_grad_()
    off = torch.tensor([0, 4096], dtype=torch.int32, device=DEV)
    for call, cols, out in ((lambda k: tdb.linear_grouped(x + 1, w, off, checkpoint=k), 1024, 64),
                            (lambda k: tdb.gated_silu(wide + 1, checkpoint=k), 2048, 1024)):
        held = []
        for keep in (False, True):
            torch.cuda.synchronize()
            before = torch.cuda.memory_allocated()
            y = call(keep)
            held.append(torch.cuda.memory_allocated() - before - 2 * 4096 * out)
            del y
        assert held[0] >= 2 * 4096 * cols
        assert held[1] <= 4096 * cols * (1 + 4 / 128) + (1 << 20), held


# --------------------------------------------------------------- streams, graphs, together
def _step_calls():
    """name -> (make(seed) -> inputs, call(inputs) -> outputs), each a training step or a call."""
    E = 6
    order, offsets = _groups((30, 0, 25, 9, 16, 10), 100, 5)

    def make_route(seed):
        return [_logits(3000, 40, torch.float32, seed).requires_grad_(), _randn(_gen(seed), 3000, 4)]

    def route(v):
        gates, experts, counts, loss = tdb.route_experts(v[0], 4, renormalize=True)
        return [gates, experts, counts, loss,
                *torch.autograd.grad((gates, loss), v[0], (v[1], torch.ones_like(loss)))]

    def make_group(seed):
        return [torch.randint(-1, 70, (20000,), generator=_gen(seed)).to(DEV)]

    def group(v):
        return list(tdb.group_rows(v[0], 64))

    def make_adapters(seed):
        y, x, a, b, d, s = _adapter_inputs(100, E, 9, 520, 300, torch.bfloat16, seed)
        return [*(t.requires_grad_() for t in (y, x, a, b)), d, s]

    def adapters(v):
        out = tdb.add_adapters(*v[:4], order, offsets, scale=v[5])
        return [out, *torch.autograd.grad(out, v[:4], v[4])]

    def make_gated(seed):
        return [_wide(100, 600, torch.bfloat16, seed).requires_grad_(), _wide(100, 300, torch.bfloat16, seed + 1)]

    def gated(v):
        h = tdb.gated_silu(v[0], checkpoint=True)
        return [h, *torch.autograd.grad(h, v[0], v[1])]

    def make_kept(seed):
        g = _gen(seed)
        return [_randn(g, 100, 200, dtype=torch.bfloat16).requires_grad_(),
                _randn(g, E, 200, 130, dtype=torch.bfloat16).requires_grad_(), _randn(g, 100, 130, dtype=torch.bfloat16)]

    def kept(v):
        y = tdb.linear_grouped(v[0], v[1], offsets, checkpoint=True)
        return [y, *torch.autograd.grad(y, v[:2], v[2])]

    return dict(route=(make_route, route), group=(make_group, group), adapters=(make_adapters, adapters),
                gated=(make_gated, gated), kept=(make_kept, kept))


CALLS = ["route", "group", "adapters", "gated", "kept"]


@pytest.mark.parametrize("name", CALLS)
def test_same_bits_on_another_stream(name):
    make, call = _step_calls()[name]
    v = make(1)
    ref = call(v)
    again = call(v)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = call(v)
    torch.cuda.current_stream().wait_stream(side)
    for a, b, c in zip(ref, got, again):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("name", CALLS)
def test_two_calls_at_once(name):
    """Two streams, different inputs, many calls: workspaces are each call's own."""
    make, call = _step_calls()[name]
    v = [make(1), make(2)]
    ref = [call(v[0]), call(v[1])]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(call(v[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            for a, b in zip(ref[i], g):
                assert torch.equal(a, b)


@pytest.mark.parametrize("name", CALLS)
def test_graph_replays_follow_their_inputs(name):
    """Captured once, replayed with new inputs, eager work in between."""
    make, call = _step_calls()[name]
    v = make(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(v)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(v)
    for seed in (2, 3, 1):
        fresh = make(seed)
        with torch.no_grad():
            for a, b in zip(v, fresh):
                a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        ref = call(fresh)
        for a, b in zip(out, ref):
            assert torch.equal(a, b), seed


@pytest.mark.parametrize("name", CALLS)
def test_two_graphs_at_once(name):
    """Captured one after the other, replayed on two streams at once: each has its own workspace."""
    make, call = _step_calls()[name]
    v = [make(1), make(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ref = [[t.detach() for t in call(w)] for w in v]
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for w in v:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call(w)
        graphs.append(graph), outs.append(out)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for out, r in zip(outs, ref):
            assert all(torch.equal(a, b) for a, b in zip(out, r))


@pytest.mark.parametrize("name", ["route", "adapters", "gated", "kept"])
def test_saved_tensors_kept_on_the_host(name):
    """What the backward pass gets back need not have the strides that were saved."""
    make, call = _step_calls()[name]
    v = make(1)
    ref = call(v)
    with torch.autograd.graph.save_on_cpu():
        got = call(v)
    assert all(torch.equal(a, b) for a, b in zip(ref, got))


@pytest.mark.parametrize("call", ["group", "dequantize"])
def test_a_given_stream(call):
    """stream=: operands may be dropped at once, and a stream of another device is refused."""
    side = torch.cuda.Stream()
    ids = torch.randint(0, 50, (100000,), generator=_gen(1)).to(DEV)
    q, s = tdb.quantize_fp8(_wide(500, 700, torch.bfloat16, 1))
    ref = tdb.group_rows(ids, 50) if call == "group" else [tdb.dequantize_fp8(q, s)]
    torch.cuda.synchronize()
    for _ in range(5):
        i, u, t = ids.clone(), q.clone(), s.clone()
        side.wait_stream(torch.cuda.current_stream())
        got = tdb.group_rows(i, 50, stream=side) if call == "group" else [tdb.dequantize_fp8(u, t, stream=side)]
        del i, u, t
        torch.zeros(500, 700, device=DEV)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, got))


# ---------------------------------------------------------------------- past 32-bit offsets
def test_offsets_past_32_bits():
    """Tensors of more than 2^32 bytes and 2^31 elements: the last rows against the same rows alone."""
    g = torch.Generator(device="cuda").manual_seed(1)
    T, N = 300000, 8192

    def rows(cols):
        return torch.randn(T, cols, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)
    x, y = rows(N), rows(64)
    assert x.numel() > 1 << 31
    last = slice(T - 40, T)
    # gated: x as gate and up; its gradient
    leaf = x.requires_grad_()
    h = tdb.gated_silu(leaf, checkpoint=True)
    dx, = torch.autograd.grad(h, leaf, torch.ones_like(h))
    few = x[last].detach().requires_grad_()
    ref = tdb.gated_silu(few, checkpoint=True)
    assert torch.equal(h[last], ref)
    assert torch.equal(dx[last], torch.autograd.grad(ref, few, torch.ones_like(ref))[0])
    del h, dx, ref
    x = x.detach()
    q, s = tdb.quantize_fp8(x)
    back = tdb.dequantize_fp8(q, s)
    assert torch.equal(back[last], tdb.dequantize_fp8(q[last], s[last]))
    del q, s, back
    # adapters: the wide axis in, and out
    a, b = _randn(_gen(1), 2, 4, N, scale=0.01, dtype=torch.bfloat16), _randn(_gen(2), 2, 4, 64, dtype=torch.bfloat16)
    order, offsets = torch.arange(T, device=DEV), torch.tensor([0, 1000, T], dtype=torch.int32, device=DEV)
    few = (torch.arange(40, device=DEV), torch.tensor([0, 0, 40], dtype=torch.int32, device=DEV))
    for ins, outs, p, r in ((x, y, a, b), (y, x, b, a)):
        full = tdb.add_adapters(outs, ins, p, r, order, offsets)
        ref = tdb.add_adapters(outs[last], ins[last], p, r, *few)
        # (the contraction's order of sums depends on the rows: half a step of bf16 each)
        assert float((full[last] - ref).abs().max()) <= 2.0 ** -8 * float(ref.abs().max())
        del full
    # router: 2^31 logits
    z = x.view(-1, 1024)
    gates, experts, _, _ = tdb.route_experts(z, 2)
    ref = tdb.route_experts(z[-50:], 2)
    assert torch.equal(gates[-50:], ref[0]) and torch.equal(experts[-50:], ref[1])


# ------------------------------------------------------------------------------- as one layer
def _plain_layer(layer, x, requests, valid):
    """RoutedLayer without its shared layer in 64 bits, from elementary operations: (y, loss), of the
    experts that the layer takes (they are compared on their own)."""
    up = {n: getattr(layer, n).detach().double().cpu().requires_grad_() for n in ("router", "w_in", "w_out", "down", "up")}
    z = x.detach().double().cpu().requires_grad_()
    T, E, k = x.shape[0], layer.experts, layer.top
    p = torch.softmax(z @ up["router"][0], 1)
    with torch.no_grad():
        logits = tdb.linear_grouped(x.detach().float(), layer.router.detach(), torch.tensor([0, T], dtype=torch.int32, device=DEV))
        _, experts, counts, _ = tdb.route_experts(logits, k, valid=valid, renormalize=True)
    experts, on = experts.cpu().long(), valid.cpu()
    best = torch.topk(p.detach(), k, 1).values[:, -1]
    assert (p.detach().gather(1, experts.clamp_min(0)).amin(1)[on] >= best[on] * (1 - 1e-4)).all()
    g = p.gather(1, experts.clamp_min(0)) * on[:, None]
    g = g / g.sum(1, keepdim=True).clamp_min(1e-300)
    H = layer.w_out.shape[1]
    y = torch.zeros_like(z)
    for j in range(k):
        e = experts[:, j].clamp_min(0)
        h = torch.einsum("tk,tkn->tn", z, up["w_in"][e])
        h = h[:, :H] * torch.sigmoid(h[:, :H]) * h[:, H:]
        y = y + g[:, j, None] * torch.einsum("tk,tkn->tn", h, up["w_out"][e])
    a = requests.cpu().clamp_min(0)
    u = torch.einsum("tk,trk->tr", z, up["down"][a])
    y = y + torch.einsum("tr,trn->tn", u, up["up"][a]) * (requests.cpu() >= 0)[:, None]
    f = counts.cpu().double() / max(int(counts.sum()), 1)
    loss = E * (f * (p * on[:, None]).sum(0)).sum() / int(on.sum())
    return y, loss, z, up


def test_routed_layer_as_a_whole():
    """All operators together in FP32: results and every gradient against 64 bits.  Each is a chain of
    at most six FP32 sums of up to 260 terms, and so within 6 * 2 * 260 u = 4e-4 of its norm even if
    all roundings went one way."""
    from tiled_double_buffered_amd.expert_layer import RoutedLayer
    T, width, hidden = 90, 72, 130
    layer = RoutedLayer(width, hidden, 6, DEV, top=2, adapters=3, rank=5, dtype=torch.float32, checkpoint=False)
    with torch.no_grad():
        layer.shared.zero_()
    g = _gen(4)
    x = _randn(g, T, width).requires_grad_()
    requests = torch.randint(-1, 3, (T,), generator=g).to(DEV)
    valid = (torch.arange(T) % 7 != 3).to(DEV)
    dy = _randn(g, T, width)
    y, loss = layer(x, requests, valid)
    names = ("router", "w_in", "w_out", "down", "up")
    got = torch.autograd.grad((y, loss), [x, *(getattr(layer, n) for n in names)], (dy, torch.tensor(3.0, device=DEV)))
    ry, rloss, z, up = _plain_layer(layer, x, requests, valid)
    ref = torch.autograd.grad((ry, rloss), [z, *(up[n] for n in names)], (dy.double().cpu(), torch.tensor(3.0, dtype=torch.float64)))
    for name, a, b in zip(("y", "loss", "x", *names), (y, loss, *got), (ry, rloss, *ref)):
        off = float((a.detach().double().cpu() - b.detach()).norm() / b.detach().norm())
        assert off <= 4e-4, (name, off)


def test_routed_layer_with_8_bit_checkpoints():
    """The forward pass does not change; the gradients of what is kept move by the 8-bit rounding,
    2^-4 of a value at most, twice (the hidden values' input, and they themselves)."""
    from tiled_double_buffered_amd.expert_layer import RoutedLayer
    x = _randn(_gen(1), 200, 256, dtype=torch.bfloat16)
    requests = torch.randint(-1, 4, (200,), generator=_gen(2)).to(DEV)
    res = []
    for keep in (False, True):
        layer = RoutedLayer(256, 192, 5, DEV, checkpoint=keep)
        y, loss = layer(x, requests)
        res.append((y, loss, *torch.autograd.grad((y.float().square().sum(), loss), layer.parameters())))
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])
    for a, b in zip(res[0][2:], res[1][2:]):
        assert float((a - b).float().norm() / a.float().norm()) <= 2 * 2.0 ** -4 + 2.0 ** -6


def test_routed_layer_trains_and_serves():
    from tiled_double_buffered_amd import expert_layer
    layer = expert_layer.RoutedLayer(256, 128, 8, DEV, top=2)
    losses, x, requests = expert_layer.train_routed(layer, 300, 256, 3, DEV)
    assert len(losses) == 3 and all(math.isfinite(v) for pair in losses for v in pair)
    serve = layer.served()
    with torch.no_grad():
        whole = serve(x, requests)
        assert whole.shape == x.shape and torch.isfinite(whole.float()).all()
        for n in (1, 7):
            assert serve(x[:n], requests[:n]).shape == (n, 256)
        # the experts and the adapters of one token are its own: a batch of it alone gives the same
        # but for the tiles' order of sums
        one = serve(x[5:6], requests[5:6]).float()
        assert float((one - whole[5:6].float()).norm() / one.norm()) <= 2.0 ** -6
    assert expert_layer.main(["--tokens", "64", "--width", "128", "--hidden", "64", "--experts", "4", "--steps", "2", "--top", "2"]) == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("checkpoint", [False, True])
def test_routed_layer_of_other_types_trains_and_serves(checkpoint, dtype):
    from tiled_double_buffered_amd import expert_layer
    layer = expert_layer.RoutedLayer(128, 72, 5, DEV, top=2, dtype=dtype, checkpoint=checkpoint)
    losses, x, requests = expert_layer.train_routed(layer, 130, 128, 2, DEV)
    assert x.dtype == dtype and len(losses) == 2
    assert all(math.isfinite(v) for pair in losses for v in pair)
    with torch.no_grad():
        y = layer.served()(x, requests)
    assert y.dtype == dtype and y.shape == x.shape and torch.isfinite(y.float()).all()
