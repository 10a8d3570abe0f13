"""The operators around the experts' products on the host: exports, refusals before any HIP call,
workspace queries, argument checks of the tensor-level calls.  No call here passes validation with
made-up pointers: a call that passed would launch a kernel on them."""
import os
import re

import pytest

torch = pytest.importorskip("torch")
import tiled_double_buffered_amd as tdb  # noqa: E402
from tiled_double_buffered_amd import build, experts  # noqa: E402

HEADER = os.path.join(build.INCLUDE, "gemm_experts.h")
P = [0x7F0000000000 + i * 0x1000000000 for i in range(12)]
BF16, F16, F32 = 0, 1, 2


def test_header_binding_and_exports_agree():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^(?:int|int64_t) (gemm_\w+)\s*\(", text, flags=re.M))
    assert names == set(experts.SIGNATURES)
    out = os.popen(f"nm -D --defined-only {tdb._binding.LIB_PATH}").read()
    for n in names:
        assert re.search(rf"\bT {n}$", out, re.M), n
        assert hasattr(tdb, n) and n in dir(tdb)
    for name, value in (("GEMM_ROUTE_MAX_EXPERTS", experts.MAX_EXPERTS),
                        ("GEMM_ROUTE_MAX_CHOSEN", experts.MAX_CHOSEN),
                        ("GEMM_GROUP_MAX_EXPERTS", experts.MAX_GROUPS),
                        ("GEMM_ADAPTERS_MAX_RANK", experts.MAX_RANK)):
        assert re.search(rf"#define {name} {value}\b", text), name


def _route(rows=4, E=8, k=2, X=P[0], ldx=8, t=F32, valid=P[1], norm=0, gates=P[2], experts=P[3],
           counts=P[4], sums=P[5], loss=P[6], ws=None, n=0):
    return tdb.gemm_route(rows, E, k, X, ldx, t, valid, norm, gates, experts, counts, sums, loss,
                          ws, n, None)


@pytest.mark.parametrize("change, code", [
    (dict(rows=-1), tdb.ERR_NEGATIVE_DIM), (dict(E=-1), tdb.ERR_NEGATIVE_DIM),
    (dict(k=-1), tdb.ERR_NEGATIVE_DIM), (dict(t=3), tdb.ERR_BAD_TYPE),
    (dict(k=0), tdb.ERR_BAD_CONFIG), (dict(k=9), tdb.ERR_BAD_CONFIG),
    (dict(E=0), tdb.ERR_BAD_CONFIG), (dict(E=1025, ldx=1025), tdb.ERR_BAD_CONFIG),
    (dict(E=32, ldx=32, k=17), tdb.ERR_BAD_CONFIG), (dict(ldx=7), tdb.ERR_BAD_LD),
    (dict(rows=100000), tdb.ERR_BAD_LD), (dict(rows=100000, n=1 << 30), tdb.ERR_NULL_PTR),
    (dict(X=None), tdb.ERR_NULL_PTR), (dict(gates=None), tdb.ERR_NULL_PTR),
    (dict(experts=None), tdb.ERR_NULL_PTR), (dict(counts=None), tdb.ERR_NULL_PTR),
    (dict(sums=None), tdb.ERR_NULL_PTR), (dict(loss=None), tdb.ERR_NULL_PTR),
    (dict(X=P[0] + 2), tdb.ERR_MISALIGNED), (dict(loss=P[6] + 2), tdb.ERR_MISALIGNED),
    (dict(rows=100000, n=1 << 30, ws=P[7] + 4), tdb.ERR_MISALIGNED),
    (dict(gates=P[0] + 8), tdb.ERR_ALIAS), (dict(experts=P[2]), tdb.ERR_ALIAS),
    (dict(loss=P[5]), tdb.ERR_ALIAS), (dict(counts=P[1]), tdb.ERR_ALIAS),
    (dict(rows=1 << 31), tdb.ERR_BAD_LD), (dict(ldx=1 << 61), tdb.ERR_TOO_LARGE),
    (dict(rows=1 << 31, n=1 << 40, ws=P[7]), tdb.ERR_TOO_LARGE),
    (dict(rows=1 << 30, n=1 << 40, ws=P[7]), tdb.ERR_TOO_LARGE),  # counts past 32 bits
])
def test_route_refusals(change, code):
    assert _route(**change) == code


def _route_grad(rows=4, E=8, k=2, X=P[0], ldx=8, t=F32, valid=P[1], norm=1, gates=P[2],
                experts=P[3], counts=P[4], sums=P[5], dg=P[6], dl=P[7], DX=P[8], lddx=8):
    return tdb.gemm_route_grad(rows, E, k, X, ldx, t, valid, norm, gates, experts, counts, sums, dg,
                               dl, DX, lddx, None)


@pytest.mark.parametrize("change, code", [
    (dict(rows=-1), tdb.ERR_NEGATIVE_DIM), (dict(t=-1), tdb.ERR_BAD_TYPE),
    (dict(k=9), tdb.ERR_BAD_CONFIG), (dict(ldx=7), tdb.ERR_BAD_LD), (dict(lddx=7), tdb.ERR_BAD_LD),
    (dict(X=None), tdb.ERR_NULL_PTR), (dict(DX=None), tdb.ERR_NULL_PTR),
    (dict(gates=None), tdb.ERR_NULL_PTR), (dict(sums=None), tdb.ERR_NULL_PTR),
    (dict(DX=P[8] + 2), tdb.ERR_MISALIGNED), (dict(dl=P[7] + 1), tdb.ERR_MISALIGNED),
    (dict(DX=P[0]), tdb.ERR_ALIAS), (dict(DX=P[6]), tdb.ERR_ALIAS), (dict(DX=P[7]), tdb.ERR_ALIAS),
    (dict(rows=1 << 31), tdb.ERR_TOO_LARGE),
])
def test_route_grad_refusals(change, code):
    assert _route_grad(**change) == code


def _group(n=64, E=8, ids=P[0], size=4, order=P[1], place=P[2], off=P[3], ws=None, bytes_=0):
    return tdb.gemm_group_rows(n, E, ids, size, order, place, off, ws, bytes_, None)


@pytest.mark.parametrize("change, code", [
    (dict(n=-1), tdb.ERR_NEGATIVE_DIM), (dict(E=-1), tdb.ERR_NEGATIVE_DIM),
    (dict(size=2), tdb.ERR_BAD_TYPE), (dict(E=4097), tdb.ERR_BAD_CONFIG),
    (dict(n=1 << 31), tdb.ERR_TOO_LARGE), (dict(n=100000), tdb.ERR_BAD_LD),
    (dict(n=100000, bytes_=1 << 30), tdb.ERR_NULL_PTR), (dict(ids=None), tdb.ERR_NULL_PTR),
    (dict(order=None), tdb.ERR_NULL_PTR), (dict(off=None), tdb.ERR_NULL_PTR),
    (dict(ids=P[0] + 2), tdb.ERR_MISALIGNED), (dict(ids=P[0] + 4, size=8), tdb.ERR_MISALIGNED),
    (dict(place=P[2] + 4), tdb.ERR_MISALIGNED), (dict(order=P[0]), tdb.ERR_ALIAS),
    (dict(place=P[1] + 8), tdb.ERR_ALIAS), (dict(off=P[0] + 4), tdb.ERR_ALIAS),
])
def test_group_refusals(change, code):
    assert _group(**change) == code


def _down(rows=4, K=64, r=8, E=2, order=P[0], off=P[1], X=P[2], ldx=64, A=P[3], lda=64, sA=512,
          scale=P[4], U=P[5], splits=1, join=0, t=BF16):
    return tdb.gemm_adapters_down(rows, K, r, E, order, off, X, ldx, A, lda, sA, scale, U, splits,
                                  join, t, None)


@pytest.mark.parametrize("change, code", [
    (dict(K=-1), tdb.ERR_NEGATIVE_DIM), (dict(t=5), tdb.ERR_BAD_TYPE),
    (dict(r=129), tdb.ERR_BAD_CONFIG), (dict(splits=0), tdb.ERR_BAD_CONFIG),
    (dict(splits=65), tdb.ERR_BAD_CONFIG), (dict(ldx=63), tdb.ERR_BAD_LD),
    (dict(lda=63), tdb.ERR_BAD_LD), (dict(sA=-1), tdb.ERR_BAD_LD),
    (dict(order=None), tdb.ERR_NULL_PTR), (dict(U=None), tdb.ERR_NULL_PTR),
    (dict(X=None), tdb.ERR_NULL_PTR), (dict(order=P[0] + 4), tdb.ERR_MISALIGNED),
    (dict(A=P[3] + 1), tdb.ERR_MISALIGNED), (dict(scale=P[4] + 2), tdb.ERR_MISALIGNED),
    (dict(U=P[2]), tdb.ERR_ALIAS), (dict(U=P[4]), tdb.ERR_ALIAS), (dict(U=P[0] + 16), tdb.ERR_ALIAS),
    (dict(U=P[5] + 8), tdb.ERR_MISALIGNED),
    (dict(rows=1 << 31), tdb.ERR_TOO_LARGE), (dict(sA=1 << 61), tdb.ERR_TOO_LARGE),
])
def test_down_refusals(change, code):
    assert _down(**change) == code


def _up(rows=4, N=64, r=8, E=2, order=P[0], off=P[1], U=P[2], splits=1, B=P[3], ldb=64, sB=512,
        Y=P[4], ldy=64, O=P[5], ldo=64, t=BF16):
    return tdb.gemm_adapters_up(rows, N, r, E, order, off, U, splits, B, ldb, sB, Y, ldy, O, ldo, t,
                                None)


@pytest.mark.parametrize("change, code", [
    (dict(N=-1), tdb.ERR_NEGATIVE_DIM), (dict(t=5), tdb.ERR_BAD_TYPE),
    (dict(r=129), tdb.ERR_BAD_CONFIG), (dict(splits=0), tdb.ERR_BAD_CONFIG),
    (dict(ldb=63), tdb.ERR_BAD_LD), (dict(ldy=63), tdb.ERR_BAD_LD), (dict(ldo=63), tdb.ERR_BAD_LD),
    (dict(off=None), tdb.ERR_NULL_PTR), (dict(O=None), tdb.ERR_NULL_PTR),
    (dict(U=None), tdb.ERR_NULL_PTR), (dict(O=P[5] + 1), tdb.ERR_MISALIGNED),
    (dict(Y=P[4] + 1), tdb.ERR_MISALIGNED), (dict(O=P[4]), tdb.ERR_ALIAS),
    (dict(O=P[2]), tdb.ERR_ALIAS), (dict(O=P[0]), tdb.ERR_ALIAS),
    (dict(N=1 << 31, ldb=1 << 31, ldy=1 << 31, ldo=1 << 31), tdb.ERR_TOO_LARGE),
    (dict(ldo=1 << 61), tdb.ERR_TOO_LARGE),
])
def test_up_refusals(change, code):
    assert _up(**change) == code


def _grad(rows=4, r=8, E=2, order=P[0], off=P[1], K=64, V=P[2], vs=1, X=P[3], ldx=64, DA=P[4], ldda=64,
          sA=512, N=32, U=P[5], us=1, DO=P[6], ldd=32, DB=P[7], lddb=32, sB=256, ws=None, n=0, t=BF16):
    return tdb.gemm_adapters_grad(rows, r, E, order, off, K, V, vs, X, ldx, DA, ldda, sA, N, U, us, DO,
                                  ldd, DB, lddb, sB, ws, n, t, None)


@pytest.mark.parametrize("change, code", [
    (dict(E=-1), tdb.ERR_NEGATIVE_DIM), (dict(N=-1), tdb.ERR_NEGATIVE_DIM), (dict(t=5), tdb.ERR_BAD_TYPE),
    (dict(r=129), tdb.ERR_BAD_CONFIG), (dict(vs=0), tdb.ERR_BAD_CONFIG), (dict(us=65), tdb.ERR_BAD_CONFIG),
    (dict(ldx=63), tdb.ERR_BAD_LD), (dict(ldda=63), tdb.ERR_BAD_LD), (dict(ldd=31), tdb.ERR_BAD_LD),
    (dict(sA=511), tdb.ERR_BAD_LD), (dict(sB=255), tdb.ERR_BAD_LD),
    (dict(rows=100000), tdb.ERR_BAD_LD), (dict(rows=100000, n=1 << 30), tdb.ERR_NULL_PTR),
    (dict(DA=None), tdb.ERR_NULL_PTR), (dict(X=None), tdb.ERR_NULL_PTR), (dict(DB=None), tdb.ERR_NULL_PTR),
    (dict(order=None), tdb.ERR_NULL_PTR), (dict(off=None), tdb.ERR_NULL_PTR),
    (dict(DA=P[4] + 1), tdb.ERR_MISALIGNED), (dict(U=P[5] + 4), tdb.ERR_MISALIGNED),
    (dict(order=P[0] + 4), tdb.ERR_MISALIGNED), (dict(DB=P[3]), tdb.ERR_ALIAS), (dict(DA=P[7]), tdb.ERR_ALIAS),
    (dict(DA=P[2]), tdb.ERR_ALIAS), (dict(DB=P[1]), tdb.ERR_ALIAS),
    (dict(rows=100000, n=1 << 30, ws=P[4]), tdb.ERR_ALIAS), (dict(rows=1 << 31), tdb.ERR_TOO_LARGE),
    (dict(K=0, N=0, order=None), tdb.OK), (dict(N=0, DA=None), tdb.ERR_NULL_PTR),
    (dict(K=0, DA=None, X=None, V=None, DB=P[6]), tdb.ERR_ALIAS),
])
def test_adapter_grad_refusals(change, code):
    assert _grad(**change) == code


def _gated(rows=4, N=200, X=P[0], ldx=400, t=BF16, H=P[1], ldh=200, Q=P[2], ldq=400, S=P[3], lds=4):
    return tdb.gemm_gated(rows, N, X, ldx, t, H, ldh, Q, ldq, S, lds, None)


@pytest.mark.parametrize("change, code", [
    (dict(rows=-1), tdb.ERR_NEGATIVE_DIM), (dict(t=3), tdb.ERR_BAD_TYPE),
    (dict(S=None), tdb.ERR_NULL_PTR), (dict(X=None), tdb.ERR_NULL_PTR),
    (dict(H=None), tdb.ERR_NULL_PTR), (dict(ldx=399), tdb.ERR_BAD_LD), (dict(ldh=199), tdb.ERR_BAD_LD),
    (dict(ldq=399), tdb.ERR_BAD_LD), (dict(lds=3), tdb.ERR_BAD_LD),
    (dict(H=P[1] + 1), tdb.ERR_MISALIGNED), (dict(S=P[3] + 2), tdb.ERR_MISALIGNED),
    (dict(H=P[0]), tdb.ERR_ALIAS), (dict(Q=P[1]), tdb.ERR_ALIAS), (dict(S=P[0] + 4), tdb.ERR_ALIAS),
    (dict(rows=1 << 31), tdb.ERR_TOO_LARGE),
    (dict(rows=1 << 30, N=1 << 20, ldx=1 << 21, ldh=1 << 20, ldq=1 << 21, lds=1 << 14), tdb.ERR_ALIAS),
])
def test_gated_refusals(change, code):
    assert _gated(**change) == code


def _gated_grad(rows=4, N=200, X=None, ldx=0, Q=P[2], ldq=400, S=P[3], lds=4, DH=P[0], lddh=200,
                DX=P[1], lddx=400, t=BF16):
    return tdb.gemm_gated_grad(rows, N, X, ldx, Q, ldq, S, lds, DH, lddh, DX, lddx, t, None)


@pytest.mark.parametrize("change, code", [
    (dict(N=-1), tdb.ERR_NEGATIVE_DIM), (dict(t=3), tdb.ERR_BAD_TYPE),
    (dict(Q=None), tdb.ERR_NULL_PTR), (dict(Q=None, S=None), tdb.ERR_NULL_PTR),
    (dict(DH=None), tdb.ERR_NULL_PTR), (dict(DX=None), tdb.ERR_NULL_PTR),
    (dict(X=P[4], ldx=399), tdb.ERR_BAD_LD), (dict(lddh=199), tdb.ERR_BAD_LD),
    (dict(lddx=399), tdb.ERR_BAD_LD), (dict(lds=3), tdb.ERR_BAD_LD),
    (dict(DX=P[1] + 1), tdb.ERR_MISALIGNED), (dict(DX=P[0]), tdb.ERR_ALIAS),
    (dict(DX=P[3]), tdb.ERR_ALIAS), (dict(X=P[1], ldx=400), tdb.ERR_ALIAS),
])
def test_gated_grad_refusals(change, code):
    assert _gated_grad(**change) == code


def _dequantize(rows=4, cols=200, Q=P[0], ldq=200, S=P[1], lds=2, br=1, Y=P[2], ldy=200, t=BF16):
    return tdb.gemm_fp8_dequantize(rows, cols, Q, ldq, S, lds, br, Y, ldy, t, None)


@pytest.mark.parametrize("change, code", [
    (dict(rows=-1), tdb.ERR_NEGATIVE_DIM), (dict(t=3), tdb.ERR_BAD_TYPE),
    (dict(br=64), tdb.ERR_BAD_CONFIG), (dict(ldq=199), tdb.ERR_BAD_LD), (dict(lds=1), tdb.ERR_BAD_LD),
    (dict(ldy=199), tdb.ERR_BAD_LD), (dict(Q=None), tdb.ERR_NULL_PTR), (dict(S=None), tdb.ERR_NULL_PTR),
    (dict(Y=P[2] + 1), tdb.ERR_MISALIGNED), (dict(Y=P[0]), tdb.ERR_ALIAS), (dict(Y=P[1]), tdb.ERR_ALIAS),
    (dict(cols=1 << 31, ldq=1 << 31, ldy=1 << 31, lds=1 << 25), tdb.ERR_TOO_LARGE),
])
def test_dequantize_refusals(change, code):
    assert _dequantize(**change) == code


def test_empty_calls_launch_nothing():
    assert _route_grad(rows=0, X=None) == tdb.OK
    assert _down(rows=0, X=None) == tdb.OK
    assert _down(E=0, A=None) == tdb.OK
    assert _up(rows=0, O=None) == tdb.OK
    assert _up(N=0, O=None) == tdb.OK
    assert _grad(r=0, DA=None) == tdb.OK
    assert _gated(rows=0, X=None) == tdb.OK
    assert _gated_grad(N=0, DX=None) == tdb.OK
    assert _dequantize(cols=0, Q=None) == tdb.OK


def test_workspace_and_split_queries():
    assert tdb.gemm_route_workspace(64, 256) == 0
    assert tdb.gemm_route_workspace(65, 256) == 2 * (2 * 256 + 1) * 4
    assert tdb.gemm_route_workspace(1 << 20, 64) == 256 * (2 * 64 + 1) * 4
    assert tdb.gemm_route_workspace(-1, 64) == tdb.ERR_NEGATIVE_DIM
    assert tdb.gemm_route_workspace(1, 2000) == tdb.ERR_BAD_CONFIG
    assert tdb.gemm_group_rows_workspace(2048, 64) == 0
    assert tdb.gemm_group_rows_workspace(2049, 64) == 16 * 65 * 4
    for n in (10000, 1 << 20, 1 << 30):  # a bounded number of workgroups, whatever the rows
        assert tdb.gemm_group_rows_workspace(n, 64) <= 128 * 65 * 4
    assert tdb.gemm_group_rows_workspace(1, 5000) == tdb.ERR_BAD_CONFIG
    assert tdb.gemm_adapters_splits(1, 4096, 16, 4) > 1
    assert tdb.gemm_adapters_splits(100000, 4096, 16, 4) == 1
    assert tdb.gemm_adapters_splits(0, 0, 1, 0) == 1
    assert tdb.gemm_adapters_splits(1, 4096, 129, 4) == tdb.ERR_BAD_CONFIG
    assert tdb.gemm_adapters_grad_workspace(4, 4096, 4096, 16, 4, BF16) == 0
    assert tdb.gemm_adapters_grad_workspace(100000, 128, 0, 16, 1, F32) > 0
    assert tdb.gemm_adapters_grad_workspace(-4, 128, 128, 16, 1, F16) == tdb.ERR_NEGATIVE_DIM
    assert tdb.gemm_adapters_grad_workspace(4, 128, 128, 16, 1, 3) == tdb.ERR_BAD_TYPE
    most = (1 << 31) - 2000
    assert tdb.gemm_adapters_grad_workspace(most, most, most, 128, most, F32) == 0  # one run each
    assert 0 < tdb.gemm_adapters_grad_workspace(most, 4096, 1024, 128, most, F32) < 1 << 60


def test_gradient_workspace_goes_by_rows_and_not_by_adapters():
    """Sums that another launch adds there are only of adapters with more rows than a run has: at
    most twice as many as the rows fill, whatever the number of adapters."""
    few = tdb.gemm_adapters_grad_workspace(8192, 4096, 4096, 64, 8, BF16)
    assert few > 0
    for E in (16, 512, 4096, 100000):
        assert tdb.gemm_adapters_grad_workspace(8192, 4096, 4096, 64, E, BF16) <= few
    for rows, E in ((8192, 4), (20000, 1000), (100000, 1), (1000, 1000)):
        need = tdb.gemm_adapters_grad_workspace(rows, 4096, 4096, 64, E, BF16)
        # (a run has 128 rows at least: the bytes of half of x's in FP32, a rank of 64 for its 128)
        assert need <= 2 * 2 * rows // 128 * 64 * 4096 * 4, (rows, E)


def test_tensor_calls_refuse_what_they_cannot_take():
    x = torch.zeros(4, 64)
    q = torch.zeros(4, 256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    order, off = torch.arange(4), torch.zeros(3, dtype=torch.int32)
    a, b = torch.zeros(2, 8, 64), torch.zeros(2, 8, 32)
    y = torch.zeros(4, 32)
    for call in (
        lambda: tdb.route_experts(x, 2),                                  # not on the GPU
        lambda: tdb.route_experts(x, 2, valid=torch.ones(3, dtype=torch.bool)),
        lambda: tdb.group_rows(off, 4),
        lambda: tdb.group_rows(off, -1),
        lambda: tdb.group_rows(off, 5000),
        lambda: tdb.add_adapters(y, x, a, b, order, off),
        lambda: tdb.add_adapters(y, x, a, b[:1], order, off),
        lambda: tdb.add_adapters(y, x, a[:, :, :60], b, order, off),
        lambda: tdb.add_adapters(y[:3], x, a, b, order, off),
        lambda: tdb.add_adapters(y, x, a[:, :0], b[:, :0], order, off),
        lambda: tdb.add_adapters(y, x, torch.zeros(2, 129, 64), torch.zeros(2, 129, 32), order, off),
        lambda: tdb.add_adapters(y, x, a, b, order, off, scale=torch.ones(3)),
        lambda: tdb.gated_silu(x),
        lambda: tdb.gated_silu(x[:, :63]),
        lambda: tdb.dequantize_fp8(q, torch.ones(4, 2)),
    ):
        with pytest.raises(ValueError):
            call()
    for call in (
        lambda: tdb.route_experts(x.int(), 2),
        lambda: tdb.route_experts(x[0], 2),
        lambda: tdb.route_experts(x, 2, valid=torch.ones(4)),
        lambda: tdb.group_rows(x, 4),
        lambda: tdb.group_rows([1, 2], 4),
        lambda: tdb.add_adapters(y.half(), x, a, b, order, off),
        lambda: tdb.add_adapters(y, x, a.half(), b, order, off),
        lambda: tdb.add_adapters(y, x, a[0], b[0], order, off),
        lambda: tdb.add_adapters(y, x, a, b, order, off, scale=torch.ones(2).double()),
        lambda: tdb.gated_silu(x.int()),
        lambda: tdb.gated_silu(None),
        lambda: tdb.dequantize_fp8(x, torch.ones(4, 1)),
        lambda: tdb.dequantize_fp8(q, torch.ones(4, 2), torch.float64),
    ):
        with pytest.raises(TypeError):
            call()


def test_forward_mode_derivatives_are_refused():
    """A dual tensor does not require a gradient, and no call answers it without its tangent."""
    from torch.autograd import forward_ad
    x, y = torch.randn(4, 64), torch.zeros(4, 32)
    a, b, scale = torch.zeros(2, 8, 64), torch.zeros(2, 8, 32), torch.ones(2)
    order, off = torch.arange(4), torch.zeros(3, dtype=torch.int32)

    def adapters(i, t):
        ops = [y, x, a, b, scale]
        ops[i] = t
        return tdb.add_adapters(*ops[:4], order, off, scale=ops[4])
    with forward_ad.dual_level():
        for t, call in ((x, lambda d: tdb.gated_silu(d)), (x, lambda d: tdb.gated_silu(d, checkpoint=True)),
                        (x, lambda d: tdb.route_experts(d, 2)),
                        *((t, lambda d, i=i: adapters(i, d)) for i, t in enumerate((y, x, a, b, scale)))):
            with pytest.raises(NotImplementedError):
                call(forward_ad.make_dual(t, torch.ones_like(t)))
            with pytest.raises(ValueError, match="GPU"):  # (no tangent: as outside)
                call(t)
    with pytest.raises(ValueError, match="GPU"):
        tdb.gated_silu(x)
