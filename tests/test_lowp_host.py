"""The low-precision and expert-grouped products on the host: exports, refusals before any HIP
call, argument checks of the tensor-level calls.  No call here passes validation with made-up
pointers: a call that passed would launch a kernel on them."""
import os
import re

import pytest

torch = pytest.importorskip("torch")
import tiled_double_buffered_amd as tdb  # noqa: E402
from tiled_double_buffered_amd import build, lowp  # noqa: E402

HEADER = os.path.join(build.INCLUDE, "gemm_lp.h")
PA, PB, PC, PS, PT, PO = (0x7F0000000000 + i * 0x1000000000 for i in range(6))
BF16, F16, F32 = 0, 1, 2


def test_header_binding_and_exports_agree():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^int (gemm_\w+)\s*\(", text, flags=re.M))
    assert names == set(lowp.SIGNATURES)
    out = os.popen(f"nm -D --defined-only {tdb._binding.LIB_PATH}").read()
    for n in names:
        assert re.search(rf"\bT {n}$", out, re.M), n
        assert hasattr(tdb, n)


def test_bad_type_has_a_message():
    assert tdb.gemm_f32_strerror(tdb.ERR_BAD_TYPE) == "unknown element type"


def _quant(rows=4, cols=200, X=PA, ldx=200, t=BF16, br=1, Q=PB, ldq=208, S=PS, lds=2, QT=None,
           ldqt=0, ST=None, ldst=0):
    return lowp.gemm_fp8_quantize(rows, cols, X, ldx, t, br, Q, ldq, S, lds, QT, ldqt, ST, ldst,
                                  None)


@pytest.mark.parametrize("change, code", [
    (dict(rows=-1), tdb.ERR_NEGATIVE_DIM), (dict(cols=-1), tdb.ERR_NEGATIVE_DIM),
    (dict(t=3), tdb.ERR_BAD_TYPE), (dict(br=64), tdb.ERR_BAD_CONFIG),
    (dict(ldx=199), tdb.ERR_BAD_LD), (dict(ldq=199), tdb.ERR_BAD_LD),
    (dict(lds=1), tdb.ERR_BAD_LD), (dict(S=None), tdb.ERR_NULL_PTR),
    (dict(Q=None, S=None), tdb.ERR_NULL_PTR), (dict(X=None), tdb.ERR_NULL_PTR),
    (dict(QT=PC), tdb.ERR_NULL_PTR), (dict(QT=PC, ldqt=3, ST=PT, ldst=1), tdb.ERR_BAD_LD),
    (dict(X=PA + 1), tdb.ERR_MISALIGNED), (dict(S=PS + 2), tdb.ERR_MISALIGNED),
    (dict(Q=PA + 16), tdb.ERR_ALIAS), (dict(S=PB + 4), tdb.ERR_ALIAS),
    (dict(rows=1 << 31), tdb.ERR_TOO_LARGE), (dict(ldx=1 << 61), tdb.ERR_TOO_LARGE),
])
def test_quantize_refusals(change, code):
    assert _quant(**change) == code


def _quant_exp(rows=4, cols=200, X=PA, ldx=200, t=BF16, br=1, Q=PB, ldq=208, S=PS, lds=4, QT=None,
               ldqt=0, ST=None, ldst=0):
    return lowp.gemm_fp8_quantize_exp(rows, cols, X, ldx, t, br, Q, ldq, S, lds, QT, ldqt, ST,
                                      ldst, None)


@pytest.mark.parametrize("change, code", [
    (dict(rows=-1), tdb.ERR_NEGATIVE_DIM), (dict(t=3), tdb.ERR_BAD_TYPE),
    (dict(br=2), tdb.ERR_BAD_CONFIG), (dict(lds=3), tdb.ERR_BAD_LD),
    (dict(QT=PC, ldqt=4, ST=PT, ldst=199), tdb.ERR_BAD_LD), (dict(S=None), tdb.ERR_NULL_PTR),
    (dict(S=PB + 4), tdb.ERR_ALIAS), (dict(X=PA + 1), tdb.ERR_MISALIGNED),
])
def test_quantize_exp_refusals(change, code):
    assert _quant_exp(**change) == code


def _fp8_exp(M=4, N=200, K=300, A=PA, lda=300, SA=PS, ldsa=4, B=PB, ldb=300, SB=PT, ldsb=200,
             C=PC, ldc=200, t=BF16):
    return lowp.gemm_fp8_exp(M, N, K, A, lda, SA, ldsa, B, ldb, SB, ldsb, C, ldc, t, None)


@pytest.mark.parametrize("change, code", [
    (dict(K=-1), tdb.ERR_NEGATIVE_DIM), (dict(t=-1), tdb.ERR_BAD_TYPE),
    (dict(ldsa=3), tdb.ERR_BAD_LD), (dict(ldsa=6), tdb.ERR_BAD_LD),
    (dict(ldsb=199), tdb.ERR_BAD_LD), (dict(ldb=299), tdb.ERR_BAD_LD),
    (dict(SA=None), tdb.ERR_NULL_PTR), (dict(SB=PT + 1), tdb.ERR_MISALIGNED),
    (dict(C=PT), tdb.ERR_ALIAS), (dict(N=1 << 31, ldc=1 << 31, ldsb=1 << 31), tdb.ERR_TOO_LARGE),
])
def test_fp8_exp_refusals(change, code):
    assert _fp8_exp(**change) == code


def test_empty_calls_launch_nothing():
    assert _quant(rows=0, X=None) == tdb.OK
    assert _fp8(M=0, A=None) == tdb.OK
    assert _fp8_exp(M=0, A=None) == tdb.OK
    assert _quant_exp(cols=0, X=None) == tdb.OK
    assert _fp8(N=0, C=None, ldc=1) == tdb.OK
    assert _grouped(rows=0, X=None) == tdb.OK
    assert _wgrad(E=0, D=None) == tdb.OK


def _fp8(M=4, N=200, K=300, E=1, off=None, A=PA, lda=300, SA=PS, ldsa=3, B=PB, ldb=300, sB=0,
         SB=PT, ldsb=3, sSB=0, bb=128, C=PC, ldc=200, t=BF16):
    return lowp.gemm_fp8(M, N, K, E, off, A, lda, SA, ldsa, B, ldb, sB, SB, ldsb, sSB, bb, C,
                         ldc, t, None)


@pytest.mark.parametrize("change, code", [
    (dict(M=-1), tdb.ERR_NEGATIVE_DIM), (dict(K=-1), tdb.ERR_NEGATIVE_DIM),
    (dict(E=-1), tdb.ERR_NEGATIVE_DIM), (dict(t=7), tdb.ERR_BAD_TYPE),
    (dict(bb=32), tdb.ERR_BAD_CONFIG), (dict(E=2), tdb.ERR_BAD_CONFIG),
    (dict(lda=299), tdb.ERR_BAD_LD), (dict(ldb=299), tdb.ERR_BAD_LD),
    (dict(ldc=199), tdb.ERR_BAD_LD), (dict(ldsa=2), tdb.ERR_BAD_LD),
    (dict(ldsb=2), tdb.ERR_BAD_LD), (dict(sB=-1), tdb.ERR_BAD_LD),
    (dict(A=None), tdb.ERR_NULL_PTR), (dict(SB=None), tdb.ERR_NULL_PTR),
    (dict(C=None), tdb.ERR_NULL_PTR), (dict(C=PC + 1), tdb.ERR_MISALIGNED),
    (dict(C=PC + 2, t=F32), tdb.ERR_MISALIGNED), (dict(SA=PS + 2), tdb.ERR_MISALIGNED),
    (dict(off=PO + 2), tdb.ERR_MISALIGNED), (dict(C=PB), tdb.ERR_ALIAS),
    (dict(C=PS), tdb.ERR_ALIAS), (dict(off=PC + 4), tdb.ERR_ALIAS),
    (dict(M=1 << 31), tdb.ERR_TOO_LARGE), (dict(lda=1 << 61), tdb.ERR_TOO_LARGE),
    (dict(ldsa=1 << 22), tdb.ERR_TOO_LARGE), (dict(ldsb=1 << 22), tdb.ERR_TOO_LARGE),
    (dict(E=1 << 30, off=PO, sB=1 << 40), tdb.ERR_TOO_LARGE),
])
def test_fp8_refusals(change, code):
    assert _fp8(**change) == code


def _grouped(rows=4, N=64, K=32, E=2, off=PO, X=PA, ldx=32, W=PB, ldw=64, sW=2048, tw=0, Y=PC,
             ldy=64, t=BF16):
    return lowp.gemm_grouped(rows, N, K, E, off, X, ldx, W, ldw, sW, tw, Y, ldy, t, None)


@pytest.mark.parametrize("change, code", [
    (dict(N=-1), tdb.ERR_NEGATIVE_DIM), (dict(t=-1), tdb.ERR_BAD_TYPE),
    (dict(ldx=31), tdb.ERR_BAD_LD), (dict(ldw=63), tdb.ERR_BAD_LD),
    (dict(tw=1, ldw=31), tdb.ERR_BAD_LD), (dict(ldy=63), tdb.ERR_BAD_LD),
    (dict(sW=-2), tdb.ERR_BAD_LD), (dict(off=None), tdb.ERR_NULL_PTR),
    (dict(W=None), tdb.ERR_NULL_PTR), (dict(Y=None), tdb.ERR_NULL_PTR),
    (dict(X=PA + 1), tdb.ERR_MISALIGNED), (dict(off=PO + 1), tdb.ERR_MISALIGNED),
    (dict(W=PB + 2, t=F32), tdb.ERR_MISALIGNED), (dict(Y=PA), tdb.ERR_ALIAS),
    (dict(Y=PB + 4096), tdb.ERR_ALIAS), (dict(K=1 << 31, ldx=1 << 31), tdb.ERR_TOO_LARGE),
])
def test_grouped_refusals(change, code):
    assert _grouped(**change) == code


def _wgrad(rows=8, M=16, N=32, E=2, off=PO, A=PA, lda=16, B=PB, ldb=32, D=PC, ldw=32, sW=512,
           t=F32):
    return lowp.gemm_grouped_wgrad(rows, M, N, E, off, A, lda, B, ldb, D, ldw, sW, t, None)


@pytest.mark.parametrize("change, code", [
    (dict(E=-1), tdb.ERR_NEGATIVE_DIM), (dict(t=9), tdb.ERR_BAD_TYPE),
    (dict(lda=15), tdb.ERR_BAD_LD), (dict(ldb=31), tdb.ERR_BAD_LD), (dict(ldw=31), tdb.ERR_BAD_LD),
    (dict(sW=511), tdb.ERR_BAD_LD), (dict(D=None), tdb.ERR_NULL_PTR),
    (dict(off=None), tdb.ERR_NULL_PTR), (dict(B=PB + 2), tdb.ERR_MISALIGNED),
    (dict(D=PA), tdb.ERR_ALIAS), (dict(D=PO), tdb.ERR_ALIAS),
    (dict(M=1 << 31, lda=1 << 31, sW=1 << 40), tdb.ERR_TOO_LARGE),
])
def test_wgrad_refusals(change, code):
    assert _wgrad(**change) == code


def test_tensor_calls_refuse_what_they_cannot_take():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    q = torch.zeros(4, 256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.ones(4, 2)
    off = torch.zeros(3, dtype=torch.int32)
    w = torch.zeros(2, 256, 64, dtype=torch.bfloat16)
    for call in (
        lambda: tdb.quantize_fp8(x),                              # not on the GPU
        lambda: tdb.quantize_fp8(x, block=(1, 64)),
        lambda: tdb.quantize_fp8(x.t()),                          # column stride
        lambda: tdb.quantize_fp8(x[:1].expand(4, 256)),           # overlapping rows
        lambda: tdb.matmul_fp8(q, s, q, s),
        lambda: tdb.matmul_grouped(x, w, off),
        lambda: tdb.linear_grouped(x, w, off),
        lambda: tdb.linear_fp8(x, x[:, :128]),                    # inner dimensions
    ):
        with pytest.raises(ValueError):
            call()
    for call in (
        lambda: tdb.quantize_fp8(x.int()),
        lambda: tdb.quantize_fp8(x[0]),
        lambda: tdb.quantize_fp8(None),
        lambda: tdb.matmul_fp8(x, s, q, s),
        lambda: tdb.matmul_fp8(q, s, q, s, out_dtype=torch.float64),
        lambda: tdb.matmul_fp8_grouped(q, s, q, s, None),
        lambda: tdb.linear_grouped(x[0], w, off),
        lambda: tdb.linear_fp8(x, x.float()),
        lambda: tdb.linear_fp8(x.int(), x.int()),
    ):
        with pytest.raises(TypeError):
            call()


# ------------------------------------------------------------------------- compiled structure
def test_compiled_kernels():
    """This library's own gfx950 assembly: no register spills, no packed FP32 arithmetic, and M0
    written only for a direct-to-LDS copy, one wait state and the load right behind it (the
    copies are inline assembly, whose M0 the compiler does not track)."""
    asm = build.device_asm()
    meta = build.kernel_metadata(asm)
    names = [n for n in meta if "gemmlp" in n]
    assert len(names) > 60
    for n in names:
        assert meta[n]["private_segment_fixed_size"] == 0, n
        assert meta[n]["group_segment_fixed_size"] <= 160 * 1024, n
        start = re.search(rf"^{re.escape(n)}:", asm, re.M).end()
        lines = [t.strip() for t in asm[start:asm.index(".Lfunc_end", start)].split("\n")]
        lines = [t for t in lines if t and not t.startswith((";", "."))]
        for i, t in enumerate(lines):
            assert not re.match(r"v_pk_(fma|mul|add)_f32\b", t), (n, t)
            if re.search(r"\bm0\b", t):
                assert t.startswith("s_mov_b32 m0,"), (n, t)
                assert lines[i + 1] == "s_nop 0", (n, lines[i + 1])
                assert re.match(r"buffer_load_dword(x4)? .*\blds$", lines[i + 2]), (n, lines[i + 2])


def test_8_bit_values_are_multiplied_in_16():
    """The 8-bit matrix instructions hold 13 bits below the largest of eight products: none of
    them may sum what the interface says is held in 32."""
    asm = build.device_asm()
    for n in [n for n in build.kernel_metadata(asm) if "gemmlp" in n]:
        start = re.search(rf"^{re.escape(n)}:", asm, re.M).end()
        body = asm[start:asm.index(".Lfunc_end", start)]
        assert not re.search(r"v_mfma\w*(f8f6f4|fp8|bf8)", body), n


def test_linear_fp8_of_no_depth_and_leading_axes_reaches_the_checks():
    """(3, 5, 0): the leading axes are 15 rows, which no -1 can stand for; refused on the CPU for
    living there alone."""
    for shape in ((3, 5, 0), (0,), (2, 0, 0)):
        with pytest.raises(ValueError, match="must live on the GPU"):
            tdb.linear_fp8(torch.zeros(shape), torch.zeros(4, 0))
