"""Low-precision and expert-grouped products on GPU tensors, through the C ABI of
include/gemm_lp.h: 8-bit floating point with a scale for each block of 128, and products with
one weight matrix per expert over ragged groups of rows, each with its gradient.

As in `matmul`, this module only checks arguments, allocates outputs and passes pointers,
strides and the stream; every value is computed in the library's HIP kernels, and there is no
other path: without the library, or on tensors that are not on the GPU, every call raises.

Calls are asynchronous.  `stream` (a torch.cuda.Stream of the operands' GPU) is where they run,
the current stream by default; what a call allocates belongs to that stream.  It does not wait for
work on other streams: what made the operands has to be done or waited for.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math

import torch
from torch.autograd import forward_ad

from . import _binding
from ._binding import GemmError

BLOCK = 128          # columns along the contraction that share a scale
E4M3_MAX = 448.0

_i64, _int, _vp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
# Every exported symbol and its C signature (kept in step with include/gemm_lp.h).
SIGNATURES = {
    "gemm_fp8_quantize": (_int, [_i64, _i64, _vp, _i64, _int, _int, _vp, _i64, _vp, _i64,
                                 _vp, _i64, _vp, _i64, _vp]),
    "gemm_fp8": (_int, [_i64, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _i64, _vp, _i64, _i64,
                        _vp, _i64, _i64, _int, _vp, _i64, _int, _vp]),
    "gemm_fp8_quantize_exp": (_int, [_i64, _i64, _vp, _i64, _int, _int, _vp, _i64, _vp, _i64,
                                     _vp, _i64, _vp, _i64, _vp]),
    "gemm_fp8_exp": (_int, [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp,
                            _i64, _int, _vp]),
    "gemm_grouped": (_int, [_i64, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _i64, _i64, _int,
                            _vp, _i64, _int, _vp]),
    "gemm_grouped_wgrad": (_int, [_i64, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _i64, _vp,
                                  _i64, _i64, _int, _vp]),
}
TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}  # GEMM_LP_*
_F8 = torch.float8_e4m3fn
_lib = None


def load():
    """The library with this module's entry points typed.  Raises if it is not built."""
    global _lib
    if _lib is None:
        lib = _binding.load()
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _lib = lib
    return _lib


# ----------------------------------------------------------------------------- raw C ABI
def gemm_fp8_quantize(*args) -> int:
    return load().gemm_fp8_quantize(*args)


def gemm_fp8(*args) -> int:
    return load().gemm_fp8(*args)


def gemm_fp8_quantize_exp(*args) -> int:
    return load().gemm_fp8_quantize_exp(*args)


def gemm_fp8_exp(*args) -> int:
    return load().gemm_fp8_exp(*args)


def gemm_grouped(*args) -> int:
    return load().gemm_grouped(*args)


def gemm_grouped_wgrad(*args) -> int:
    return load().gemm_grouped_wgrad(*args)


# ------------------------------------------------------------------------------- arguments
def _matrix(t, name, dtypes):
    """(pointer, row stride) of a 2-D GPU tensor with unit column stride."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.dtype not in dtypes:
        raise TypeError(f"{name} must be a 2-D tensor of {_names(dtypes)}")
    rows, cols = t.shape
    ld, unit = t.stride()
    if cols > 1 and unit != 1:
        raise ValueError(f"{name} must have unit column stride (row-major)")
    if rows > 1:
        if ld < cols:
            raise ValueError(f"{name} has row stride {ld} < row length {cols}: "
                             "broadcast or overlapping rows are not supported")
    else:
        ld = cols
    if not t.is_cuda:
        raise ValueError(f"{name} must live on the GPU (the library takes device pointers)")
    return t.data_ptr(), ld if ld > 1 else 1


def _stack(t, name, dtypes):
    """(pointer, row stride, matrix stride) of a 3-D GPU tensor: one matrix per expert."""
    if not isinstance(t, torch.Tensor) or t.dim() != 3 or t.dtype not in dtypes:
        raise TypeError(f"{name} must be a 3-D tensor of {_names(dtypes)}")
    E, rows, cols = t.shape
    step, ld, unit = t.stride()
    if cols > 1 and unit != 1:
        raise ValueError(f"{name} must have unit column stride (row-major)")
    if rows > 1:
        if ld < cols:
            raise ValueError(f"{name} has row stride {ld} < row length {cols}: "
                             "broadcast or overlapping rows are not supported")
    else:
        ld = cols
    if E <= 1:
        step = 0
    elif step < 0:
        raise ValueError(f"{name} has a negative stride between experts")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on the GPU (the library takes device pointers)")
    return t.data_ptr(), ld if ld > 1 else 1, step


def _names(dtypes):
    return " or ".join(sorted(str(d).replace("torch.", "") for d in dtypes))


def _same_device(first, *others):
    for t in others:
        if t.device != first.device:
            raise ValueError(f"operands live on {first.device} and {t.device}")


def _offsets(t, like, E=None):
    """(pointer, number of experts) of the row offsets."""
    if not isinstance(t, torch.Tensor) or t.dim() != 1 or t.dtype != torch.int32 or \
            t.numel() < 1 or (t.numel() > 1 and t.stride(0) != 1):
        raise TypeError("offsets must be a contiguous 1-D int32 tensor of E + 1 elements")
    if E is not None and t.numel() != E + 1:
        raise ValueError(f"offsets has {t.numel()} elements; {E} experts need {E + 1}")
    if t.device != like.device:
        raise ValueError("offsets must live on the operands' GPU")
    return t.data_ptr(), t.numel() - 1


_nothing = contextlib.nullcontext()
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _here(t, stream):
    """Whether a call can run as it is: on the current stream, its tensors on the current GPU
    (or not on any, which the argument checks refuse)."""
    if stream is not None or not isinstance(t, torch.Tensor):
        return stream is None
    index = t.get_device()
    return index < 0 or index == _device()


def _on(stream, *tensors):
    """The context another call runs in: the first tensor's device, and `stream` where one is
    given.  The tensors' memory then waits for what runs on `stream` before it is used again, so
    that the caller may drop them at once."""
    t = tensors[0]
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        return _nothing  # the argument checks refuse it
    if stream is None:
        return torch.cuda.device(t.device)
    if stream.device != t.device:
        raise ValueError(f"stream is on {stream.device}, the operands on {t.device}")
    for u in tensors:
        if isinstance(u, torch.Tensor) and u.is_cuda:
            u.record_stream(stream)
    return torch.cuda.stream(stream)


# the current stream's handle without a torch.cuda.Stream around it (2 us less a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _current(t):
    if _raw_stream is not None:
        return _raw_stream(t.device.index)
    return torch.cuda.current_stream(t.device).cuda_stream


def _check(rc, what):
    if rc != 0:
        raise GemmError(rc, what)


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _rows16(rows, cols, device):
    """An empty rows x cols 8-bit matrix whose rows start at multiples of 16 bytes."""
    ld = (cols + 15) // 16 * 16
    q = torch.empty((rows, ld), dtype=_F8, device=device)
    return q if ld == cols else q[:, :cols]


# ---------------------------------------------------------------------------- quantization
def _block_rows(block):
    rows, cols = block
    if cols != BLOCK or rows not in (1, BLOCK):
        raise ValueError(f"block must be (1, {BLOCK}) or ({BLOCK}, {BLOCK})")
    return rows


def _quantize(x, block_rows, plain, turned):
    """(q, s, qt, st); the first two or the last two None where not asked for."""
    px, ldx = _matrix(x, "x", TYPES)
    rows, cols = x.shape
    q = s = qt = st = None
    a = [None, 0, None, 0, None, 0, None, 0]
    if plain:
        q = _rows16(rows, cols, x.device)
        s = torch.empty((rows if block_rows == 1 else _blocks(rows), _blocks(cols)),
                        dtype=torch.float32, device=x.device)
        a[0:4] = q.data_ptr(), max(q.stride(0), 1), s.data_ptr(), max(s.shape[1], 1)
    if turned:
        qt = _rows16(cols, rows, x.device)
        st = torch.empty((cols if block_rows == 1 else _blocks(cols), _blocks(rows)),
                         dtype=torch.float32, device=x.device)
        a[4:8] = qt.data_ptr(), max(qt.stride(0), 1), st.data_ptr(), max(st.shape[1], 1)
    if rows and cols:
        _check(load().gemm_fp8_quantize(rows, cols, px, ldx, TYPES[x.dtype], block_rows, *a,
                                        _current(x)), "gemm_fp8_quantize")
    return q, s, qt, st


def quantize_fp8(x, block=(1, BLOCK), stream=None):
    """(q, s): x as 8-bit floating point (e4m3fn) with one float32 scale for each block.

    x is a 2-D row-major bfloat16, float16 or float32 tensor; block is (1, 128), for
    activations and gradients, or (128, 128), for weights.  A block's scale is the smallest
    power of two (at least 2^-126) that brings its largest finite magnitude to 448 or less,
    and q the nearest 8-bit value of x / scale, ties to even.  Inf and NaN become NaN and
    leave the scale to the block's other values.  q's rows start at multiples of 16 bytes."""
    rows = _block_rows(block)
    if _here(x, stream):
        return _quantize(x, rows, True, False)[:2]
    with _on(stream, x):
        return _quantize(x, rows, True, False)[:2]


def quantize_fp8_pair(x, block=(1, BLOCK), stream=None):
    """(q, s, qt, st): `quantize_fp8` of x and of its transpose from one reading of x, for a
    training step, which contracts over both.  With (128, 128) blocks qt and st are the
    transposes of q and s; with (1, 128) ones qt has blocks of 128 rows of x of its own."""
    rows = _block_rows(block)
    if _here(x, stream):
        return _quantize(x, rows, True, True)
    with _on(stream, x):
        return _quantize(x, rows, True, True)


# -------------------------------------------------------------------------------- products
def _out_type(out_dtype):
    if out_dtype not in TYPES:
        raise TypeError(f"out_dtype must be {_names(TYPES)}")
    return TYPES[out_dtype]


def _fp8(a, sa, b, sb, out_dtype, offsets=None):
    code = _out_type(out_dtype)
    pa, lda = _matrix(a, "a", (_F8,))
    psa, ldsa = _matrix(sa, "sa", (torch.float32,))
    M, K = a.shape
    kb = _blocks(K)
    if offsets is None:
        po, E = None, 1
        pb, ldb = _matrix(b, "b", (_F8,))
        psb, ldsb = _matrix(sb, "sb", (torch.float32,))
        step_b = step_sb = 0
        N, K2 = b.shape
    else:
        pb, ldb, step_b = _stack(b, "b", (_F8,))
        psb, ldsb, step_sb = _stack(sb, "sb", (torch.float32,))
        E, N, K2 = b.shape
        po, _ = _offsets(offsets, a, E)
        if sb.shape[0] != E:
            raise ValueError(f"sb holds scales of {sb.shape[0]} experts, b {E} experts")
    _same_device(a, sa, b, sb)
    if K != K2:
        raise ValueError(f"inner dimensions differ: {tuple(a.shape)} and {tuple(b.shape)}")
    if tuple(sa.shape) != (M, kb):
        raise ValueError(f"sa must be {(M, kb)}, one scale for each row and block of {BLOCK}")
    if tuple(sb.shape[-2:]) == (_blocks(N), kb):
        b_block = BLOCK
    elif tuple(sb.shape[-2:]) == (N, kb):
        b_block = 1
    else:
        raise ValueError(f"sb must be {(_blocks(N), kb)} (blocks of {BLOCK} x {BLOCK}) or "
                         f"{(N, kb)} (blocks of 1 x {BLOCK})")
    c = torch.empty((M, N), dtype=out_dtype, device=a.device)
    if M and N:
        _check(load().gemm_fp8(M, N, K, E, po, pa, lda, psa, ldsa, pb, ldb, step_b, psb, ldsb,
                               step_sb, b_block, c.data_ptr(), N, code, _current(a)),
               "gemm_fp8")
    return c


def matmul_fp8(a, sa, b, sb, out_dtype=torch.bfloat16, stream=None):
    """(a * sa) @ (b * sb)^T: a is M x K and b N x K, both float8_e4m3fn; sa is M x
    ceil(K/128), one float32 scale for each row and block of 128 columns; sb is ceil(N/128) x
    ceil(K/128), one for each block of 128 x 128, or N x ceil(K/128), one for each row and
    block.  Sums are held in float32 and rounded once to out_dtype.  Scales are any float32
    numbers, and the product of two is formed in float32: where it overflows, so does the block's
    part of the result; where it falls below 2^-149 that part is lost."""
    if _here(a, stream):
        return _fp8(a, sa, b, sb, out_dtype)
    with _on(stream, a, sa, b, sb):
        return _fp8(a, sa, b, sb, out_dtype)


def matmul_fp8_grouped(a, sa, b, sb, offsets, out_dtype=torch.bfloat16, stream=None):
    """`matmul_fp8` with one b per expert: rows offsets[e] .. offsets[e+1] - 1 of a meet b[e]
    (E x N x K) with sb[e].  offsets is an int32 GPU tensor of E + 1 elements that do not
    decrease; rows before the first and from the last on give zeros."""
    if offsets is None:
        raise TypeError("offsets must be a contiguous 1-D int32 tensor of E + 1 elements")
    if _here(a, stream):
        return _fp8(a, sa, b, sb, out_dtype, offsets)
    with _on(stream, a, sa, b, sb, offsets):
        return _fp8(a, sa, b, sb, out_dtype, offsets)


def _grouped(x, w, offsets, transpose_w):
    px, ldx = _matrix(x, "x", TYPES)
    pw, ldw, step = _stack(w, "w", (x.dtype,))
    E = w.shape[0]
    po, _ = _offsets(offsets, x, E)
    _same_device(x, w)
    rows, K = x.shape
    K2, N = (w.shape[2], w.shape[1]) if transpose_w else (w.shape[1], w.shape[2])
    if K != K2:
        raise ValueError(f"inner dimensions differ: {tuple(x.shape)} and {tuple(w.shape)}"
                         f"{' transposed' if transpose_w else ''}")
    y = torch.empty((rows, N), dtype=x.dtype, device=x.device)
    if rows and N:
        _check(load().gemm_grouped(rows, N, K, E, po, px, ldx, pw, ldw, step,
                                   1 if transpose_w else 0, y.data_ptr(), N, TYPES[x.dtype],
                                   _current(x)), "gemm_grouped")
    return y


def matmul_grouped(x, w, offsets, transpose_w=False, stream=None):
    """y[t] = x[t] @ w[e] for the rows t of expert e, offsets[e] .. offsets[e+1] - 1: x is
    rows x K and w E x K x N (E x N x K with transpose_w), of one type, bfloat16, float16 or
    float32.  offsets as in `matmul_fp8_grouped`.  Sums are held in float32."""
    if _here(x, stream):
        return _grouped(x, w, offsets, transpose_w)
    with _on(stream, x, w, offsets):
        return _grouped(x, w, offsets, transpose_w)


def _grouped_wgrad(a, b, offsets):
    pa, lda = _matrix(a, "a", TYPES)
    pb, ldb = _matrix(b, "b", (a.dtype,))
    po, E = _offsets(offsets, a)
    _same_device(a, b)
    if a.shape[0] != b.shape[0]:
        raise ValueError(f"a has {a.shape[0]} rows, b {b.shape[0]}")
    rows, M = a.shape
    N = b.shape[1]
    dw = torch.empty((E, M, N), dtype=a.dtype, device=a.device)
    if dw.numel():
        _check(load().gemm_grouped_wgrad(rows, M, N, E, po, pa, lda, pb, ldb, dw.data_ptr(), N,
                                         M * N, TYPES[a.dtype], _current(a)),
               "gemm_grouped_wgrad")
    return dw


def matmul_grouped_wgrad(a, b, offsets, stream=None):
    """dw[e] = a_e^T @ b_e, E x M x N, over the rows of expert e: a is rows x M, b rows x N.
    An expert without rows gets zeros."""
    if _here(a, stream):
        return _grouped_wgrad(a, b, offsets)
    with _on(stream, a, b, offsets):
        return _grouped_wgrad(a, b, offsets)


# -------------------------------------------------------------------------- training steps
def _row_major(t):
    """t with unit column stride and rows that do not overlap (a copy where it is neither)."""
    ok = (t.shape[1] <= 1 or t.stride(1) == 1) and (t.shape[0] <= 1 or t.stride(0) >= t.shape[1])
    return t if ok else t.contiguous()


def _exp_half(rows, cols, device):
    """Empty 8-bit rows x cols and their exponents, one plane of rows for each block of 128
    columns, with their row strides."""
    ld, lds = (cols + 15) // 16 * 16, (rows + 15) // 16 * 16
    q = torch.empty((rows, ld), dtype=_F8, device=device)
    return q, ld, torch.empty((_blocks(cols), lds), dtype=torch.uint8, device=device), lds


def _quantize_exp(x, block_rows, plain, turned):
    """(q, s, qt, st) of a training step, scales as exponents; the rows of q and qt may be
    longer than x's (qt's: x's columns)."""
    px, ldx = _matrix(x, "x", TYPES)
    rows, cols = x.shape
    q = s = qt = st = None
    a = [None, 0, None, 0, None, 0, None, 0]
    if plain:
        q, ld, s, lds = _exp_half(rows, cols, x.device)
        a[0:4] = q.data_ptr(), max(ld, 1), s.data_ptr(), max(lds, 1)
    if turned:
        qt, ld, st, lds = _exp_half(cols, rows, x.device)
        a[4:8] = qt.data_ptr(), max(ld, 1), st.data_ptr(), max(lds, 1)
    if rows and cols and (plain or turned):
        _check(load().gemm_fp8_quantize_exp(rows, cols, px, ldx, TYPES[x.dtype], block_rows, *a,
                                            _current(x)), "gemm_fp8_quantize_exp")
    return q, s, qt, st


def _fp8_exp(a, sa, b, sb, M, N, K, dtype):
    c = torch.empty((M, N), dtype=dtype, device=a.device)
    if M and N:
        _check(load().gemm_fp8_exp(M, N, K, a.data_ptr(), max(a.shape[1], 1), sa.data_ptr(),
                                   max(sa.shape[1], 4), b.data_ptr(), max(b.shape[1], 1),
                                   sb.data_ptr(), max(sb.shape[1], 4), c.data_ptr(), N,
                                   TYPES[dtype], _current(a)), "gemm_fp8_exp")
    return c


def _once(backward):
    """torch's once_differentiable, which refuses a second derivative, without its cost (7 us) where
    no graph of the backward pass is asked for."""
    checked = torch.autograd.function.once_differentiable(backward)

    @functools.wraps(backward)
    def call(ctx, *grads):
        return (checked if torch.is_grad_enabled() else backward)(ctx, *grads)
    return call


def _no_tangents(what, *tensors):
    """Refuses dual tensors of forward-mode differentiation: they need not require a gradient, and a
    call that goes round its autograd function for such would answer without their tangents, which
    counts as a derivative of zero."""
    if getattr(forward_ad, "_current_level", 0) < 0:  # (outside of it, without asking each: 1 us)
        return
    for t in tensors:
        if t is not None and forward_ad.unpack_dual(t).tangent is not None:
            raise NotImplementedError(f"{what} has no forward-mode derivative")


class _LinearFp8(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, grads):
        need_x, need_w = (n and grads for n in ctx.needs_input_grad[:2])
        q, s, qt, st = _quantize_exp(x, 1, True, need_w)
        wq, ws, wqt, wst = _quantize_exp(w, BLOCK, True, need_x)
        ctx.save_for_backward(qt, st, wqt, wst)
        ctx.sizes = x.shape[0], w.shape[0], x.shape[1]
        return _fp8_exp(q, s, wq, ws, *ctx.sizes, x.dtype)

    @staticmethod
    @_once
    def backward(ctx, dy):
        need_x, need_w = ctx.needs_input_grad[:2]
        qt, st, wqt, wst = ctx.saved_tensors
        M, N, K = ctx.sizes
        g, sg, gt, sgt = _quantize_exp(_row_major(dy), 1, need_x, need_w)
        dx = _fp8_exp(g, sg, wqt, wst, M, K, N, dy.dtype) if need_x else None
        dw = _fp8_exp(gt, sgt, qt, st, N, K, M, dy.dtype) if need_w else None
        return dx, dw, None


def linear_fp8(x, w):
    """y = x w^T with both operands in 8 bits: x (..., K) by blocks of 1 x 128, w (N, K) by
    blocks of 128 x 128, of one type (bfloat16, float16 or float32), which y has too.

    Differentiable in both: the gradient of y is quantized by blocks of 1 x 128 along N for
    dx = dy w, with w's 8-bit values, and along the rows for dw = dy^T x, with x quantized
    along its rows; quantization itself counts as the identity.  Sums are held in float32 and
    rounded once.  As in `matmul_fp8`, blocks whose scales' product leaves float32's range are
    lost or overflow: magnitudes whose product is below about 2^-131 or above 2^143."""
    if not isinstance(x, torch.Tensor) or x.dtype not in TYPES:
        raise TypeError(f"x must be a tensor of {_names(TYPES)}")
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise TypeError("w must be a 2-D tensor of x's type")
    if x.dim() < 1 or x.shape[-1] != w.shape[1]:
        raise ValueError(f"inner dimensions differ: {tuple(x.shape)} and {tuple(w.shape)}")
    if w.dtype != x.dtype:
        raise TypeError(f"x is {x.dtype}, w {w.dtype}")
    _same_device(x, w)
    # (rows counted: -1 is ambiguous where K is 0)
    flat = _row_major(x.reshape(math.prod(x.shape[:-1]), x.shape[-1]) if x.dim() != 2 else x)
    w = _row_major(w)
    grads = torch.is_grad_enabled()  # without, no transpose is quantized for the backward pass
    if _here(x, None):
        y = _LinearFp8.apply(flat, w, grads)
    else:
        with _on(None, x):
            y = _LinearFp8.apply(flat, w, grads)
    return y if x.dim() == 2 else y.view(*x.shape[:-1], w.shape[0])


class _LinearGrouped(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, offsets, transpose_w, keep):
        need_x, need_w = ctx.needs_input_grad[:2]
        y = _grouped(x, w, offsets, transpose_w)
        q = s = None
        if keep and need_w:
            q, s = _quantize(x, 1, True, False)[:2]
        ctx.save_for_backward(x if need_w and not keep else None, q, s, w if need_x else None,
                              offsets)
        ctx.transpose_w = transpose_w
        return y

    @staticmethod
    @_once
    def backward(ctx, dy):
        need_x, need_w = ctx.needs_input_grad[:2]
        x, q, s, w, offsets = ctx.saved_tensors
        dy = _row_major(dy)
        dx = _grouped(dy, w, offsets, not ctx.transpose_w) if need_x else None
        dw = None
        if need_w:
            if x is None:
                from .experts import _dequantize
                x = _dequantize(q, s, dy.dtype)
            dw = _grouped_wgrad(dy, x, offsets) if ctx.transpose_w else \
                _grouped_wgrad(x, dy, offsets)
        return dx, dw, None, None, None


def linear_grouped(x, w, offsets, transpose_w=False, checkpoint=False):
    """`matmul_grouped`, differentiable in x and w.  Rows of no expert get zeros in dx, and
    experts without rows zeros in dw.

    With checkpoint, w's gradient is that of the 8-bit values that `quantize_fp8` has of x's rows,
    by blocks of 1 x 128, and x itself need not be kept for it: 8 bits a value and a scale for every
    128.  y and dx do not change; Inf in x, which has no 8-bit value, gives NaN in dw."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or x.dtype not in TYPES:
        raise TypeError(f"x must be a 2-D tensor of {_names(TYPES)}")
    x, transpose_w, keep = _row_major(x), bool(transpose_w), bool(checkpoint)
    keep = keep and torch.is_grad_enabled()  # without, nothing is kept
    if _here(x, None):
        return _LinearGrouped.apply(x, w, offsets, transpose_w, keep)
    with _on(None, x):
        return _LinearGrouped.apply(x, w, offsets, transpose_w, keep)
