"""What a layer of experts needs around its products, on GPU tensors, through the C ABI of
include/gemm_experts.h: a router with its balance loss, rows by expert, adapters of low rank for
many requests at once, gated units whose input is kept in 8 bits, and 8-bit values as numbers.

As in `lowp`, this module only checks arguments, allocates outputs and workspaces and passes
pointers, strides and the stream; every value is computed in the library's HIP kernels, and there is
no other path.  Calls are asynchronous and run on the current stream, or on `stream` where there is
one, under `lowp`'s rules.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _binding
from .lowp import (BLOCK, TYPES, _F8, _blocks, _check, _current, _here, _matrix, _names, _no_tangents,
                   _offsets, _on, _once, _out_type, _row_major, _rows16, _same_device)

MAX_EXPERTS = 1024         # of a router; GEMM_ROUTE_MAX_EXPERTS
MAX_CHOSEN = 16            # GEMM_ROUTE_MAX_CHOSEN
MAX_GROUPS = 4096          # of group_rows; GEMM_GROUP_MAX_EXPERTS
MAX_RANK = 128             # GEMM_ADAPTERS_MAX_RANK
# Rows from which on u's partial sums are joined by a launch of their own (3 us) rather than by each
# of its readers.
JOINED_ROWS = 1024

_i64, _int, _vp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
# Every exported symbol and its C signature (kept in step with include/gemm_experts.h).
SIGNATURES = {
    "gemm_route": (_int, [_i64, _i64, _i64, _vp, _i64, _int, _vp, _int, _vp, _vp, _vp, _vp, _vp,
                          _vp, _i64, _vp]),
    "gemm_route_workspace": (_i64, [_i64, _i64]),
    "gemm_route_grad": (_int, [_i64, _i64, _i64, _vp, _i64, _int, _vp, _int, _vp, _vp, _vp, _vp,
                               _vp, _vp, _vp, _i64, _vp]),
    "gemm_group_rows": (_int, [_i64, _i64, _vp, _int, _vp, _vp, _vp, _vp, _i64, _vp]),
    "gemm_group_rows_workspace": (_i64, [_i64, _i64]),
    "gemm_adapters_down": (_int, [_i64, _i64, _i64, _i64, _vp, _vp, _vp, _i64, _vp, _i64, _i64,
                                  _vp, _vp, _int, _int, _int, _vp]),
    "gemm_adapters_up": (_int, [_i64, _i64, _i64, _i64, _vp, _vp, _vp, _int, _vp, _i64, _i64, _vp,
                                _i64, _vp, _i64, _int, _vp]),
    "gemm_adapters_grad": (_int, [_i64, _i64, _i64, _vp, _vp] +
                           2 * [_i64, _vp, _int, _vp, _i64, _vp, _i64, _i64] +
                           [_vp, _i64, _int, _vp]),
    "gemm_adapters_splits": (_int, [_i64, _i64, _i64, _i64]),
    "gemm_adapters_grad_workspace": (_i64, [_i64, _i64, _i64, _i64, _i64, _int]),
    "gemm_gated": (_int, [_i64, _i64, _vp, _i64, _int, _vp, _i64, _vp, _i64, _vp, _i64, _vp]),
    "gemm_gated_grad": (_int, [_i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64,
                               _int, _vp]),
    "gemm_fp8_dequantize": (_int, [_i64, _i64, _vp, _i64, _vp, _i64, _int, _vp, _i64, _int, _vp]),
}
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
def gemm_route(*args) -> int:
    return load().gemm_route(*args)


def gemm_route_workspace(rows, E) -> int:
    return load().gemm_route_workspace(rows, E)


def gemm_route_grad(*args) -> int:
    return load().gemm_route_grad(*args)


def gemm_group_rows(*args) -> int:
    return load().gemm_group_rows(*args)


def gemm_group_rows_workspace(n, E) -> int:
    return load().gemm_group_rows_workspace(n, E)


def gemm_adapters_down(*args) -> int:
    return load().gemm_adapters_down(*args)


def gemm_adapters_up(*args) -> int:
    return load().gemm_adapters_up(*args)


def gemm_adapters_grad(*args) -> int:
    return load().gemm_adapters_grad(*args)


def gemm_adapters_splits(rows, K, rank, E) -> int:
    return load().gemm_adapters_splits(rows, K, rank, E)


def gemm_adapters_grad_workspace(rows, K, N, rank, E, type_code) -> int:
    return load().gemm_adapters_grad_workspace(rows, K, N, rank, E, type_code)


def gemm_gated(*args) -> int:
    return load().gemm_gated(*args)


def gemm_gated_grad(*args) -> int:
    return load().gemm_gated_grad(*args)


def gemm_fp8_dequantize(*args) -> int:
    return load().gemm_fp8_dequantize(*args)


# ------------------------------------------------------------------------------- arguments
def _size(n, what):
    """A workspace query's answer, or its error raised."""
    if n < 0:
        _check(n, what)
    return n


def _workspace(n, device):
    """(tensor that holds it, pointer): n bytes, none for 0."""
    if n == 0:
        return None, None
    w = torch.empty((n + 7) // 8, dtype=torch.int64, device=device)
    return w, w.data_ptr()


def _flat(x):
    """x as rows of its last axis (rows counted: -1 is ambiguous where the last axis is empty)."""
    return x if x.dim() == 2 else x.reshape(math.prod(x.shape[:-1]), x.shape[-1])


def _pointer(t):
    return None if t is None else t.data_ptr()


# ---------------------------------------------------------------------------------- router
def _route(logits, k, valid, renormalize):
    """(gates, experts, counts, sums, loss)."""
    px, ldx = _matrix(logits, "logits", TYPES)
    rows, E = logits.shape
    if not 1 <= E <= MAX_EXPERTS:
        raise ValueError(f"logits must have 1 to {MAX_EXPERTS} columns, one for each expert")
    if not 1 <= k <= min(E, MAX_CHOSEN):
        raise ValueError(f"k must be 1 to {min(E, MAX_CHOSEN)} for {E} experts")
    if valid is not None:
        if valid.device != logits.device:
            raise ValueError("valid must live on the logits' GPU")
    dev = logits.device
    gates = torch.empty((rows, k), dtype=torch.float32, device=dev)
    experts = torch.empty((rows, k), dtype=torch.int32, device=dev)
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    sums = torch.empty(2, dtype=torch.int32, device=dev)
    loss = torch.empty((), dtype=torch.float32, device=dev)
    need = _size(load().gemm_route_workspace(rows, E), "gemm_route_workspace")
    hold, pw = _workspace(need, dev)
    _check(load().gemm_route(rows, E, k, px, max(ldx, E), TYPES[logits.dtype], _pointer(valid),
                             1 if renormalize else 0, gates.data_ptr(), experts.data_ptr(),
                             counts.data_ptr(), sums.data_ptr(), loss.data_ptr(), pw, need,
                             _current(logits)), "gemm_route")
    return gates, experts, counts, sums, loss


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, valid, renormalize):
        gates, experts, counts, sums, loss = _route(logits, k, valid, renormalize)
        ctx.save_for_backward(logits, valid, gates, experts, counts, sums)
        ctx.k, ctx.renormalize = k, 1 if renormalize else 0
        ctx.mark_non_differentiable(experts, counts)
        ctx.set_materialize_grads(False)
        return gates, experts, counts, loss

    @staticmethod
    @_once
    def backward(ctx, dgates, dexperts, dcounts, dloss):
        logits, valid, gates, experts, counts, sums = ctx.saved_tensors
        rows, E = logits.shape
        dgates = None if dgates is None else dgates.contiguous()
        dx = logits.new_empty((rows, E))
        _check(load().gemm_route_grad(
            rows, E, ctx.k, logits.data_ptr(), max(logits.stride(0), E), TYPES[logits.dtype],
            _pointer(valid), ctx.renormalize, gates.data_ptr(), experts.data_ptr(),
            counts.data_ptr(), sums.data_ptr(), _pointer(dgates), _pointer(dloss), dx.data_ptr(), E,
            _current(logits)), "gemm_route_grad")
        return dx, None, None, None


def route_experts(logits, k, valid=None, renormalize=False):
    """(gates, experts, counts, loss): the k experts of every row, and how evenly they are used.

    logits is T x E (bfloat16, float16 or float32; E up to 1024, k up to 16), valid T truth values,
    False for rows to be left out (padding), or None.  With p the softmax of a row,
      experts  T x k int32, the largest logits first, of equal ones the lowest index
      gates    T x k float32, their p, with renormalize over the sum of the row's
      counts   E int32, how often each expert was taken
      loss     float32: E sum_e f_e P_e, f_e the share of counts that is e's, P_e the mean of p_e
               over the rows that count; 1 where all experts are used alike, E where one is, and 0
               where no row counts
    An expert whose logit is -Inf is never taken.  Where a row has none left, its place holds -1
    with a gate of 0 (`group_rows` puts such places last); rows that are not valid, or have no
    logit above -Inf, hold nothing else and do not count.  NaN is taken before every number; it, or
    +Inf, makes the row's gates and the loss NaN.  Probabilities below 2^-126 may count as 0.

    Differentiable (once, backward) in logits through gates and loss; counts are constants in it, as
    usual."""
    if valid is not None:
        if not isinstance(valid, torch.Tensor) or valid.dtype != torch.bool or valid.dim() != 1:
            raise TypeError("valid must be a 1-D bool tensor")
        if not isinstance(logits, torch.Tensor) or logits.dim() != 2 or \
                valid.shape[0] != logits.shape[0]:
            raise ValueError("valid must have one value for each row of logits")
        valid = valid.contiguous()
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2 or logits.dtype not in TYPES:
        raise TypeError(f"logits must be a 2-D tensor of {_names(TYPES)}")
    _no_tangents("route_experts", logits)
    logits, k = _row_major(logits), int(k)
    if not (logits.requires_grad and torch.is_grad_enabled()):
        if _here(logits, None):
            gates, experts, counts, _, loss = _route(logits, k, valid, renormalize)
        else:
            with _on(None, logits):
                gates, experts, counts, _, loss = _route(logits, k, valid, renormalize)
        return gates, experts, counts, loss
    if _here(logits, None):
        return _Route.apply(logits, k, valid, renormalize)
    with _on(None, logits):
        return _Route.apply(logits, k, valid, renormalize)


# --------------------------------------------------------------------------------- grouping
def _group(experts, count):
    ids = experts.contiguous()
    n, dev = ids.numel(), ids.device
    order = torch.empty(n, dtype=torch.int64, device=dev)
    place = torch.empty(experts.shape, dtype=torch.int64, device=dev)
    offsets = torch.empty(count + 1, dtype=torch.int32, device=dev)
    need = _size(load().gemm_group_rows_workspace(n, count), "gemm_group_rows_workspace")
    hold, pw = _workspace(need, dev)
    _check(load().gemm_group_rows(n, count, ids.data_ptr(), ids.element_size(), order.data_ptr(),
                                  place.data_ptr(), offsets.data_ptr(), pw, need, _current(ids)),
           "gemm_group_rows")
    return order, place, offsets


def group_rows(experts, count, stream=None):
    """(order, place, offsets): rows sorted by expert, as the grouped products and `add_adapters`
    take them.  experts is an int32 or int64 GPU tensor of any shape, its n elements counted in
    row-major order; those outside 0 .. count - 1 belong to no expert and come last.

    order (n int64) holds the element at each place, equal experts in the order of the elements;
    place (int64, experts' shape) the place of each element; offsets (count + 1 int32) each
    expert's first place, and that of the elements of none.  For k experts a row, as `route_experts`
    gives them, order // k is the row at a place.  count is 4096 at most."""
    if not isinstance(experts, torch.Tensor) or experts.dtype not in (torch.int32, torch.int64):
        raise TypeError("experts must be an int32 or int64 tensor")
    count = int(count)
    if not 0 <= count <= MAX_GROUPS:
        raise ValueError(f"count must be 0 to {MAX_GROUPS}")
    if not experts.is_cuda:
        raise ValueError("experts must live on the GPU (the library takes device pointers)")
    if _here(experts, stream):
        return _group(experts, count)
    with _on(stream, experts):
        return _group(experts, count)


# --------------------------------------------------------------------------------- adapters
# (operands that `add_adapters` has checked: row-major with unit column stride)
def _ld(t):
    """The row stride of a 2-D tensor (of a stack: of its matrices); of one row, any will do."""
    return max(t.stride(-2), t.shape[-1], 1)


def _down(x, a, order, offsets, scale):
    """(u, splits): the contraction of x's rows with their adapter's, by place, as so many partial
    sums."""
    rows, K = x.shape
    E, rank = a.shape[:2]
    lib = load()
    splits = lib.gemm_adapters_splits(rows, K, rank, E)
    if splits < 0:
        _check(splits, "gemm_adapters_splits")
    # (whole fragments of 16, the columns past the rank zeros)
    u = torch.empty((splits, rows, (rank + 15) // 16 * 16), dtype=torch.float32, device=x.device)
    join = rows >= JOINED_ROWS
    _check(lib.gemm_adapters_down(rows, K, rank, E, order.data_ptr(), offsets.data_ptr(),
                                  x.data_ptr(), _ld(x), a.data_ptr(), _ld(a), a.stride(0),
                                  _pointer(scale), u.data_ptr(), splits, 1 if join else 0,
                                  TYPES[x.dtype], _current(x)), "gemm_adapters_down")
    return u, 1 if join else splits


def _up(u, splits, b, y, order, offsets):
    """y + u b of each row's adapter; y None for 0."""
    E, rank, N = b.shape
    rows = u.shape[1]
    out = b.new_empty((rows, N))
    py, ldy = (None, 0) if y is None else (y.data_ptr(), _ld(y))
    _check(load().gemm_adapters_up(rows, N, rank, E, order.data_ptr(), offsets.data_ptr(),
                                   u.data_ptr(), splits, b.data_ptr(), _ld(b), b.stride(0), py,
                                   ldy, out.data_ptr(), max(N, 1), TYPES[b.dtype], _current(b)),
           "gemm_adapters_up")
    return out


_NO_SIDE = 0, None, 1, None, 0, None, 0, 0


def _adapter_grads(shape, order, offsets, *sides):
    """E x rank x width: u^T x over each adapter's rows, for each (u, splits, x) of two sides; None
    for a side that is None."""
    E, rank = shape
    lib, like = load(), next(s[2] for s in sides if s is not None)
    rows, code = like.shape[0], TYPES[like.dtype]
    grads, args, widths = [], [], []
    for s in sides:
        if s is None:
            grads.append(None)
            args += _NO_SIDE
            widths.append(0)
            continue
        u, splits, x = s
        width = x.shape[1]
        d = x.new_empty((E, rank, width))
        grads.append(d)
        args += (width, u.data_ptr(), splits, x.data_ptr(), _ld(x), d.data_ptr(), max(width, 1),
                 rank * width)
        widths.append(width)
    need = _size(lib.gemm_adapters_grad_workspace(rows, *widths, rank, E, code),
                 "gemm_adapters_grad_workspace")
    hold, pw = _workspace(need, like.device)
    _check(lib.gemm_adapters_grad(rows, rank, E, order.data_ptr(), offsets.data_ptr(), *args, pw,
                                  need, code, _current(like)), "gemm_adapters_grad")
    return grads


class _Adapters(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, x, a, b, order, offsets, scale):
        u, ctx.splits = _down(x, a, order, offsets, scale)
        need_y, need_x, need_a, need_b = ctx.needs_input_grad[:4]
        ctx.save_for_backward(x if need_a else None, a if need_x else None,
                              b if need_x or need_a else None, u if need_b else None, order,
                              offsets, scale)
        ctx.size = a.shape[:2]
        return _up(u, ctx.splits, b, y, order, offsets)

    @staticmethod
    @_once
    def backward(ctx, dout):
        need_y, need_x, need_a, need_b = ctx.needs_input_grad[:4]
        x, a, b, u, order, offsets, scale = ctx.saved_tensors
        dx = da = db = None
        rows = _row_major(dout)
        if need_x or need_a:
            v, splits = _down(rows, b, order, offsets, scale)
            dx = _up(v, splits, a, None, order, offsets) if need_x else None
        if need_a or need_b:
            da, db = _adapter_grads(ctx.size, order, offsets, (v, splits, x) if need_a else None,
                                    (u, ctx.splits, rows) if need_b else None)
        return dout if need_y else None, dx, da, db, None, None, None


def add_adapters(y, x, a, b, order, offsets, scale=None):
    """y + scale[e] (x a[e]^T) b[e] for the rows of each adapter e: adapters of low rank beside a
    projection that all rows share, whose result y is and which x went into.

    x is (..., K) and y (..., N), with T rows each; a is E x rank x K and b E x rank x N (both with
    the wide axis contiguous, so that the forward and the backward pass read whole lines), rank up
    to 128; all of one type, bfloat16, float16 or float32.  order (T int64) and offsets (E + 1
    int32) are `group_rows` of the rows' adapters, made once for all projections of a batch: order
    holds every row once.  scale is E float32 on the GPU, or None for 1.  Rows of no adapter keep y.
    The contraction over K is kept in float32 (in bfloat16 without its bits below 2^-133); all sums
    are, and are rounded once.  Inf and NaN stay in their rows and adapters (in bfloat16 Inf in b, and
    for the gradients in x, a or the incoming one, may come out as NaN).

    Differentiable (once, backward) in y, x, a and b; adapters without rows get zeros."""
    if not isinstance(x, torch.Tensor) or x.dim() < 1 or x.dtype not in TYPES:
        raise TypeError(f"x must be a tensor of {_names(TYPES)}")
    if not isinstance(y, torch.Tensor) or y.dim() < 1 or y.dtype != x.dtype:
        raise TypeError("y must be a tensor of x's type")
    for name, t in (("a", a), ("b", b)):
        if not isinstance(t, torch.Tensor) or t.dim() != 3 or t.dtype != x.dtype:
            raise TypeError(f"{name} must be a 3-D tensor of x's type")
    E, rank, K = a.shape
    N = b.shape[2]
    if tuple(b.shape[:2]) != (E, rank):
        raise ValueError(f"a is {tuple(a.shape)}, b {tuple(b.shape)}: experts or ranks differ")
    if not 1 <= rank <= MAX_RANK:
        raise ValueError(f"the rank must be 1 to {MAX_RANK}")
    if x.shape[-1] != K or y.shape[-1] != N or x.shape[:-1] != y.shape[:-1]:
        raise ValueError(f"x is {tuple(x.shape)}, y {tuple(y.shape)}: the adapters take (..., {K}) "
                         f"to (..., {N})")
    _same_device(x, y, a, b)
    if scale is not None:
        if not isinstance(scale, torch.Tensor) or scale.dtype != torch.float32 or \
                scale.dim() != 1 or (E > 1 and scale.stride(0) != 1):
            raise TypeError("scale must be a contiguous 1-D float32 tensor")
        if scale.shape[0] != E:
            raise ValueError(f"scale has {scale.shape[0]} elements for {E} adapters")
        _same_device(x, scale)
        if scale.requires_grad and torch.is_grad_enabled():
            raise ValueError("scale has no gradient here: detach it")
    _no_tangents("add_adapters", y, x, a, b, scale)
    if not x.is_cuda:
        raise ValueError("x must live on the GPU (the library takes device pointers)")
    rows, base = _row_major(_flat(x)), _row_major(_flat(y))
    if not isinstance(order, torch.Tensor) or order.dim() != 1 or order.dtype != torch.int64 or \
            (order.numel() > 1 and order.stride(0) != 1):
        raise TypeError("order must be a contiguous 1-D int64 tensor")
    if order.shape[0] != rows.shape[0]:
        raise ValueError(f"order has {order.shape[0]} elements for {rows.shape[0]} rows")
    _same_device(x, order)
    _offsets(offsets, x, E)
    args = base, rows, _unit_columns(a), _unit_columns(b), order, offsets, scale
    if _here(x, None):
        out = _adapted(*args)
    else:
        with _on(None, x):
            out = _adapted(*args)
    return out if y.dim() == 2 else out.view(y.shape)


def _adapted(y, x, a, b, order, offsets, scale):
    if torch.is_grad_enabled() and (y.requires_grad or x.requires_grad or a.requires_grad or
                                    b.requires_grad):
        return _Adapters.apply(y, x, a, b, order, offsets, scale)
    return _up(*_down(x, a, order, offsets, scale), b, y, order, offsets)


def _unit_columns(w):
    """w with unit column stride and rows that do not overlap (a copy where it is neither)."""
    ok = (w.shape[2] <= 1 or w.stride(2) == 1) and (w.shape[1] <= 1 or w.stride(1) >= w.shape[2])
    return w if ok else w.contiguous()


# ------------------------------------------------------------------------------- gated unit
def _gated(x, keep):
    """(h, q, s) of row-major x: q and s None where nothing is kept."""
    rows, cols = x.shape
    N = cols // 2
    h = x.new_empty((rows, N))
    q = s = pq = ps = None
    ldq = lds = 0
    if keep:
        q = _rows16(rows, cols, x.device)
        s = torch.empty((rows, 2 * _blocks(N)), dtype=torch.float32, device=x.device)
        pq, ldq, ps, lds = q.data_ptr(), q.stride(0), s.data_ptr(), s.shape[1]
    if rows and N:
        rc = load().gemm_gated(rows, N, x.data_ptr(), max(x.stride(0), cols), TYPES[x.dtype],
                               h.data_ptr(), N, pq, ldq, ps, lds, _current(x))
        if rc:
            _check(rc, "gemm_gated")
    return h, q, s


class _Gated(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, keep):
        h, q, s = _gated(x, keep)
        if keep:
            ctx.save_for_backward(q, s)
        else:
            ctx.save_for_backward(x)
        return h

    @staticmethod
    @_once
    def backward(ctx, dh):
        if not dh.is_contiguous():
            dh = _row_major(dh)
        rows, N = dh.shape
        dx = dh.new_empty((rows, 2 * N))
        if rows and N:
            kept = ctx.saved_tensors
            if len(kept) == 2:
                q, s = kept
                kept = None, 0, q.data_ptr(), q.stride(0), s.data_ptr(), s.shape[1]
            else:
                x, = kept
                kept = x.data_ptr(), max(x.stride(0), 2 * N), None, 0, None, 0
            rc = load().gemm_gated_grad(rows, N, *kept, dh.data_ptr(), max(dh.stride(0), N),
                                        dx.data_ptr(), 2 * N, TYPES[dh.dtype], _current(dh))
            if rc:
                _check(rc, "gemm_gated_grad")
        return dx, None


def gated_silu(x, checkpoint=False):
    """silu(gate) * up, silu(g) = g / (1 + exp(-g)): gate is the first half of x's last axis, up the
    second (the two results of one product with twice the columns), of bfloat16, float16 or
    float32; sums and functions in float32, rounded once.

    Differentiable (once, backward).  With checkpoint the backward pass works on the 8-bit values that `quantize_fp8`
    has of gate and of up, by blocks of 1 x 128 each, and x itself need not be kept: 8 bits a value
    and a scale for every 128, and a gradient of these values (of the type's largest number where x's
    own rounds to more, NaN where x is Inf, which has no 8-bit value); the forward result is x's own."""
    if not isinstance(x, torch.Tensor) or x.dim() < 1 or x.dtype not in TYPES:
        raise TypeError(f"x must be a tensor of {_names(TYPES)}")
    if x.shape[-1] % 2:
        raise ValueError(f"x has {x.shape[-1]} columns: gate and up need as many each")
    _no_tangents("gated_silu", x)
    if not x.is_cuda:
        raise ValueError("x must live on the GPU (the library takes device pointers)")
    flat = x if x.dim() == 2 and x.is_contiguous() else _row_major(_flat(x))
    if x.requires_grad and torch.is_grad_enabled():
        if _here(x, None):
            h = _Gated.apply(flat, bool(checkpoint))
        else:
            with _on(None, x):
                h = _Gated.apply(flat, bool(checkpoint))
    elif _here(x, None):
        h = _gated(flat, False)[0]
    else:
        with _on(None, x):
            h = _gated(flat, False)[0]
    return h if x.dim() == 2 else h.view(*x.shape[:-1], x.shape[-1] // 2)


# --------------------------------------------------------------------------- 8-bit values
def _dequantize(q, s, out_dtype):
    code = _out_type(out_dtype)
    pq, ldq = _matrix(q, "q", (_F8,))
    ps, lds = _matrix(s, "s", (torch.float32,))
    rows, cols = q.shape
    _same_device(q, s)
    if tuple(s.shape) == (rows, _blocks(cols)):
        block = 1
    elif tuple(s.shape) == (_blocks(rows), _blocks(cols)):
        block = BLOCK
    else:
        raise ValueError(f"s must be {(rows, _blocks(cols))} (blocks of 1 x {BLOCK}) or "
                         f"{(_blocks(rows), _blocks(cols))} (blocks of {BLOCK} x {BLOCK})")
    y = torch.empty((rows, cols), dtype=out_dtype, device=q.device)
    if rows and cols:
        _check(load().gemm_fp8_dequantize(rows, cols, pq, ldq, ps, lds, block, y.data_ptr(), cols,
                                          code, _current(q)), "gemm_fp8_dequantize")
    return y


def dequantize_fp8(q, s, out_dtype=torch.bfloat16, stream=None):
    """The numbers q * s that `quantize_fp8`'s results stand for, in out_dtype: q is 2-D
    float8_e4m3fn, s float32 with one scale for each block of 1 x 128 or of 128 x 128.  s may be any
    numbers: the product is formed in float32, which rounds it unless s is a power of two, as
    `quantize_fp8`'s are, and then rounded to out_dtype.  Finite products past out_dtype's range become
    its largest number."""
    if _here(q, stream):
        return _dequantize(q, s, out_dtype)
    with _on(stream, q, s):
        return _dequantize(q, s, out_dtype)
