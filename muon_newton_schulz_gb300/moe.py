"""Tokens sorted by expert, and back with their weights, and the gradients.

The matrices the Muon step updates are mostly experts (TorchTitan section 2.1:
top-2 routing, capacity factor 1.25).  ``sort_tokens`` turns the router's
choices into a ``Route``; ``dispatch`` lays the tokens out expert by expert;
``combine`` sums the experts' answers back with the router's weights.  Both
take part in autograd.  Everything runs in the library's kernels, on the
current stream; no call waits on the host.
"""
from __future__ import annotations

from functools import lru_cache

import torch

from . import binding as B

_DTYPES = {torch.float32: B.MUON_F32, torch.bfloat16: B.MUON_BF16}


class Route:
    """Where each token's choices stand among the sorted rows.

    ``row`` (tokens x topk, int32): the row of each choice, -1 for a dropped
    one.  ``offsets`` (experts + 1, int32): each expert's first row, and the
    end.  ``counts`` (experts, int32): each expert's rows that hold a token.
    ``capacity``: rows of every expert, or 0 where nothing is dropped and each
    expert's first row is a multiple of ``align``.  ``rows``: rows of a buffer
    of sorted tokens, known on the host."""

    __slots__ = ("row", "offsets", "counts", "capacity", "align", "shape", "rows")

    def __init__(self, row, offsets, counts, capacity=0, align=1):
        if row.dim() != 2 or counts.dim() != 1 or offsets.dim() != 1 or offsets.numel() != counts.numel() + 1:
            raise ValueError("row must be tokens x topk, counts of length experts and offsets of length experts + 1")
        for t in (row, offsets, counts):
            if t.dtype != torch.int32 or not t.is_contiguous():
                raise ValueError("row, offsets and counts must be contiguous int32 tensors")
            if t.device.type != "cuda" or t.device != row.device:
                raise ValueError("row, offsets and counts must be on one CUDA device")
        self._fill(row, offsets, counts, capacity, align,
                   *_sizes(row.shape[0], row.shape[1], counts.numel(), capacity, align)[:2])

    def _fill(self, row, offsets, counts, capacity, align, shape, rows):
        self.row, self.offsets, self.counts, self.capacity, self.align = row, offsets, counts, capacity, align
        self.shape, self.rows = shape, rows
        return self

    @property
    def experts(self) -> int:
        return self.counts.numel()


@lru_cache(maxsize=256)
def _sizes(tokens, topk, experts, capacity, align):
    """The shape struct, the rows of the sorted buffer and the sort's workspace bytes."""
    shape = B.muon_moe_shape(tokens, topk, experts, capacity, align)
    st, rows = B.muon_moe_rows(shape)
    if st != B.MUON_OK:
        raise B.MuonError(st, f"tokens={tokens}, topk={topk}, experts={experts}, capacity={capacity}, align={align}")
    return shape, rows, B.muon_moe_sort_workspace_size(shape)[1]


def _check(st, h):
    if st != B.MUON_OK:
        raise B.MuonError(st, B.muon_last_error_message(h))


def _matrix(t, name, rows, device):
    """A matrix argument with unit column stride, copied only when it has another."""
    if t.dim() != 2 or t.shape[0] != rows:
        raise ValueError(f"{name} must have {rows} rows, got shape {tuple(t.shape)}")
    if t.dtype not in _DTYPES:
        raise ValueError(f"{name} must be bf16 or fp32, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the route on {device}")
    if t.shape[1] > 1 and t.stride(1) != 1 or t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        t = t.contiguous()
    return t


def _ld(t):
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def _weights(w, route):
    if w.shape != route.row.shape:
        raise ValueError(f"weights must have shape {tuple(route.row.shape)}, got {tuple(w.shape)}")
    if w.dtype not in _DTYPES:
        raise ValueError(f"weights must be bf16 or fp32, got {w.dtype}")
    if w.device != route.row.device:
        raise ValueError(f"weights are on {w.device}, the route on {route.row.device}")
    return w.contiguous()


def sort_tokens(expert_ids, experts: int, capacity: int = 0, align: int = 1) -> Route:
    """The route of ``expert_ids`` (tokens x topk, int32 or int64), stable in
    the order of tokens and choices.  With ``capacity`` every expert has that
    many rows and the choices beyond it are dropped; without, none is dropped
    and each expert starts at a multiple of ``align``.  A choice outside
    [0, experts), -1 for a padding token for instance, is dropped."""
    if expert_ids.dim() != 2:
        raise ValueError(f"expert_ids must be tokens x topk, got shape {tuple(expert_ids.shape)}")
    if expert_ids.dtype not in (torch.int32, torch.int64):
        raise ValueError(f"expert_ids must be int32 or int64, got {expert_ids.dtype}")
    device, index = expert_ids.device, expert_ids.get_device()
    if index < 0:
        raise ValueError(f"expert_ids must be a CUDA tensor, got one on {device}")
    ids = expert_ids.contiguous()
    tokens, topk = ids.shape
    shape, rows, need = _sizes(tokens, topk, experts, capacity, align)
    row = torch.empty((tokens, topk), dtype=torch.int32, device=device)
    ends = torch.empty(2 * experts + 1, dtype=torch.int32, device=device)
    ws = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    h, at = B.thread_handle(index), ends.data_ptr()
    _check(B.muon_moe_sort(h, shape, ids.data_ptr(), 64 if ids.dtype == torch.int64 else 32, row.data_ptr(), at,
                           at + 4 * (experts + 1), ws.data_ptr() if need else None, need, B.current_stream(index)), h)
    return Route.__new__(Route)._fill(row, ends[:experts + 1], ends[experts + 1:], capacity, align, shape, rows)


def _dispatch(x, route):
    device, index = route.row.device, route.row.get_device()
    x = _matrix(x, "x", route.row.shape[0], device)
    hidden = x.shape[1]
    xs = torch.empty(route.rows, hidden, dtype=x.dtype, device=device)
    h = B.thread_handle(index)
    _check(B.muon_moe_dispatch(h, route.shape, route.row.data_ptr(), route.offsets.data_ptr(),
                               route.counts.data_ptr(), x.data_ptr(), _ld(x), xs.data_ptr(), max(hidden, 1), hidden,
                               _DTYPES[x.dtype], B.current_stream(index)), h)
    return xs


def _combine(y, weights, route):
    device, index = route.row.device, route.row.get_device()
    y = _matrix(y, "y", route.rows, device)
    hidden = y.shape[1]
    out = torch.empty(route.row.shape[0], hidden, dtype=y.dtype, device=device)
    w = _weights(weights, route) if weights is not None else None
    h = B.thread_handle(index)
    _check(B.muon_moe_combine(h, route.shape, route.row.data_ptr(), y.data_ptr(), _ld(y),
                              w.data_ptr() if w is not None else None, _DTYPES[w.dtype] if w is not None else 0,
                              out.data_ptr(), max(hidden, 1), hidden, _DTYPES[y.dtype],
                              B.current_stream(index)), h)
    return out


def combine_backward(dout, y, weights, route: Route):
    """(dy, dweights) of ``combine`` for the gradient ``dout`` of its result."""
    device, index = route.row.device, route.row.get_device()
    dout = _matrix(dout, "dout", route.row.shape[0], device)
    y = _matrix(y, "y", route.rows, device)
    if dout.shape[1] != y.shape[1] or dout.dtype != y.dtype:
        raise ValueError(f"dout and y must have one row length and type, got {tuple(dout.shape)} {dout.dtype} and "
                         f"{tuple(y.shape)} {y.dtype}")
    w = _weights(weights, route)
    hidden = y.shape[1]
    dy = torch.empty(route.rows, hidden, dtype=y.dtype, device=device)
    dw = torch.empty_like(w)
    h = B.thread_handle(index)
    _check(B.muon_moe_combine_backward(h, route.shape, route.row.data_ptr(), route.offsets.data_ptr(),
                                       route.counts.data_ptr(), dout.data_ptr(), _ld(dout), y.data_ptr(), _ld(y),
                                       w.data_ptr(), _DTYPES[w.dtype], dy.data_ptr(), max(hidden, 1), dw.data_ptr(),
                                       hidden, _DTYPES[y.dtype], B.current_stream(index)), h)
    return dy, dw


def dispatch_backward(dxs, route: Route):
    """dx of ``dispatch`` for the gradient ``dxs`` of its result: a token's
    gradient is the sum over its rows, that is ``combine`` without weights."""
    return _combine(dxs, None, route)


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, route):
        ctx.route = route
        return _dispatch(x, route)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dxs):
        return dispatch_backward(dxs, ctx.route), None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, weights, route):
        ctx.route = route
        ctx.save_for_backward(*(() if weights is None else (y, weights)))
        return _combine(y, weights, route)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        if not ctx.saved_tensors:   # weights of 1: the gradient lays dout out by expert
            return _dispatch(dout, ctx.route), None, None
        y, weights = ctx.saved_tensors
        dy, dw = combine_backward(dout, y, weights, ctx.route)
        return dy, dw, None


def dispatch(x, route: Route):
    """The sorted rows (route.rows x hidden) of ``x`` (tokens x hidden, fp32 or
    bf16): each token's row at the place of each of its choices, zero in rows
    without a token."""
    if torch.is_grad_enabled() and x.requires_grad:
        return _Dispatch.apply(x, route)
    return _dispatch(x, route)


def combine(y, weights, route: Route):
    """out[t] = sum over k of weights[t, k] * y[row[t, k]] for sorted rows ``y``
    (fp32 or bf16) and ``weights`` (tokens x topk, fp32 or bf16; None for 1),
    summed in fp32.  Dropped choices are left out."""
    if torch.is_grad_enabled() and (y.requires_grad or (weights is not None and weights.requires_grad)):
        return _Combine.apply(y, weights, route)
    return _combine(y, weights, route)
