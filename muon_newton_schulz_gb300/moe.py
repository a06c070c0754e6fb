"""Tokens sorted by expert, and back with their weights, and the gradients.

The matrices the Muon step updates are mostly experts (TorchTitan section 2.1:
top-2 routing, capacity factor 1.25).  ``sort_tokens`` turns the router's
choices into a ``Route``; ``dispatch`` lays the tokens out expert by expert;
``combine`` sums the experts' answers back with the router's weights.  Both
take part in autograd, backward and forward.  Everything runs in the library's kernels, on the
current stream; no call waits on the host.
"""
from __future__ import annotations

import ctypes
import operator
from functools import lru_cache

import torch
import torch.autograd.forward_ad as fwAD

from . import binding as B


class Route:
    """Where each token's choices stand among the sorted rows.

    ``row`` (tokens x topk, int32): the row of each choice, -1 for a dropped
    one.  ``offsets`` (experts + 1, int32): each expert's first row, and the
    end.  ``counts`` (experts, int32): each expert's rows that hold a token.
    ``capacity``: rows of every expert, or 0 where nothing is dropped and each
    expert's first row is a multiple of ``align``.  ``rows``: rows of a buffer
    of sorted tokens, known on the host."""

    __slots__ = ("row", "offsets", "counts", "capacity", "align", "shape", "rows", "_args", "index")

    def __init__(self, row, offsets, counts, capacity=0, align=1):
        if row.dim() != 2 or counts.dim() != 1 or offsets.dim() != 1 or offsets.numel() != counts.numel() + 1:
            raise ValueError("row must be tokens x topk, counts of length experts and offsets of length experts + 1")
        index = row.get_device()
        for t in (row, offsets, counts):
            if t.dtype != torch.int32 or not t.is_contiguous():
                raise ValueError("row, offsets and counts must be contiguous int32 tensors")
            if index < 0 or t.get_device() != index:
                raise ValueError("row, offsets and counts must be on one CUDA device")
        self._fill(row, offsets, counts, capacity, align,
                   *_sizes(row.shape[0], row.shape[1], counts.numel(), capacity, align)[:2])

    def _fill(self, row, offsets, counts, capacity, align, shape, rows):
        self.row, self.offsets, self.counts, self.capacity, self.align = row, offsets, counts, capacity, align
        self.shape, self.rows, self.index = shape, rows, row.get_device()
        self._args = (row, offsets, counts, ctypes.addressof(shape), rows)
        return self

    def _call(self):
        """The route, the thread's handle and the current stream, as a call takes them."""
        return (*self._args, B.thread_handle(self.index).value, B.current_stream(self.index))

    @property
    def experts(self) -> int:
        return self.counts.numel()


@lru_cache(maxsize=256, typed=True)
def _sizes(tokens, topk, experts, capacity, align):
    """The shape struct, the rows of the sorted buffer and the sort's workspace bytes."""
    numbers = dict(tokens=tokens, topk=topk, experts=experts, capacity=capacity, align=align)
    for name, x in numbers.items():
        numbers[name] = operator.index(x)
        bits = 63 if name == "tokens" else 31
        if not -(1 << bits) <= numbers[name] < 1 << bits:     # the struct would keep its low bits alone
            raise ValueError(f"{name} must be less than 2^{bits}, got {x}")
    shape = B.muon_moe_shape(**numbers)
    st, rows = B.muon_moe_rows(shape)
    if st != B.MUON_OK:
        raise B.MuonError(st, f"tokens={tokens}, topk={topk}, experts={experts}, capacity={capacity}, align={align}")
    return shape, rows, B.muon_moe_sort_workspace_size(shape)[1]


def _result(x, index, refuse):
    """What a call returned; else the error it stands for."""
    if x is None:
        refuse()
        raise ValueError("the tensors must be strided")
    if isinstance(x, int):
        raise B.MuonError(x, B.muon_last_error_message(B.thread_handle(index)))
    return x


def _refuse_matrix(t, name, rows, device):
    if t.dim() != 2 or t.shape[0] != rows:
        raise ValueError(f"{name} must have {rows} rows, got shape {tuple(t.shape)}")
    if t.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"{name} must be bf16 or fp32, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the route on {device}")


def _refuse_weights(w, route):
    if w is None:
        raise ValueError("weights of 1 have no gradient: dispatch lays dout out by expert")
    if w.shape != route.row.shape:
        raise ValueError(f"weights must have shape {tuple(route.row.shape)}, got {tuple(w.shape)}")
    if w.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"weights must be bf16 or fp32, got {w.dtype}")
    if w.device != route.row.device:
        raise ValueError(f"weights are on {w.device}, the route on {route.row.device}")


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
    index = expert_ids.get_device()
    if index < 0:
        raise ValueError(f"expert_ids must be a CUDA tensor, got one on {expert_ids.device}")
    tokens, topk = expert_ids.shape
    shape, rows, need = _sizes(tokens, topk, experts, capacity, align)
    row, offsets, counts = _result(
        B.torch_calls().sort(expert_ids, ctypes.addressof(shape), need, B.thread_handle(index).value,
                             B.current_stream(index)), index, lambda: None)
    return Route.__new__(Route)._fill(row, offsets, counts, capacity, align, shape, rows)


def _has_tangent(*tensors):
    """Whether one of the tensors carries a forward-mode derivative."""
    return fwAD._current_level >= 0 and any(t is not None and fwAD.unpack_dual(t).tangent is not None for t in tensors)


def _dispatch(x, route):
    return _result(B.torch_calls().dispatch(x, *route._call()), route.index,
                   lambda: _refuse_matrix(x, "x", route.row.shape[0], route.row.device))


def _combine(y, weights, route):
    def refuse():
        _refuse_matrix(y, "y", route.rows, route.row.device)
        if weights is not None:
            _refuse_weights(weights, route)

    return _result(B.torch_calls().combine(y, weights, *route._call()), route.index, refuse)


def combine_backward(dout, y, weights, route: Route):
    """(dy, dweights) of ``combine`` for the gradient ``dout`` of its result.
    Not differentiable itself."""
    if _has_tangent(dout, y, weights):
        raise RuntimeError("combine's gradient has no forward-mode derivative")

    def refuse():
        _refuse_matrix(dout, "dout", route.row.shape[0], route.row.device)
        _refuse_matrix(y, "y", route.rows, route.row.device)
        if dout.shape[1] != y.shape[1] or dout.dtype != y.dtype:
            raise ValueError(f"dout and y must have one row length and type, got {tuple(dout.shape)} {dout.dtype} and "
                             f"{tuple(y.shape)} {y.dtype}")
        _refuse_weights(weights, route)

    return _result(B.torch_calls().combine_backward(dout, y, weights, *route._call()), route.index, refuse)


def dispatch_backward(dxs, route: Route):
    """dx of ``dispatch`` for the gradient ``dxs`` of its result: a token's
    gradient is the sum over its rows, that is ``combine`` without weights."""
    return combine(dxs, None, route)


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, route):
        ctx.route = route
        return _dispatch(x, route)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dxs):
        return dispatch_backward(dxs, ctx.route), None

    @staticmethod
    def jvp(ctx, tx, _):
        return dispatch(tx, ctx.route)


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, weights, route):
        ctx.route = route
        ctx.set_materialize_grads(False)    # an input without a tangent adds nothing
        ctx.save_for_backward(*(() if weights is None else (y, weights)))
        ctx.save_for_forward(*(() if weights is None else (y, weights)))
        return _combine(y, weights, route)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        if dout is None:
            return None, None, None
        if not ctx.saved_tensors:   # weights of 1: the gradient lays dout out by expert
            return dispatch(dout, ctx.route), None, None
        y, weights = ctx.saved_tensors
        dy, dw = combine_backward(dout, y, weights, ctx.route)
        return dy, dw, None

    @staticmethod
    def jvp(ctx, ty, tw, _):
        # linear in the rows and in the weights
        y, weights = ctx.saved_tensors or (None, None)
        out = None if ty is None else combine(ty, weights, ctx.route)
        if tw is None:
            return out
        by_weights = combine(y, tw, ctx.route)
        return by_weights if out is None else out + by_weights


def dispatch(x, route: Route):
    """The sorted rows (route.rows x hidden) of ``x`` (tokens x hidden, fp32 or
    bf16): each token's row at the place of each of its choices, zero in rows
    without a token."""
    if (torch.is_grad_enabled() and x.requires_grad) or _has_tangent(x):
        return _Dispatch.apply(x, route)
    return _dispatch(x, route)


def combine(y, weights, route: Route):
    """out[t] = sum over k of weights[t, k] * y[row[t, k]] for sorted rows ``y``
    (fp32 or bf16) and ``weights`` (tokens x topk, fp32 or bf16; None for 1),
    summed in fp32.  Dropped choices are left out."""
    recorded = torch.is_grad_enabled() and (y.requires_grad or (weights is not None and weights.requires_grad))
    if recorded or _has_tangent(y, weights):
        return _Combine.apply(y, weights, route)
    return _combine(y, weights, route)
