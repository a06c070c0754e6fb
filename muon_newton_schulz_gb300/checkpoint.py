"""Activations kept in 8 bits between the forward and the backward pass.

What a training step keeps for its gradients takes more memory than its
weights.  ``pack`` stores a tensor as e4m3 codes with a power-of-two scale for each
32 elements of its last dimension, half the bytes of bf16, and ``unpack`` gives the
values back.  ``saved_in_8_bits`` does so for the activations that operations of torch save.
``ffn.gated_ffn`` keeps its own activations this way with ``saved_bits=8``.
Everything runs in the library's kernels, on the current stream.
"""
from __future__ import annotations

import torch

from . import binding as B
from .moe import _has_tangent, _result

BLOCK = 32   # elements of a row that share a scale


class Packed:
    """A tensor in 8 bits: ``codes`` (e4m3, its shape) times ``scales`` (powers of
    two, one for each 32 elements of the last dimension); ``dtype`` is its own.  With
    ``special`` the codes of 448 and -448 stand for infinities."""

    __slots__ = ("codes", "scales", "dtype", "special")

    def __init__(self, codes, scales, dtype, special=False):
        self.codes, self.scales, self.dtype, self.special = codes, scales, dtype, special

    @property
    def shape(self):
        return self.codes.shape


def pack(x, special: bool = False) -> Packed:
    """``x`` (fp32 or bf16, one dimension or more) in 8 bits.  An element is off
    by at most 2^-4 of itself, or 2^-17 of its block's largest or 2^-136 where that is more
    (a magnitude from 1.9375 * 2^127 on becomes infinite);
    one that is not finite becomes NaN.  With ``special`` each stays of its kind:
    infinities, finite numbers, and numbers that are not zero (at 2^-16 of the block's largest
    at least).  Not differentiable."""
    if _has_tangent(x):
        raise RuntimeError("packing has no forward-mode derivative")

    def refuse():
        if x.dtype not in (torch.float32, torch.bfloat16):
            raise ValueError(f"x must be bf16 or fp32, got {x.dtype}")
        if x.dim() < 1:
            raise ValueError("x must have a dimension")
        if x.get_device() < 0:
            raise ValueError(f"x must be a CUDA tensor, got one on {x.device}")

    index = x.get_device()
    if index < 0:
        refuse()
    codes, scales = _result(B.torch_calls().pack8(x, B.thread_handle(index).value, B.current_stream(index), special), index, refuse)
    return Packed(codes, scales, x.dtype, special)


def unpack(p: Packed, dtype=None):
    """The values of a packed tensor, in its own type or ``dtype``."""
    dtype = p.dtype if dtype is None else dtype
    if dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"dtype must be bf16 or fp32, got {dtype}")

    def refuse():
        for t, kind, name in ((p.codes, torch.float8_e4m3fn, "codes"), (p.scales, torch.float8_e8m0fnu, "scales")):
            if t.dtype != kind:
                raise ValueError(f"{name} must be {kind}, got {t.dtype}")
            if t.get_device() < 0 or t.device != p.codes.device:
                raise ValueError(f"codes and scales must be on one CUDA device, got {p.codes.device} and {p.scales.device}")
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        want = (*p.codes.shape[:-1], -(-p.codes.shape[-1] // BLOCK)) if p.codes.dim() else "a dimension"
        raise ValueError(f"scales must have shape {want}, got {tuple(p.scales.shape)}")

    index = p.codes.get_device()
    if index < 0:
        refuse()
    return _result(B.torch_calls().unpack8(p.codes, p.scales, dtype == torch.bfloat16, B.thread_handle(index).value,
                                           B.current_stream(index), p.special), index, refuse)


def _is_parameter(t):
    base = t if t._base is None else t._base
    return base.is_leaf and base.requires_grad


# Results that are logarithms: what saves them takes their exponential, where an error of 2^-4 of
# the value is no small one.
_LOGARITHMS = frozenset(("LogSoftmaxBackward0", "LogsumexpBackward0", "LogcumsumexpBackward0"))


def _is_statistic(t):
    """Whether t is something an operation keeps beside its activations: without a gradient of its own (a softmax's
    normalizer in attention, a mask, what a torch.autograd.Function computed), a second result (a norm's mean), one
    number for each row (its root mean square), or a logarithm."""
    node = t.grad_fn
    if node is None:
        return not t.requires_grad
    return t.shape[-1] == 1 or node.name() in _LOGARITHMS or (t.output_nr > 0 and not t._is_view())


def saved_in_8_bits(min_elements: int = 65536, which=None):
    """A context in which torch keeps in 8 bits the activations that operations save
    for their backward pass: bf16 and fp32 CUDA tensors of at least ``min_elements``
    elements that a gradient goes through and for which ``which`` (a function of the tensor, if
    given) is true, but not parameters or views of them (a cast copy of one is no
    view).  A tensor that several operations save is packed for each.

    Elements are off as ``pack`` with ``special`` says.  Left alone as they are:
    inputs, masks and statistics without a gradient, an operation's second and further results, tensors
    whose last dimension is 1, and the results of log_softmax and logsumexp.  An operation that takes an exponential, sine or
    the like of what it saves (logsumexp of its argument, for one), or divides by elements far smaller than
    others of their row, needs more bits than this: leave such tensors out with ``which``, or the operation out of the context."""
    @torch.no_grad()
    def keep(t):
        if (not t.is_cuda or t.dtype not in (torch.float32, torch.bfloat16) or t.layout != torch.strided or t.dim() < 1
                or t.numel() < min_elements or _is_statistic(t) or _is_parameter(t) or (which is not None and not which(t))):
            return t
        return pack(t, special=True)

    @torch.no_grad()
    def give(kept):
        return unpack(kept) if isinstance(kept, Packed) else kept

    return torch.autograd.graph.saved_tensors_hooks(keep, give)
