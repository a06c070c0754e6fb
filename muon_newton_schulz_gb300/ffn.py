"""The gated feed-forward block of experts, or of one dense layer.

Its matrices are what the Muon step updates (TorchTitan section 2.1: experts
8192 wide).  Between ``moe.dispatch`` and ``moe.combine``, ``gated_ffn`` takes the
sorted rows through every expert's

    h = act(x gate^T) * (x up^T),   y = h down^T

and takes part in autograd.  What it keeps for the backward pass can be kept
in 8 bits.  Everything runs in the library's kernels, on the current stream; no call
waits on the host but ``check_status``.
"""
from __future__ import annotations

import torch

from . import binding as B
from .moe import _has_tangent, _result

ACTIVATIONS = {"silu": B.MUON_SILU, "gelu": B.MUON_GELU}


class Saved:
    """What a forward pass keeps: the inputs (``x`` itself, or with ``bits=8`` their
    codes and scales) and the pre-activations, with the route and the activation."""

    __slots__ = ("x", "kept", "route", "activation", "bits", "shape", "ffn", "dtype", "_versions")

    def __init__(self, x, kept, route, activation, bits, shape, ffn, dtype):
        self.x, self.kept, self.route, self.activation, self.bits = x, kept, route, activation, bits
        self.shape, self.ffn, self.dtype = shape, ffn, dtype
        self._versions = self._now()

    def _now(self):
        """How often what is not copied has been written (an inference tensor does not count)."""
        held = (self.x, *((None, None) if self.route is None else (self.route.offsets, self.route.counts)))
        return tuple(None if t is None or t.is_inference() else t._version for t in held)


def _refuse(rows, gate, up, down, route, name):
    if rows.dim() != 2:
        raise ValueError(f"{name} must be rows x hidden, got shape {tuple(rows.shape)}")
    if rows.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"{name} must be bf16 or fp32, got {rows.dtype}")
    if rows.get_device() < 0:
        raise ValueError(f"{name} must be a CUDA tensor, got one on {rows.device}")
    hidden = rows.shape[1]
    dims = () if route is None else (route.experts,)
    if gate.dim() != len(dims) + 2:
        raise ValueError(f"w_gate must be {'experts x ' if dims else ''}ffn x hidden, got shape {tuple(gate.shape)}")
    ffn = gate.shape[-2]
    for t, shape, what in ((gate, (*dims, ffn, hidden), "w_gate"), (up, (*dims, ffn, hidden), "w_up"), (down, (*dims, hidden, ffn), "w_down")):
        if tuple(t.shape) != shape:
            raise ValueError(f"{what} must have shape {shape}, got {tuple(t.shape)}")
        if t.dtype != rows.dtype:
            raise ValueError(f"{what} must be {rows.dtype} as {name} is, got {t.dtype}")
        if t.device != rows.device:
            raise ValueError(f"{what} is on {t.device}, {name} on {rows.device}")


def _check_route(rows, route, name):
    if route is not None:
        if rows.shape[0] != route.rows:
            raise ValueError(f"{name} must have the route's {route.rows} rows, got shape {tuple(rows.shape)}")
        if rows.get_device() != route.index:
            raise ValueError(f"{name} is on {rows.device}, the route on {route.row.device}")


def _forward(x, gate, up, down, route, activation, bits):
    """What the built module returns."""
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, got {activation!r}")
    index = x.get_device()
    if index < 0 or x.dim() != 2:
        _refuse(x, gate, up, down, route, "x")
    _check_route(x, route, "x")
    offsets, counts = (None, None) if route is None else (route.offsets, route.counts)
    return _result(B.torch_calls().ffn_forward(x, gate, up, down, offsets, counts, act, bits, B.thread_handle(index).value,
                                               B.current_stream(index)), index,
                   lambda: _refuse(x, gate, up, down, route, "x"))


def _bits(saved_bits, dtype):
    if saved_bits not in (None, 8):
        raise ValueError(f"saved_bits must be None (the type's own) or 8, got {saved_bits}")
    return 8 if saved_bits == 8 else 16 if dtype == torch.bfloat16 else 32


def gated_ffn_saved(x, w_gate, w_up, w_down, route=None, activation="silu", saved_bits=None):
    """(y, saved) of ``gated_ffn``: ``saved`` is what ``gated_ffn_backward``
    needs.  Not recorded by autograd."""
    if _has_tangent(x, w_gate, w_up, w_down):
        raise RuntimeError("gated_ffn_saved has no forward-mode derivative")
    bits = _bits(saved_bits, x.dtype)
    y, *kept = _forward(x, w_gate, w_up, w_down, route, activation, bits)
    return y, Saved(None if bits == 8 else x.detach(), kept, route, activation, bits, x.shape, w_gate.shape[-2], x.dtype)


def _backward(dy, x, gate, up, down, kept, route, activation, bits, want):
    def refuse():
        _refuse(dy, gate, up, down, route, "dy")
        raise ValueError("saved must be what gated_ffn_saved returned for these weights")

    index = dy.get_device()
    if index < 0:
        refuse()
    offsets, counts = (None, None) if route is None else (route.offsets, route.counts)
    return _result(B.torch_calls().ffn_backward(dy, x, gate, up, down, offsets, counts, kept, ACTIVATIONS[activation], bits, want,
                                                B.thread_handle(index).value, B.current_stream(index)), index, refuse)


def gated_ffn_backward(dy, saved: Saved, w_gate, w_up, w_down):
    """(dx, dw_gate, dw_up, dw_down) of ``gated_ffn`` for the gradient ``dy`` of
    its result, from what its forward pass kept.  Not differentiable itself."""
    if _has_tangent(dy, w_gate, w_up, w_down):
        raise RuntimeError("gated_ffn's gradient has no forward-mode derivative")
    if dy.shape != saved.shape or dy.dtype != saved.dtype:
        raise ValueError(f"dy must have the result's shape {tuple(saved.shape)} and type {saved.dtype}, got {tuple(dy.shape)} {dy.dtype}")
    if w_gate.dim() < 2 or w_gate.shape[-2] != saved.ffn:
        raise ValueError(f"w_gate must be {saved.ffn} wide as in the forward pass, got shape {tuple(w_gate.shape)}")
    if saved._now() != saved._versions:
        raise RuntimeError("x or the route has been modified since the forward pass")
    return _backward(dy, saved.x, w_gate, w_up, w_down, saved.kept, saved.route, saved.activation, saved.bits, 15)


class _GatedFfn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate, up, down, route, activation, bits):
        y, *kept = _forward(x, gate, up, down, route, activation, bits)
        # the route's tensors too, so that a change to them is noticed
        ctx.save_for_backward(None if bits == 8 else x, gate, up, down, *((None, None) if route is None else (route.offsets, route.counts)), *kept)
        ctx.route, ctx.activation, ctx.bits = route, activation, bits
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, gate, up, down, _, _, *kept = ctx.saved_tensors
        want = sum(1 << i for i in range(4) if ctx.needs_input_grad[i])
        return (*_backward(dy, x, gate, up, down, kept, ctx.route, ctx.activation, ctx.bits, want), None, None, None)


def gated_ffn(x, w_gate, w_up, w_down, route=None, activation="silu", saved_bits=None):
    """y = h w_down^T with h = act(x w_gate^T) * (x w_up^T), for every expert's
    rows of ``x`` (route.rows x hidden, as ``moe.dispatch`` gives them) with
    its own matrices: w_gate and w_up experts x ffn x hidden, w_down experts x
    hidden x ffn.  Without a route one dense layer: matrices of two dimensions,
    any number of rows.  All bf16 or all fp32; matrices may be transposed
    views.  ``activation``: "silu" or "gelu" (with the normal distribution).
    What rows that hold no token hold counts for nothing; they are 0 in the result and in x's
    gradient.

    Where a gradient is needed, x, both pre-activations and h are kept in as many
    bits as the inputs (the pre-activations of bf16 as fp16 numbers with a power of
    two for each 32); with ``saved_bits=8`` x and the pre-activations in 8 bits
    alone, as ``checkpoint.pack`` keeps them."""
    bits = _bits(saved_bits, x.dtype)
    if _has_tangent(x, w_gate, w_up, w_down):
        raise RuntimeError("gated_ffn has no forward-mode derivative")
    if torch.is_grad_enabled() and any(t.requires_grad for t in (x, w_gate, w_up, w_down)):
        return _GatedFfn.apply(x, w_gate, w_up, w_down, route, activation, bits)
    return _forward(x, w_gate, w_up, w_down, route, activation, 0)


def check_status(device=None) -> int:
    """Waits for the current stream of ``device`` (torch's current one by default):
    ``binding.MUON_ERR_TIMEOUT`` if a kernel of this module gave up a bounded wait on the device since
    the last such call, from whichever thread and in whichever direction it was called (what
    these calls returned is incomplete), else ``binding.MUON_OK``."""
    device = torch.device("cuda" if device is None else device)
    if device.type != "cuda":
        raise ValueError(f"device must be a CUDA device, got {device}")
    index = torch.cuda.current_device() if device.index is None else device.index
    if B.stream_is_capturing(index):
        raise RuntimeError("the status cannot be read while the stream is being captured")
    st = B.muon_ffn_check_status(B.thread_handle(index), B.current_stream(index))
    if st not in (B.MUON_OK, B.MUON_ERR_TIMEOUT):
        raise B.MuonError(st, B.muon_last_error_message(B.thread_handle(index)))
    return st
