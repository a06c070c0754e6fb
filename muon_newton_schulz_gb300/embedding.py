"""Embedding rows with scaling, and their gradient by sorted tokens.

The embedding is the first of what the Muon step leaves to AdamW
(ZAYA1/MI300X section 4.3).  ``embed`` reads and scales the rows of a batch's
token ids and takes part in autograd, backward and forward; its gradient sums each
id's tokens in a fixed order, so a step gives the same bits every time.
Everything runs in the library's kernels, on the current stream; no call waits on
the host.
"""
from __future__ import annotations

import operator

import torch

from . import binding as B
from .moe import _has_tangent, _result


def _refuse(ids, matrix, name):
    if ids.dtype not in (torch.int32, torch.int64):
        raise ValueError(f"ids must be int32 or int64, got {ids.dtype}")
    if ids.get_device() < 0:
        raise ValueError(f"ids must be a CUDA tensor, got one on {ids.device}")
    if matrix.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"{name} must be bf16 or fp32, got {matrix.dtype}")
    if matrix.device != ids.device:
        raise ValueError(f"{name} is on {matrix.device}, the ids on {ids.device}")


def _embed(ids, table, scale):
    def refuse():
        _refuse(ids, table, "table")
        if table.dim() != 2:
            raise ValueError(f"table must be vocab x hidden, got shape {tuple(table.shape)}")

    index = ids.get_device()
    if index < 0:
        refuse()
    return _result(B.torch_calls().embed(ids, table, scale, B.thread_handle(index).value, B.current_stream(index)), index, refuse)


def embed_backward(dout, ids, vocab: int, scale: float = 1.0):
    """The gradient (vocab x hidden) of ``embed``'s table for the gradient
    ``dout`` (the ids' shape x hidden, fp32 or bf16) of its result.  Not
    differentiable itself."""
    if _has_tangent(dout):
        raise RuntimeError("embed's gradient has no forward-mode derivative")
    vocab = operator.index(vocab)

    def refuse():
        _refuse(ids, dout, "dout")
        if dout.dim() != ids.dim() + 1 or dout.shape[:-1] != ids.shape:
            raise ValueError(f"dout must have the ids' shape {tuple(ids.shape)} x hidden, got {tuple(dout.shape)}")
        if vocab < 0:
            raise ValueError(f"vocab must not be negative, got {vocab}")

    index = ids.get_device()
    if index < 0:
        refuse()
    if not -(1 << 63) <= vocab < 1 << 63:
        raise ValueError(f"vocab must be less than 2^63, got {vocab}")
    return _result(B.torch_calls().embed_backward(dout, ids, vocab, scale, B.thread_handle(index).value, B.current_stream(index)),
                   index, refuse)


class _Embed(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, table, scale):
        ctx.save_for_backward(ids)
        ctx.save_for_forward(ids)
        ctx.vocab, ctx.scale = table.shape[0], scale
        return _embed(ids, table, scale)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        ids, = ctx.saved_tensors
        return None, embed_backward(dout, ids, ctx.vocab, ctx.scale), None

    @staticmethod
    def jvp(ctx, _, ttable, __):
        ids, = ctx.saved_tensors
        return embed(ids, ttable, ctx.scale)


def embed(ids, table, scale: float = 1.0):
    """``scale`` times the rows of ``table`` (vocab x hidden, fp32 or bf16) for
    ``ids`` (int32 or int64, any shape), of the ids' shape x hidden.  An id outside
    the table, -1 for a padding token for instance, gives zeros and has no
    gradient."""
    if (torch.is_grad_enabled() and table.requires_grad) or _has_tangent(table):
        return _Embed.apply(ids, table, scale)
    return _embed(ids, table, scale)
