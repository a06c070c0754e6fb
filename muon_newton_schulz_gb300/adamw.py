"""AdamW over many tensors, and gradient clipping by the global norm.

The Muon step covers the weight matrices; embeddings, LM head, router and
norms are left to AdamW (ZAYA1/MI300X section 4.3; EU-1T, optimizer-state
paragraph).  ``adamw_step`` runs the library's ``muon_adamw_step``: one launch
for all tensors, with the states m and v in fp32 or in 8 bits.  ``clip_grads``
runs ``muon_clip_grads`` over the gradients of both optimizers.  ``optim.AdamW``
and ``optim.clip_grad_norm`` put torch.optim conventions in front of them.
"""
from __future__ import annotations

import torch

from . import binding as B

STATE_BLOCK = 256   # elements of an 8-bit state that share its scales


def is_dense(t: torch.Tensor) -> bool:
    """True when t's elements fill one block of memory, in any order of its dimensions."""
    if t.is_contiguous():
        return True
    expect = 1
    for stride, size in sorted((st, n) for st, n in zip(t.stride(), t.shape) if n != 1):
        if stride != expect:
            return False
        expect *= size
    return True


def state8_like(p: torch.Tensor):
    """Fresh 8-bit states of ``p``: (m, v, scales), all zero.

    m holds e4m3 codes and v e5m2 codes in p's memory order; scales has one
    row (m's scale, v's scale) of powers of two per 256 elements."""
    n = p.numel()
    m = torch.zeros_like(p, dtype=torch.uint8).view(torch.float8_e4m3fn)
    v = torch.zeros_like(p, dtype=torch.uint8).view(torch.float8_e5m2)
    scales = torch.zeros(-(-n // STATE_BLOCK), 2, dtype=torch.uint8, device=p.device).view(torch.float8_e8m0fnu)
    return m, v, scales


def state8_values(m: torch.Tensor, v: torch.Tensor, scales: torch.Tensor):
    """The fp32 values that 8-bit states stand for (contiguous m and v)."""
    n = m.numel()
    each = scales.float().repeat_interleave(STATE_BLOCK, 0)[:n]
    return (m.float().flatten() * each[:, 0]).view_as(m), (v.float().flatten() * each[:, 1]).view_as(v)


def _check_dtypes(i, **tensors):
    for name, t in tensors.items():
        if t.dtype not in (torch.float32, torch.bfloat16):
            raise ValueError(f"tensor {i}: a {name} must be bf16 or fp32, got {t.dtype}")


def _check_state(p, m, v, s, i, index):
    if s is None:
        kinds = (torch.float32, torch.float32)
    else:
        kinds = (torch.float8_e4m3fn, torch.float8_e5m2)
        if s.dtype != torch.float8_e8m0fnu or not s.is_contiguous() or s.numel() != 2 * -(-p.numel() // STATE_BLOCK):
            raise ValueError(f"tensor {i}: scales must be a contiguous float8_e8m0fnu tensor with two entries per "
                             f"{STATE_BLOCK} elements")
        if s.get_device() != index:
            raise ValueError(f"tensor {i}: scales must be on CUDA device {index}, got {s.device}")
    for t, kind, name in ((m, kinds[0], "m"), (v, kinds[1], "v")):
        if t.dtype != kind:
            raise ValueError(f"tensor {i}: {name} must be {kind}, got {t.dtype}")


def _check_layout(p, g, m, v, i, index):
    size, stride = p.shape, p.stride()
    for t, name in ((p, "parameter"), (g, "gradient"), (m, "m"), (v, "v")):
        if t.get_device() != index:
            raise ValueError(f"tensor {i}: {name} must be on CUDA device {index}, got {t.device}")
        if t.shape != size or (t.stride() != stride and not (t.is_contiguous() and p.is_contiguous())):
            raise ValueError(f"tensor {i}: {name} must have its parameter's shape and strides")
    if not is_dense(p):
        raise ValueError(f"tensor {i}: a parameter must fill its memory without gaps, got shape {tuple(size)} with "
                         f"strides {stride}")


def adamw_step(params, grads, ms, vs, scales=None, *, lr, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.0, step, seed=0,
               stream=None):
    """One AdamW step over lists of CUDA tensors on the current stream (or ``stream``).

    ``params`` (fp32 or bf16), ``ms`` and ``vs`` are updated in place; ``grads``
    (fp32 or bf16) are read.  The tensors of one entry must have the same shape
    and strides and fill their memory without gaps.  ``scales`` is None for
    fp32 states; else a list with None for a tensor with fp32 states and the
    scales of one with 8-bit states (``state8_like``), which are updated too.
    ``lr``, ``weight_decay`` and ``step`` (from 1) are numbers, or a list of
    one per tensor.  Tensor i draws the random bits of its 8-bit rounding from
    its step and its seed: ``seed + i``, or ``seed[i]`` of a list.

    Those numbers are part of the launch.  A call captured in a CUDA graph
    does step number ``step`` again on every replay, with the same bias
    corrections and random bits: a graph may replay it to repeat that step, on
    inputs set back, but not to go on to the next."""
    n = len(params)
    if not (len(grads) == len(ms) == len(vs) == n) or (scales is not None and len(scales) != n):
        raise ValueError("params, grads, ms, vs and scales must have the same length")
    for x, name in ((lr, "lr"), (weight_decay, "weight_decay"), (step, "step"), (seed, "seed")):
        if isinstance(x, list) and len(x) != n:
            raise ValueError(f"a list of {name} must have an entry for each of the {n} tensors, got {len(x)}")
    if n == 0:
        return
    index = params[0].get_device()
    if index < 0:
        raise ValueError(f"parameters must be CUDA tensors, got one on {params[0].device}")
    h = B.thread_handle(index)
    st = B.torch_calls().adamw(params, grads, ms, vs, scales, index, lr, weight_decay, step, seed, betas[0], betas[1], eps,
                               h.value, B.current_stream(index) if stream is None else stream)
    if st is None:
        for i in range(n):
            _check_layout(params[i], grads[i], ms[i], vs[i], i, index)
            _check_dtypes(i, parameter=params[i], gradient=grads[i])
            _check_state(params[i], ms[i], vs[i], scales[i] if scales is not None else None, i, index)
        raise ValueError("adamw_step takes lists of strided tensors")
    if st != B.MUON_OK:
        raise B.MuonError(st, B.muon_last_error_message(h))


def _check_clip(g, out, i, index):
    _check_dtypes(i, gradient=g, output=out)
    if g.get_device() != index or out.get_device() != index:
        raise ValueError(f"gradient {i}: all tensors must be on CUDA device {index}, got {g.device} and {out.device}")
    if g.shape != out.shape:
        raise ValueError(f"gradient {i}: the output must have its shape {tuple(g.shape)}, got {tuple(out.shape)}")
    matrices = g.dim() == 2 and (g.shape[1] == 1 or g.stride(1) == out.stride(1) == 1)
    if not matrices and not (is_dense(g) and (g.stride() == out.stride() or g.is_contiguous() and out.is_contiguous())):
        raise ValueError(f"gradient {i}: a gradient must fill its memory without gaps, its output in the same order, or "
                         "both be matrices with unit column stride")


def clip_grads(grads, max_norm: float, outs=None, stream=None) -> torch.Tensor:
    """Scales ``grads`` so that their global norm is at most ``max_norm`` and
    returns the norm before that (a 0-dim fp32 tensor on their device; the host
    does not wait).  In place, or into ``outs`` (the fp32 buffers that the Muon
    step reads, for instance).  ``max_norm=inf`` computes the norm alone and
    leaves gradients and outputs as they are; no gradients give 0, on the CPU."""
    n = len(grads)
    if outs is None:
        outs = grads
    if len(outs) != n:
        raise ValueError("grads and outs must have the same length")
    if n == 0:
        return torch.zeros(())
    index = grads[0].get_device()
    if index < 0:
        raise ValueError(f"gradients must be CUDA tensors, got one on {grads[0].device}")
    h = B.thread_handle(index)
    if stream is None:
        norm = B.torch_calls().clip(grads, outs, index, max_norm, h.value, B.current_stream(index))
    else:   # the workspace belongs to the stream that uses it
        with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=grads[0].device)):
            norm = B.torch_calls().clip(grads, outs, index, max_norm, h.value, stream)
    if norm is None:
        for i in range(n):
            _check_clip(grads[i], outs[i], i, index)
        raise ValueError("clip_grads takes lists of strided tensors")
    if isinstance(norm, int):
        raise B.MuonError(norm, B.muon_last_error_message(h))
    return norm
