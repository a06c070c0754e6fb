"""AdamW over many tensors, and gradient clipping by the global norm.

The Muon step covers the weight matrices; embeddings, LM head, router and
norms are left to AdamW (ZAYA1/MI300X section 4.3; EU-1T, optimizer-state
paragraph).  ``adamw_step`` runs the library's ``muon_adamw_step``: one launch
for all tensors, with the states m and v in fp32 or in 8 bits.  ``clip_grads``
runs ``muon_clip_grads`` over the gradients of both optimizers.  ``optim.AdamW``
and ``optim.clip_grad_norm`` put torch.optim conventions in front of them.
"""
from __future__ import annotations

import ctypes
import operator

import numpy as np
import torch

from . import binding as B

STATE_BLOCK = 256   # elements of an 8-bit state that share its scales
_DTYPES = {torch.float32: B.MUON_F32, torch.bfloat16: B.MUON_BF16}


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


_DESC = np.dtype([("n", "i8"), ("P", "u8"), ("G", "u8"), ("M", "u8"), ("V", "u8"), ("scales", "u8"), ("p_dtype", "i4"),
                  ("g_dtype", "i4"), ("state_bits", "i4"), ("reserved", "i4"), ("step", "i8"), ("seed", "u8"),
                  ("lr", "f8"), ("weight_decay", "f8")])
_CLIP_DESC = np.dtype([("rows", "i8"), ("cols", "i8"), ("G", "u8"), ("ldg", "i8"), ("out", "u8"), ("ldo", "i8"),
                       ("g_dtype", "i4"), ("out_dtype", "i4")])
assert _DESC.itemsize == ctypes.sizeof(B.muon_adamw_desc) and _CLIP_DESC.itemsize == ctypes.sizeof(B.muon_clip_desc)

# what is asked of every tensor of a list, as calls that need no Python code of ours per tensor
_shape, _dtype = operator.attrgetter("shape"), operator.attrgetter("dtype")
_contiguous, _numel, _ptr, _index = (torch.Tensor.is_contiguous, torch.Tensor.numel, torch.Tensor.data_ptr,
                                     torch.Tensor.get_device)


def _plain(lists, shapes, index):
    """True when every tensor of every list is contiguous, of the given shapes and on one CUDA device."""
    return all(list(map(_shape, ts)) == shapes and all(map(_contiguous, ts)) and set(map(_index, ts)) == index
               for ts in lists)


def _dtypes(ts, name):
    kinds = list(map(_dtype, ts))
    try:
        return _DTYPES[kinds[0]] if kinds.count(kinds[0]) == len(kinds) else [_DTYPES[k] for k in kinds]
    except KeyError:
        i = next(i for i, k in enumerate(kinds) if k not in _DTYPES)
        raise ValueError(f"tensor {i}: {name} must be bf16 or fp32, got {kinds[i]}") from None


def adamw_step(params, grads, ms, vs, scales=None, *, lr, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.0, step, seed=0,
               stream=None):
    """One AdamW step over lists of CUDA tensors on the current stream (or ``stream``).

    ``params`` (fp32 or bf16), ``ms`` and ``vs`` are updated in place; ``grads``
    (fp32 or bf16) are read.  The tensors of one entry must have the same shape
    and strides and fill their memory without gaps.  ``scales`` is None for
    fp32 states; else a list with None for a tensor with fp32 states and the
    scales of one with 8-bit states (``state8_like``), which are updated too.
    ``lr``, ``weight_decay`` and ``step`` (from 1) are numbers, or one per
    tensor.  Tensor i draws the random bits of its 8-bit rounding from
    ``seed + i`` and its step."""
    n = len(params)
    if not (len(grads) == len(ms) == len(vs) == n) or (scales is not None and len(scales) != n):
        raise ValueError("params, grads, ms, vs and scales must have the same length")
    if n == 0:
        return
    index = params[0].get_device()
    if index < 0:
        raise ValueError(f"parameters must be CUDA tensors, got one on {params[0].device}")
    if scales is None:
        scales = [None] * n
    if not _plain((params, grads, ms, vs), list(map(_shape, params)), {index}):
        for i in range(n):
            _check_layout(params[i], grads[i], ms[i], vs[i], i, index)
    d = np.zeros(n, _DESC)
    d["p_dtype"], d["g_dtype"] = _dtypes(params, "a parameter"), _dtypes(grads, "a gradient")
    d["state_bits"] = 32
    if not (all(s is None for s in scales) and set(map(_dtype, ms)) == set(map(_dtype, vs)) == {torch.float32}):
        for i in range(n):
            _check_state(params[i], ms[i], vs[i], scales[i], i, index)
            if scales[i] is not None:
                d["state_bits"][i], d["scales"][i] = 8, scales[i].data_ptr()
    d["n"] = list(map(_numel, params))
    for name, ts in (("P", params), ("G", grads), ("M", ms), ("V", vs)):
        d[name] = list(map(_ptr, ts))
    d["step"], d["lr"], d["weight_decay"] = step, lr, weight_decay
    d["seed"] = np.arange(n, dtype=np.uint64) + np.uint64(seed & 0xFFFFFFFFFFFFFFFF)
    h = B.thread_handle(index)
    st = B.muon_adamw_step(h, B.muon_adamw_config(betas[0], betas[1], eps), d.ctypes.data, n,
                           B.current_stream(index) if stream is None else stream)
    if st != B.MUON_OK:
        raise B.MuonError(st, B.muon_last_error_message(h))


def _clip_layout(g, out, i, index):
    """rows, cols, ldg, ldo of a gradient and its output that are not both contiguous."""
    if g.get_device() != index or out.get_device() != index:
        raise ValueError(f"gradient {i}: all tensors must be on CUDA device {index}, got {g.device} and {out.device}")
    if g.shape != out.shape:
        raise ValueError(f"gradient {i}: the output must have its shape {tuple(g.shape)}, got {tuple(out.shape)}")
    if (g.stride() == out.stride() or (g.is_contiguous() and out.is_contiguous())) and is_dense(g):
        return 1, g.numel(), g.numel(), g.numel()
    if g.dim() == 2 and (g.stride(1) == 1 or g.shape[1] == 1) and (out.stride(1) == 1 or out.shape[1] == 1):
        return g.shape[0], g.shape[1], g.stride(0), out.stride(0)
    raise ValueError(f"gradient {i}: a gradient must fill its memory without gaps, its output in the same order, or "
                     "both be matrices with unit column stride")


def clip_grads(grads, max_norm: float, outs=None, stream=None) -> torch.Tensor:
    """Scales ``grads`` so that their global norm is at most ``max_norm`` and
    returns the norm before that (a 0-dim fp32 tensor on their device; the host
    does not wait).  In place, or into ``outs`` (the fp32 buffers that the Muon
    step reads, for instance).  ``max_norm=inf`` computes the norm alone and
    leaves gradients and outputs as they are."""
    n = len(grads)
    if outs is not None and len(outs) != n:
        raise ValueError("grads and outs must have the same length")
    if n == 0:
        return torch.zeros(())
    index = grads[0].get_device()
    if index < 0:
        raise ValueError(f"gradients must be CUDA tensors, got one on {grads[0].device}")
    d = np.zeros(n, _CLIP_DESC)
    d["g_dtype"] = _dtypes(grads, "a gradient")
    if outs is None:
        outs = grads
        d["out_dtype"] = d["g_dtype"]
    else:
        d["out_dtype"] = _dtypes(outs, "an output")
    if _plain((grads,) if outs is grads else (grads, outs), list(map(_shape, grads)), {index}):
        d["rows"] = 1
        d["cols"] = d["ldg"] = d["ldo"] = list(map(_numel, grads))
    else:
        for i in range(n):
            d["rows"][i], d["cols"][i], d["ldg"][i], d["ldo"][i] = _clip_layout(grads[i], outs[i], i, index)
    d["G"] = list(map(_ptr, grads))
    d["out"] = d["G"] if outs is grads else list(map(_ptr, outs))
    words = B.MUON_CLIP_WORKSPACE_BYTES // 4
    if stream is None:
        stream = B.current_stream(index)
        buf = torch.empty(words + 64, dtype=torch.float32, device=grads[0].device)
    else:
        with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=grads[0].device)):
            buf = torch.empty(words + 64, dtype=torch.float32, device=grads[0].device)
    norm = buf[words]
    at = buf.data_ptr()
    h = B.thread_handle(index)
    st = B.muon_clip_grads(h, d.ctypes.data, n, max_norm, at + 4 * words, at, 4 * words, stream)
    if st != B.MUON_OK:
        raise B.MuonError(st, B.muon_last_error_message(h))
    return norm
