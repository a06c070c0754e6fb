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


def _check_state(p, m, v, s, i):
    if s is None:
        kinds = (torch.float32, torch.float32)
    else:
        kinds = (torch.float8_e4m3fn, torch.float8_e5m2)
        if s.dtype != torch.float8_e8m0fnu or not s.is_contiguous() or s.numel() != 2 * -(-p.numel() // STATE_BLOCK):
            raise ValueError(f"tensor {i}: scales must be a contiguous float8_e8m0fnu tensor with two entries per "
                             f"{STATE_BLOCK} elements")
    for t, kind, name in ((m, kinds[0], "m"), (v, kinds[1], "v")):
        if t.dtype != kind:
            raise ValueError(f"tensor {i}: {name} must be {kind}, got {t.dtype}")


def adamw_step(params, grads, ms, vs, scales=None, *, lr, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.0, step, seed=0,
               stream=None):
    """One AdamW step over lists of CUDA tensors on the current stream (or ``stream``).

    ``params`` (fp32 or bf16), ``ms`` and ``vs`` are updated in place; ``grads``
    (fp32 or bf16) are read.  The tensors of one entry must have the same number
    of elements in the same memory order without gaps.  ``scales`` is None for
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
    device = params[0].device
    if device.type != "cuda":
        raise ValueError(f"parameters must be CUDA tensors, got one on {device}")
    descs = (B.muon_adamw_desc * n)()
    for i in range(n):
        p, g, m, v = params[i], grads[i], ms[i], vs[i]
        s = scales[i] if scales is not None else None
        _check_state(p, m, v, s, i)
        size, stride = p.shape, p.stride()
        for t, name in ((p, "parameter"), (g, "gradient"), (m, "m"), (v, "v")):
            if t.device != device:
                raise ValueError(f"tensor {i}: {name} is on {t.device}, the first parameter on {device}")
            if t.shape != size or (t.stride() != stride and not (t.is_contiguous() and p.is_contiguous())):
                raise ValueError(f"tensor {i}: {name} must have its parameter's shape and strides")
        if s is not None and s.device != device:
            raise ValueError(f"tensor {i}: scales are on {s.device}, the first parameter on {device}")
        if not is_dense(p):
            raise ValueError(f"tensor {i}: a parameter must fill its memory without gaps, got shape {tuple(size)} with "
                             f"strides {stride}")
        if p.dtype not in _DTYPES or g.dtype not in _DTYPES:
            raise ValueError(f"tensor {i}: parameter and gradient must be bf16 or fp32, got {p.dtype} and {g.dtype}")
        d = descs[i]
        d.n = p.numel()
        d.P, d.G, d.M, d.V = p.data_ptr(), g.data_ptr(), m.data_ptr(), v.data_ptr()
        d.scales = s.data_ptr() if s is not None else None
        d.p_dtype, d.g_dtype, d.state_bits = _DTYPES[p.dtype], _DTYPES[g.dtype], 32 if s is None else 8
        d.step = step if isinstance(step, int) else step[i]
        d.seed = (seed + i) & 0xFFFFFFFFFFFFFFFF
        d.lr = lr if isinstance(lr, (int, float)) else lr[i]
        d.weight_decay = weight_decay if isinstance(weight_decay, (int, float)) else weight_decay[i]
    cfg = B.muon_adamw_config(betas[0], betas[1], eps)
    h = B.thread_handle(device.index)
    st = B.muon_adamw_step(h, cfg, ctypes.addressof(descs), n, _stream(device, stream))
    if st != B.MUON_OK:
        raise B.MuonError(st, B.muon_last_error_message(h))


def _stream(device, stream=None):
    return stream if stream is not None else torch.cuda.current_stream(device).cuda_stream


def _clip_desc(d, g, out, i):
    if g.dtype not in _DTYPES or out.dtype not in _DTYPES:
        raise ValueError(f"gradient {i}: gradients and outputs must be bf16 or fp32, got {g.dtype} and {out.dtype}")
    if g.shape != out.shape:
        raise ValueError(f"gradient {i}: the output must have its shape {tuple(g.shape)}, got {tuple(out.shape)}")
    if (g.stride() == out.stride() or (g.is_contiguous() and out.is_contiguous())) and is_dense(g):
        d.rows, d.cols, d.ldg, d.ldo = 1, g.numel(), g.numel(), g.numel()
    elif g.dim() == 2 and (g.stride(1) == 1 or g.shape[1] == 1) and (out.stride(1) == 1 or out.shape[1] == 1):
        d.rows, d.cols, d.ldg, d.ldo = g.shape[0], g.shape[1], g.stride(0), out.stride(0)
    else:
        raise ValueError(f"gradient {i}: a gradient must fill its memory without gaps, its output in the same order, "
                         "or both be matrices with unit column stride")
    d.G, d.out = g.data_ptr(), out.data_ptr()
    d.g_dtype, d.out_dtype = _DTYPES[g.dtype], _DTYPES[out.dtype]


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
    device = grads[0].device
    if device.type != "cuda":
        raise ValueError(f"gradients must be CUDA tensors, got one on {device}")
    descs = (B.muon_clip_desc * n)()
    for i in range(n):
        g = grads[i]
        out = outs[i] if outs is not None else g
        if g.device != device or out.device != device:
            raise ValueError(f"gradient {i}: all tensors must be on {device}")
        _clip_desc(descs[i], g, out, i)
    if stream is None:
        buf = torch.empty(B.MUON_CLIP_WORKSPACE_BYTES // 4 + 64, dtype=torch.float32, device=device)
    else:
        with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device)):
            buf = torch.empty(B.MUON_CLIP_WORKSPACE_BYTES // 4 + 64, dtype=torch.float32, device=device)
    norm = buf[-1]
    h = B.thread_handle(device.index)
    st = B.muon_clip_grads(h, ctypes.addressof(descs), n, float(max_norm), norm.data_ptr(), buf.data_ptr(),
                           B.MUON_CLIP_WORKSPACE_BYTES, _stream(device, stream))
    if st != B.MUON_OK:
        raise B.MuonError(st, B.muon_last_error_message(h))
    return norm
