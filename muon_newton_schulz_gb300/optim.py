"""``torch.optim.Optimizer`` front ends for the library's Muon and AdamW steps,
and gradient clipping for both.

``Muon`` takes a model's matrices.  Every 2-D parameter with a gradient
becomes one matrix of one ragged batch, and one ``muon_step`` call per
``step()`` runs the momentum update, the Newton-Schulz orthogonalisation and
the weight update for all of them in the library's kernels (EU-1T,
optimizer-state paragraph: Muon on whole matrices with one fp32 momentum
state; ZAYA1/MI300X section 4.3: the update scale 0.2 * sqrt(max(rows, cols))
times the learning rate).

Parameters stay where they are: bf16 or fp32, row-major (unit column
stride), all on one CUDA device.  Each keeps an fp32 momentum buffer in the
optimizer state (``state[p]["momentum_buffer"]``).  The library reads
gradients in fp32; a gradient of another dtype (a bf16 parameter's is bf16)
or layout is first copied into an fp32 buffer kept in the state.

``AdamW`` takes the parameters that Muon leaves out: embeddings, LM head,
router and norms (ZAYA1/MI300X section 4.3), of any shape, all in one launch,
with its states in fp32 or in 8 bits.
"""
from __future__ import annotations

import torch

from . import adamw as A
from . import binding as B


class Muon(torch.optim.Optimizer):
    """Muon on 2-D parameters.

    ``lr`` may differ per parameter group.  ``beta``, ``nesterov``,
    ``dampening``, ``ns_iters``, the Newton-Schulz coefficients ``(a, b, c)``,
    ``eps`` and ``scale_coeff`` are fixed for the optimizer (the library's
    handle is configured once).  Raises ValueError for a parameter that is
    not a 2-D bf16 / fp32 CUDA tensor with unit column stride, or for
    parameters on more than one device."""

    def __init__(self, params, lr: float = 2e-4, beta: float = 0.95, nesterov: bool = False,
                 dampening: bool = False, ns_iters: int = 5, a: float = 3.4445, b: float = -4.7750,
                 c: float = 2.0315, eps: float = 1e-7, scale_coeff: float = 0.2):
        if not lr >= 0.0:
            raise ValueError(f"invalid learning rate {lr}")
        super().__init__(params, dict(lr=lr))
        devices = set()
        for group in self.param_groups:
            for p in group["params"]:
                if p.dim() != 2:
                    raise ValueError(f"Muon steps 2-D parameters only, got shape {tuple(p.shape)}")
                if p.dtype not in (torch.bfloat16, torch.float32):
                    raise ValueError(f"parameters must be bf16 or fp32, got {p.dtype}")
                if p.device.type != "cuda":
                    raise ValueError(f"parameters must be CUDA tensors, got one on {p.device}")
                if p.stride(1) != 1:
                    raise ValueError("parameters must have unit column stride (row-major)")
                devices.add(p.device.index)
        if len(devices) > 1:
            raise ValueError(f"parameters on more than one device: {sorted(devices)}")
        device = devices.pop() if devices else torch.cuda.current_device()
        self._muon = B.MuonStep(device, beta=beta, a=a, b=b, c=c, eps=eps, scale_coeff=scale_coeff,
                                ns_iters=ns_iters, nesterov=nesterov, dampening=dampening)

    @torch.no_grad()
    def step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        Ws, Gs, Ms, lrs = [], [], [], []
        for group in self.param_groups:
            for p in group["params"]:
                if p.grad is None:
                    continue
                state = self.state[p]
                if "momentum_buffer" not in state:
                    state["momentum_buffer"] = torch.zeros(p.shape, dtype=torch.float32, device=p.device)
                g = p.grad
                if g.dtype != torch.float32 or g.stride(1) != 1:
                    buf = state.get("grad_fp32")
                    if buf is None:
                        buf = state["grad_fp32"] = torch.empty(p.shape, dtype=torch.float32, device=p.device)
                    buf.copy_(g)
                    g = buf
                Ws.append(p)
                Gs.append(g)
                Ms.append(state["momentum_buffer"])
                lrs.append(group["lr"])
        if Ws:
            self._muon.step(Ws, Gs, Ms, lrs)
        return loss

    def check_status(self) -> int:
        """Synchronises the current stream and returns MUON_OK, or
        MUON_ERR_TIMEOUT if a kernel of an earlier step gave up a bounded
        wait (that step left W unchanged if the time-out came before its last
        kernel started)."""
        return self._muon.check_status()


class AdamW(torch.optim.Optimizer):
    """AdamW on parameters of any shape: fp32 or bf16, all on one CUDA device,
    each without gaps in its memory.

    ``lr``, ``weight_decay``, ``betas`` and ``eps`` may differ per parameter
    group; groups with the same betas and eps share a launch.  With
    ``state_bits=8`` a parameter of at least ``min_8bit_size`` elements keeps its
    two moments in 8 bits (``state[p]["scales"]`` holds the scales of their
    blocks; ``adamw.state8_values`` gives their values); smaller ones keep fp32.
    ``seed`` starts the random numbers of the 8-bit rounding.  A gradient is
    fp32 or bf16; one whose layout differs from its parameter's is copied
    first.  ``step()`` cannot be captured in a CUDA graph: the step number is
    counted on the host, and every replay would repeat the captured one."""

    def __init__(self, params, lr: float = 2e-4, betas=(0.9, 0.95), eps: float = 1e-8, weight_decay: float = 0.1,
                 state_bits: int = 32, min_8bit_size: int = 4096, seed: int = 0):
        if not lr >= 0.0:
            raise ValueError(f"invalid learning rate {lr}")
        if not (0.0 <= betas[0] < 1.0 and 0.0 <= betas[1] < 1.0):
            raise ValueError(f"betas must be in [0, 1), got {betas}")
        if not eps >= 0.0:
            raise ValueError(f"invalid eps {eps}")
        if state_bits not in (32, 8):
            raise ValueError(f"state_bits must be 32 or 8, got {state_bits}")
        super().__init__(params, dict(lr=lr, betas=tuple(betas), eps=eps, weight_decay=weight_decay))
        self.state_bits, self.min_8bit_size, self.seed = state_bits, min_8bit_size, seed
        devices = set()
        for group in self.param_groups:
            for p in group["params"]:
                if p.dtype not in (torch.bfloat16, torch.float32):
                    raise ValueError(f"parameters must be bf16 or fp32, got {p.dtype}")
                if p.device.type != "cuda":
                    raise ValueError(f"parameters must be CUDA tensors, got one on {p.device}")
                if not A.is_dense(p):
                    raise ValueError(f"a parameter must fill its memory without gaps, got shape {tuple(p.shape)} with "
                                     f"strides {p.stride()}")
                devices.add(p.device.index)
        if len(devices) > 1:
            raise ValueError(f"parameters on more than one device: {sorted(devices)}")

    def _new_state(self, p):
        if self.state_bits == 8 and p.numel() >= self.min_8bit_size:
            m, v, scales = A.state8_like(p)
            return dict(step=0, exp_avg=m, exp_avg_sq=v, scales=scales)
        return dict(step=0, exp_avg=torch.zeros_like(p, dtype=torch.float32),
                    exp_avg_sq=torch.zeros_like(p, dtype=torch.float32))

    @torch.no_grad()
    def step(self, closure=None):
        first = next((p for group in self.param_groups for p in group["params"]), None)
        if first is not None and B.stream_is_capturing(first.get_device()):
            raise RuntimeError("AdamW.step() cannot be captured in a CUDA graph: each replay would repeat the captured "
                               "step, its bias corrections and its random bits")
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        calls = {}
        index = -1
        for group in self.param_groups:
            call = calls.setdefault((tuple(group["betas"]), group["eps"]), tuple([] for _ in range(9)))
            for p in group["params"]:
                index += 1
                g = p.grad
                if g is None:
                    continue
                state = self.state[p]
                if not state:
                    state.update(self._new_state(p))
                if g.stride() != p.stride():
                    g = torch.empty_like(p, dtype=g.dtype).copy_(g)
                for to, x in zip(call, (p, g, state["exp_avg"], state["exp_avg_sq"], state.get("scales"), group["lr"],
                                        group["weight_decay"], state["step"] + 1, self.seed + index)):
                    to.append(x)
        for (betas, eps), (ps, gs, ms, vs, scales, lrs, decays, steps, seeds) in calls.items():
            A.adamw_step(ps, gs, ms, vs, scales, lr=lrs, betas=betas, eps=eps, weight_decay=decays, step=steps,
                         seed=seeds)
            for p in ps:
                self.state[p]["step"] += 1
        return loss

    def load_state_dict(self, state_dict):
        super().load_state_dict(state_dict)
        # the base class has cast the moments to their parameters' type: take them as they were saved
        ids = [i for group in state_dict["param_groups"] for i in group["params"]]
        params = [p for group in self.param_groups for p in group["params"]]
        for i, p in zip(ids, params):
            for name, x in state_dict["state"].get(i, {}).items():
                self.state[p][name] = x.to(p.device, copy=True) if isinstance(x, torch.Tensor) else x


def clip_grad_norm(parameters, max_norm: float) -> torch.Tensor:
    """Scales the gradients of the parameters (tensors, or one tensor) in place
    so that their global norm is at most ``max_norm``; returns the norm before
    (0-dim, on the parameters' device: the host does not wait)."""
    parameters = [parameters] if isinstance(parameters, torch.Tensor) else list(parameters)
    grads = [p.grad for p in parameters if p.grad is not None]
    if not grads:
        return torch.zeros((), dtype=torch.float32, device=parameters[0].device if parameters else None)
    return A.clip_grads(grads, max_norm)
