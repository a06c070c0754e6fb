"""Batched Muon optimizer step (momentum, Frobenius normalisation, five
Newton-Schulz iterations on upper-triangle Gram tiles, scaled weight update)
as hand-written sm_103a CUDA kernels behind a C ABI.

``binding`` marshals arguments to the shared library; ``workloads`` draws the
seeded synthetic inputs; ``adamw`` (AdamW and gradient clipping) and ``moe``
(tokens by expert) are what a training step needs around the Muon step.  The library is loaded on first use and its absence
is an error, never a fallback.
"""
from . import adamw, binding, moe, workloads  # noqa: F401

__all__ = ["adamw", "binding", "moe", "workloads"]
