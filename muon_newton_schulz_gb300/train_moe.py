"""A small mixture-of-experts language model trained with the framework's
operators, as they are used together:

    python -m muon_newton_schulz_gb300.train_moe [--steps 60] [--state-bits 8] [--gated [--saved-bits 8]]

Each step routes the tokens to the top 2 of 8 experts with capacity factor
1.25 (TorchTitan section 2.1), sorts and dispatches them, runs the experts as
batched matrix products, and combines their answers with the router's weights.
After the backward pass one call clips all gradients by their global norm and
writes the experts' in fp32, where the Muon step reads them; Muon then steps
the experts' matrices and AdamW the embedding, the head, the router and the
norm gain.  With --gated the experts are gated feed-forward blocks in the
framework's kernels, whose activations --saved-bits 8 keeps in 8 bits, and the
embedding is read, scaled and given its gradient by the framework too.  The data are synthetic: each token is followed by the next one of
a fixed random permutation, or, one time in ten, by any token.
"""
from __future__ import annotations

import argparse

import torch
import torch.nn.functional as F

from . import adamw, binding, moe
from .embedding import embed
from .ffn import check_status, gated_ffn
from .optim import AdamW


class MoELayer(torch.nn.Module):
    def __init__(self, hidden, ffn, experts, topk, capacity_factor=1.25, dtype=torch.bfloat16, gated=False, saved_bits=None):
        super().__init__()
        self.topk, self.experts, self.capacity_factor = topk, experts, capacity_factor
        self.gated, self.saved_bits = gated, saved_bits
        self.router = torch.nn.Parameter(torch.randn(experts, hidden) * hidden ** -0.5)
        self.gain = torch.nn.Parameter(torch.ones(hidden))
        if gated:      # each matrix as a linear layer has it: outputs x inputs
            self.gate = torch.nn.Parameter((torch.randn(experts, ffn, hidden) * hidden ** -0.5).to(dtype))
            self.up = torch.nn.Parameter((torch.randn(experts, ffn, hidden) * hidden ** -0.5).to(dtype))
            self.down = torch.nn.Parameter((torch.randn(experts, hidden, ffn) * ffn ** -0.5).to(dtype))
        else:
            self.up = torch.nn.Parameter((torch.randn(experts, hidden, ffn) * hidden ** -0.5).to(dtype))
            self.down = torch.nn.Parameter((torch.randn(experts, ffn, hidden) * ffn ** -0.5).to(dtype))

    def matrices(self):
        """The experts' parameters, which Muon steps."""
        return [self.gate, self.up, self.down] if self.gated else [self.up, self.down]

    def forward(self, x):
        """x: tokens x hidden, fp32."""
        tokens = x.shape[0]
        h = F.rms_norm(x, (x.shape[1],)) * self.gain
        top = (h @ self.router.t()).topk(self.topk, dim=1)
        weights = torch.softmax(top.values, dim=1)
        capacity = int(self.capacity_factor * tokens * self.topk / self.experts)
        capacity = max(8, -(-capacity // 8) * 8)
        route = moe.sort_tokens(top.indices, self.experts, capacity=capacity)
        xs = moe.dispatch(h.to(self.up.dtype), route)
        if self.gated:
            ys = gated_ffn(xs, self.gate, self.up, self.down, route, saved_bits=self.saved_bits)
            return x + moe.combine(ys, weights, route).float()
        xs = xs.view(self.experts, capacity, -1)
        ys = torch.bmm(F.gelu(torch.bmm(xs, self.up)), self.down)
        return x + moe.combine(ys.view(route.rows, -1), weights, route).float()


class Model(torch.nn.Module):
    def __init__(self, vocab=512, hidden=256, ffn=512, experts=8, topk=2, gated=False, saved_bits=None):
        super().__init__()
        self.gated = gated
        self.embedding = torch.nn.Parameter(torch.randn(vocab, hidden) * 0.5)
        self.layer = MoELayer(hidden, ffn, experts, topk, gated=gated, saved_bits=saved_bits)
        self.head = torch.nn.Parameter(torch.randn(vocab, hidden) * hidden ** -0.5)

    def forward(self, ids):
        x = embed(ids, self.embedding, scale=2.0) if self.gated else self.embedding[ids]
        return F.rms_norm(self.layer(x), (self.embedding.shape[1],)) @ self.head.t()


def train(steps=60, tokens=2048, state_bits=32, seed=0, device="cuda:0", log=None, gated=False, saved_bits=None):
    """Trains for ``steps`` steps and returns their losses (fp32, on the CPU)."""
    torch.manual_seed(seed)
    dev = torch.device(device)
    model = Model(gated=gated, saved_bits=saved_bits).to(dev)
    vocab = model.embedding.shape[0]
    follows = torch.randperm(vocab, device=dev)

    experts = model.layer.matrices()
    matrices = [w[e] for w in experts for e in range(w.shape[0])]                 # whole matrices, one per expert
    momenta = [torch.zeros(w.shape, dtype=torch.float32, device=dev) for w in matrices]
    grads32 = [torch.empty(w.shape, dtype=torch.float32, device=dev) for w in experts]
    muon = binding.MuonStep(dev.index)
    others = [p for p in model.parameters() if all(p is not w for w in experts)]
    adam = AdamW(others, lr=3e-3, weight_decay=0.01, state_bits=state_bits)

    losses = []
    for step in range(steps):
        ids = torch.randint(0, vocab, (tokens,), device=dev)
        noise = torch.randint(0, vocab, (tokens,), device=dev)
        target = torch.where(torch.rand(tokens, device=dev) < 0.9, follows[ids], noise)
        loss = F.cross_entropy(model(ids), target)
        loss.backward()
        norm = adamw.clip_grads([p.grad for p in experts + others], 1.0, outs=grads32 + [p.grad for p in others])
        with torch.no_grad():
            muon.step([w.detach() for w in matrices], [g[e] for g in grads32 for e in range(g.shape[0])], momenta,
                      [1e-2] * len(matrices))
        adam.step()
        model.zero_grad()
        losses.append(loss.detach())
        if log and (step % 10 == 0 or step == steps - 1):
            log(f"step {step:4d}  loss {float(losses[-1]):.4f}  gradient norm {float(norm):.3f}")
    status = muon.check_status()
    muon.close()
    if status != binding.MUON_OK:
        raise binding.MuonError(status, "a Muon step did not finish")
    status = check_status(dev) if gated else binding.MUON_OK
    if status != binding.MUON_OK:
        raise binding.MuonError(status, "an experts' feed-forward block did not finish")
    return torch.stack(losses).cpu()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--state-bits", type=int, choices=(32, 8), default=32)
    ap.add_argument("--seed", type=int, default=0)
    ap.add_argument("--gated", action="store_true")
    ap.add_argument("--saved-bits", type=int, choices=(8,))
    a = ap.parse_args(argv)
    if a.saved_bits and not a.gated:
        ap.error("--saved-bits goes with --gated")
    train(a.steps, a.tokens, a.state_bits, a.seed, log=print, gated=a.gated, saved_bits=a.saved_bits)


if __name__ == "__main__":
    main()
