"""The gated feed-forward block against its definition in float64.

Bounds.  u = 2^-24; a sum of k products in fp32 is off by at most (k + 2) u of its
terms' magnitudes; a rounding to bf16 by 2^-8 of the value (none in fp32).  The
activation's fp32 arithmetic is within c = 2^-18 of max(1, |g|), its first
derivative is at most 1.13 and its second at most 0.8 in magnitude.  Errors of
the inputs of a product go through it by magnitude.  The backward pass is held
against the formula on what the forward pass kept, so that bound has no rounding of
g, u and x in it; what was kept is held against g and u by itself.

Besides, in bf16 a result of 256 elements or more is held in the norm.  An operand's
rounding errors are independent of each other, each at most 2^-8 / sqrt(3) of its
term in the mean square, so that a sum of terms t is off by 2^-8 / sqrt(3) * sqrt(sum
of t^2) in the mean square for each operand that was rounded.  At most two were
(a product's two operands), and the result is: 2^-8 of the norm of sqrt(sum of
t^2), which is the result's own norm for terms of random signs.  Twice that is
allowed for."""
import threading

import numpy as np
import pytest
import torch
import torch.autograd.forward_ad as fwAD

import oracle.layer_oracle as L
from muon_newton_schulz_gb300 import binding as B
from muon_newton_schulz_gb300 import checkpoint, ffn, moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U, C = 2.0 ** -24, 2.0 ** -18
F32, BF16 = torch.float32, torch.bfloat16


def host(t):
    return t.detach().double().cpu().numpy()


class Case:
    """Inputs of a block, and their float64 copies."""

    def __init__(self, T, K, E, H, F, dtype, masked=0.0, capacity=0, align=1, seed=0, turned=False, skew=1.0):
        g = torch.Generator().manual_seed(seed + 1000 * T + 10 * H + F)
        self.dtype, self.E, self.H, self.F = dtype, E, H, F
        rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        if E:
            ids = (rand(T, E) + skew * rand(E)).topk(K, 1).indices if T else torch.zeros(0, K, dtype=torch.int64)
            if masked:
                ids[torch.rand(T, generator=g) < masked] = -1
            self.route = moe.sort_tokens(ids.to(DEV), E, capacity=capacity, align=align)
            self.rows = self.route.rows
            offsets, counts = self.route.offsets.cpu().numpy(), self.route.counts.cpu().numpy()
        else:
            self.route, self.rows = None, T
            offsets, counts = [0], [T]
        self.parts = L.ranges(offsets, counts, self.rows)
        self.used = np.zeros(self.rows, bool)
        for _, a, b in self.parts:
            self.used[a:b] = True
        many = (max(E, 1),)
        self.x = self._rows(rand(self.rows, H))
        self.dy = self._rows(rand(self.rows, H))
        w = [rand(*many, F, H) * max(H, 1) ** -0.5, rand(*many, F, H) * max(H, 1) ** -0.5, rand(*many, H, F) * max(F, 1) ** -0.5]
        if turned:
            w = [t.transpose(1, 2).contiguous().to(dtype).to(DEV).transpose(1, 2) for t in w]
        else:
            w = [t.to(dtype).to(DEV) for t in w]
        self.w64 = [host(t) for t in w]
        self.w = w if E else [t[0] for t in w]
        self.x64, self.dy64 = (np.where(self.used[:, None], host(t), 0.0) for t in (self.x, self.dy))
        self.wide = 2.0 ** -8 if dtype == BF16 else 0.0

    def _rows(self, t):
        """Rows without a token hold NaN: they must not be read."""
        t = torch.where(torch.from_numpy(self.used).unsqueeze(1), t, float("nan"))
        return t.to(self.dtype).to(DEV)

    def close(self, got, want, bound, name, spread):
        """spread: the roots of the sums of the terms' squares."""
        got = host(got)
        assert got.shape == want.shape, name
        assert np.isfinite(got).all(), name
        bound = bound + self.wide * (np.abs(want) + bound)
        assert (np.abs(got - want) <= bound).all(), (name, float((np.abs(got - want) - bound).max()))
        if self.wide and want.size >= 256:
            norm = max(np.linalg.norm(want), np.linalg.norm(spread))
            assert np.linalg.norm(got - want) <= 2 * self.wide * norm, (name, np.linalg.norm(got - want) / norm)


def mul(a, b):
    return a @ np.swapaxes(b, -1, -2)


def pre_of(c, saved, i):
    """g (i = 0) or u as they were kept in 16 or 32 bits."""
    pre = host(saved.kept[0][i])
    if c.wide:
        pre = pre * np.repeat(host(saved.kept[1][i].float()), 32, axis=1)
    return pre[:, : c.F]


def check_forward(c, act, y, saved=None, bits=None):
    gate, up, down = c.w64
    g, u, mg, mu = L.ffn_pre(c.x64, gate, up, c.parts)
    eg, eu = (c.H + 2) * U * mg, (c.H + 2) * U * mu
    a, _ = L.act(g, act)
    h = a * u
    # c of max(1, |g|) for the activation, and products of errors
    eh = (1.13 * eg + C * np.maximum(1, np.abs(g))) * (np.abs(u) + eu) + np.abs(a) * eu + U * np.abs(h)
    kept_h = eh + c.wide * (np.abs(h) + eh)
    absw = np.abs(down)
    bound = L.ffn_rows(kept_h, absw, c.parts, c.H) + (c.F + 2) * U * L.ffn_rows(np.abs(h) + kept_h, absw, c.parts, c.H)
    c.close(y, L.ffn_rows(h, down, c.parts, c.H), bound, "y", np.sqrt(L.ffn_rows(h * h, down * down, c.parts, c.H)))
    assert (host(y)[~c.used] == 0).all()
    if saved is None:
        return
    sel = c.used
    if bits is None:
        # fp16 numbers under a power of two are off by at most 2^-11 of themselves, or by 2^-25 of 2^-14 of the largest
        for got, want, e in ((pre_of(c, saved, 0), g, eg), (pre_of(c, saved, 1), u, eu)):
            nb = -(-c.F // 32)
            most = np.repeat(np.pad(np.abs(want), ((0, 0), (0, nb * 32 - c.F))).reshape(-1, nb, 32).max(2, initial=0), 32, 1)[:, : c.F]
            rounding = np.maximum(2.0 ** -11 * (np.abs(want) + e), 2.0 ** -39 * most) if c.wide else 0.0
            assert (np.abs(got - want)[sel] <= (e + rounding + 0 * e)[sel]).all()
        got = host(saved.kept[-1])[:, : c.F]
        assert (np.abs(got - h)[sel] <= (eh + c.wide * (np.abs(h) + eh))[sel]).all()
    else:
        pre, scales, xc, xs = saved.kept
        for got, s, want, e in ((pre[0], scales[0], g, eg), (pre[1], scales[1], u, eu)):
            got = host(checkpoint.unpack(checkpoint.Packed(got, s, F32)))[:, : c.F]
            nb = -(-c.F // 32)
            most = np.repeat(np.pad(np.abs(want), ((0, 0), (0, nb * 32 - c.F))).reshape(-1, nb, 32).max(2), 32, 1)[:, : c.F]
            assert (np.abs(got - want)[sel] <= (e + np.maximum(2.0 ** -4 * (np.abs(want) + e), 2.0 ** -16 * most))[sel]).all()


def check_backward(c, act, saved, bits, got):
    gate, up, down = c.w64
    sel = c.used[:, None]
    if bits is None:
        g, u, h = (np.where(sel, t, 0.0) for t in (pre_of(c, saved, 0), pre_of(c, saved, 1), host(saved.kept[-1])[:, : c.F]))
        x, eh = c.x64, 0.0
    else:
        pre, scales, xc, xs = saved.kept
        g, u = (np.where(sel, host(checkpoint.unpack(checkpoint.Packed(pre[i], scales[i], F32)))[:, : c.F], 0.0) for i in (0, 1))
        x = np.where(sel, host(checkpoint.unpack(checkpoint.Packed(xc, xs, F32))), 0.0) if c.H and c.rows else c.x64
        h = L.act(g, act)[0] * u
        eh = C * np.maximum(1, np.abs(g)) * np.abs(u)
        eh = eh + c.wide * (np.abs(h) + eh)
    a, s = L.act(g, act)
    dh = L.ffn_rows(c.dy64, np.swapaxes(down, 1, 2), c.parts, c.F)
    edh = (c.H + 2) * U * L.ffn_rows(np.abs(c.dy64), np.abs(np.swapaxes(down, 1, 2)), c.parts, c.F)
    ca = C * np.maximum(1, np.abs(g))
    dg, du = dh * u * s, dh * a
    edg = (np.abs(dh) + edh) * np.abs(u) * ca + edh * np.abs(u * s)
    edu = (np.abs(dh) + edh) * ca + edh * np.abs(a)
    edg, edu = (e + c.wide * (np.abs(v) + e) for e, v in ((edg, dg), (edu, du)))
    tg, tu = np.swapaxes(gate, 1, 2), np.swapaxes(up, 1, 2)
    dx = L.ffn_rows(dg, tg, c.parts, c.H) + L.ffn_rows(du, tu, c.parts, c.H)
    mag = lambda p, q: L.ffn_rows(p, np.abs(tg), c.parts, c.H) + L.ffn_rows(q, np.abs(tu), c.parts, c.H)  # noqa: E731
    ex = mag(edg, edu) + (2 * c.F + 4) * U * mag(np.abs(dg) + edg, np.abs(du) + edu)
    E = max(c.E, 1)
    n = max([b - a_ for _, a_, b in c.parts], default=0)
    W = lambda p, q: L.ffn_weight(p, q, c.parts, E)  # noqa: E731
    one = lambda t: t if c.E else t.unsqueeze(0)  # noqa: E731
    if got[0] is not None:
        c.close(got[0], dx, ex, "dx", np.sqrt(L.ffn_rows(dg * dg, tg * tg, c.parts, c.H) + L.ffn_rows(du * du, tu * tu, c.parts, c.H)))
        assert (host(got[0])[~c.used] == 0).all()
    for t, p, ep, q, eq, name in ((got[1], dg, edg, x, 0.0, "dgate"), (got[2], du, edu, x, 0.0, "dup"), (got[3], c.dy64, 0.0, h, eh, "ddown")):
        if t is None:
            continue
        zero = np.zeros_like
        ep, eq = ep + zero(p), eq + zero(q)
        bound = W(ep, np.abs(q)) + W(np.abs(p) + ep, eq) + (n + 2) * U * W(np.abs(p) + ep, np.abs(q) + eq)
        c.close(one(t), W(p, q), bound, name, np.sqrt(W(p * p, q * q)))


CASES = [  # T, K, E, H, F, masked, capacity, align
    (1, 1, 0, 8, 8, 0.0, 0, 1), (5, 1, 0, 64, 128, 0.0, 0, 1), (300, 1, 0, 136, 264, 0.0, 0, 1), (257, 1, 0, 1, 1, 0.0, 0, 1),
    (1, 2, 16, 256, 512, 0.0, 0, 1), (7, 2, 5, 96, 40, 0.3, 0, 16), (300, 2, 4, 256, 384, 0.0, 0, 1), (130, 2, 3, 201, 333, 0.1, 60, 1),
    (500, 1, 2, 512, 256, 0.0, 0, 128), (64, 8, 100, 72, 100, 0.0, 0, 1), (90, 4, 1000, 40, 24, 0.2, 0, 1), (1, 1, 1, 33, 65, 0.0, 3, 1),
    (700, 2, 4, 320, 448, 0.0, 200, 1), (20, 2, 4, 64, 64, 1.0, 0, 1), (0, 2, 3, 64, 64, 0.0, 0, 8), (33, 3, 7, 520, 130, 0.0, 0, 1),
]


@pytest.mark.parametrize("T, K, E, H, F, masked, capacity, align", CASES)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("act, bits, turned", [("silu", None, False), ("gelu", 8, False), ("silu", 8, True), ("gelu", None, True)])
def test_forward_and_backward(T, K, E, H, F, masked, capacity, align, dtype, act, bits, turned):
    c = Case(T, K, E, H, F, dtype, masked, capacity, align, turned=turned)
    y = ffn.gated_ffn(c.x, *c.w, c.route, activation=act)
    check_forward(c, act, y)
    y2, saved = ffn.gated_ffn_saved(c.x, *c.w, c.route, activation=act, saved_bits=bits)
    check_forward(c, act, y2, saved, bits)
    got = ffn.gated_ffn_backward(c.dy, saved, *c.w)
    check_backward(c, act, saved, bits, got)
    again = ffn.gated_ffn_backward(c.dy, saved, *c.w)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_no_width():
    for H, F in ((0, 8), (8, 0)):
        c = Case(6, 1, 2, H, F, F32)
        y, saved = ffn.gated_ffn_saved(c.x, *c.w, c.route)
        assert y.shape == (6, H) and (y == 0).all()
        dx, dg, du, dd = ffn.gated_ffn_backward(c.dy, saved, *c.w)
        assert (dx == 0).all() and dg.shape == du.shape == (2, F, H) and dd.shape == (2, H, F)


def test_sizes_at_every_edge_of_a_tile():
    """Row counts around 16, 32, 64, 128 and 256, with expert after expert in one buffer."""
    for n in (15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 385):
        for dtype in (F32, BF16):
            c = Case(2 * n, 1, 2, 72, 200, dtype, seed=n, skew=0.0)
            y, saved = ffn.gated_ffn_saved(c.x, *c.w, c.route)
            check_forward(c, "silu", y, saved)
            check_backward(c, "silu", saved, None, ffn.gated_ffn_backward(c.dy, saved, *c.w))


@pytest.mark.parametrize("H, F", [(64, 96), (72, 200), (512, 1040), (24, 16), (136, 2048), (65, 129)])
def test_a_few_rows(H, F):
    """Row counts around those that stream the weights, with widths of whole 32 and 16 bytes and others, a route with and
    without room, and one layer."""
    for T, K, E, capacity, align in ((1, 2, 4, 0, 1), (4, 2, 40, 0, 1), (8, 1, 1, 0, 1), (9, 1, 3, 0, 1), (16, 1, 2, 0, 1), (17, 1, 2, 0, 1),
                                     (3, 2, 4, 3, 1), (2, 1, 4, 0, 4), (1, 1, 0, 0, 1), (7, 1, 0, 0, 1), (16, 1, 0, 0, 1)):
        for act in ("silu", "gelu"):
            c = Case(T, K, E, H, F, BF16, capacity=capacity, align=align)
            check_forward(c, act, ffn.gated_ffn(c.x, *c.w, c.route, activation=act))


@pytest.mark.parametrize("T, K, E, H, F, capacity", [(17, 1, 0, 72, 2064, 0), (300, 1, 0, 264, 1100, 0), (90, 2, 3, 130, 3001, 0),
                                                     (60, 1, 2, 64, 8192, 50), (257, 1, 1, 33, 1030, 0), (40, 2, 6, 520, 1536, 0)])
@pytest.mark.parametrize("bits", [None, 8])
def test_shared_depth(T, K, E, H, F, capacity, bits):
    """Few tiles and long sums: pairs of CTAs share them, in y and in dx."""
    c = Case(T, K, E, H, F, BF16, capacity=capacity, masked=0.1 if capacity else 0.0)
    y, saved = ffn.gated_ffn_saved(c.x, *c.w, c.route, saved_bits=bits)
    check_forward(c, "silu", y, saved, bits)
    got = ffn.gated_ffn_backward(c.dy, saved, *c.w)
    check_backward(c, "silu", saved, bits, got)
    assert torch.equal(y, ffn.gated_ffn(c.x, *c.w, c.route))
    assert all(torch.equal(a, b) for a, b in zip(got, ffn.gated_ffn_backward(c.dy, saved, *c.w)))


@pytest.mark.parametrize("T, E, H, F, capacity, skew", [(6000, 2, 512, 768, 0, 0.0), (2500, 0, 520, 1160, 0, 0.0), (1500, 10, 1024, 1536, 0, 1.0),
                                                        (4000, 3, 264, 2048, 1100, 1.0)])
@pytest.mark.parametrize("act, bits, turned", [("silu", None, False), ("gelu", 8, True)])
def test_many_tiles(T, E, H, F, capacity, skew, act, bits, turned):
    """More rows of an expert than one walk over the columns takes (8 tiles of 256), and experts whose last tiles are of 128 rows
    or 256: pairs of CTAs have several tiles of either kind after one another, many steps deep."""
    c = Case(T, 1, E, H, F, BF16, capacity=capacity, skew=skew, turned=turned)
    rows = [b - a for _, a, b in c.parts]
    pairs, tiles = 76, sum(-(-n // 256) for n in rows)
    assert tiles * -(-F // 128) > pairs and (max(rows) > 2048 or any(0 < n % 256 <= 128 for n in rows))
    y, saved = ffn.gated_ffn_saved(c.x, *c.w, c.route, activation=act, saved_bits=bits)
    check_forward(c, act, y, saved, bits)
    check_backward(c, act, saved, bits, ffn.gated_ffn_backward(c.dy, saved, *c.w))
    assert torch.equal(y, ffn.gated_ffn(c.x, *c.w, c.route, activation=act))


def test_strided_inputs():
    c = Case(100, 2, 4, 64, 96, BF16)
    want = ffn.gated_ffn(c.x, *c.w, c.route)
    wide = torch.full((c.rows, 200), float("nan"), dtype=BF16, device=DEV)
    for at in (8, 3):
        x = wide[:, at: at + 64]
        x.copy_(c.x)
        assert torch.equal(ffn.gated_ffn(x, *c.w, c.route), want)
    both = torch.cat([c.w[0], c.w[1]], 1)                      # gate and up in one tensor
    assert torch.equal(ffn.gated_ffn(c.x, both[:, :96], both[:, 96:], c.w[2], c.route), want)
    odd = torch.zeros(4, 96, 71, dtype=BF16, device=DEV)
    odd[:, :, 5:69] = c.w[0]
    assert torch.equal(ffn.gated_ffn(c.x, odd[:, :, 5:69], c.w[1], c.w[2], c.route), want)
    shared = c.w[0][:1].expand(4, -1, -1)                      # one matrix for all experts
    assert torch.equal(ffn.gated_ffn(c.x, shared, c.w[1], c.w[2], c.route), ffn.gated_ffn(c.x, shared.contiguous(), c.w[1], c.w[2], c.route))
    assert torch.equal(ffn.gated_ffn(c.x.t().contiguous().t(), *c.w, c.route), want)
    other_way = c.w[1].transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(ffn.gated_ffn(c.x, c.w[0], other_way, c.w[2], c.route), want)
    between = torch.stack([*c.w[0]], 1).transpose(0, 1)        # an expert's rows between the others'
    assert torch.equal(ffn.gated_ffn(c.x, between, c.w[1], c.w[2], c.route), want)


def test_values_that_are_not_finite_stay_with_their_expert():
    for dtype in (F32, BF16):
        c = Case(200, 1, 4, 64, 64, dtype)
        x, dy = c.x.clone(), c.dy.clone()
        e1, a1, b1 = max(c.parts, key=lambda part: part[2] - part[1])      # both rows are this expert's
        x[a1, 3], dy[a1 + 1, 4] = float("nan"), float("inf")
        y, saved = ffn.gated_ffn_saved(x, *c.w, c.route)
        dx, dg, du, dd = ffn.gated_ffn_backward(dy, saved, *c.w)
        others = torch.from_numpy(c.used).to(DEV)
        others[a1: a1 + 2] = False
        assert torch.isnan(y[a1]).all() and torch.isfinite(y[others]).all() and torch.isfinite(dx[others]).all()
        for t in (dg, du, dd):
            keep = [e for e in range(4) if e != e1]
            assert torch.isfinite(t[keep]).all() and not torch.isfinite(t[e1]).all()


def test_autograd_against_formula_and_differences():
    c = Case(40, 2, 3, 24, 40, F32, masked=0.2)
    g = torch.Generator().manual_seed(3)
    x = torch.where(torch.from_numpy(c.used).to(DEV).unsqueeze(1), c.x, 0.0).requires_grad_()
    w = [t.clone().requires_grad_() for t in c.w]
    out = torch.randn(c.rows, 24, generator=g).to(DEV)

    def f(x, w):
        return (ffn.gated_ffn(x, *w, c.route, activation="gelu").double() * out).sum()

    f(x, w).backward()
    y, saved = ffn.gated_ffn_saved(x.detach(), *c.w, c.route, activation="gelu")
    dy = torch.where(torch.from_numpy(c.used).to(DEV).unsqueeze(1), out, 0.0)
    for a, b in zip((x.grad, *(t.grad for t in w)), ffn.gated_ffn_backward(dy, saved, *c.w)):
        assert torch.equal(a, b)
    # against differences along a direction of all inputs: halving the step quarters what is left of a smooth function's error
    d = [torch.randn(t.shape, generator=g).to(DEV) * 0.5 for t in (x, *w)]
    slope = sum(float((t.grad.double() * e).sum()) for t, e in zip((x, *w), d))

    def central(step):
        at = lambda s: [t.detach() + s * step * e for t, e in zip((x, *w), d)]  # noqa: E731
        with torch.no_grad():
            p, m = at(1), at(-1)
            return float(f(p[0], p[1:]) - f(m[0], m[1:])) / (2 * step)

    a, b = central(2.0 ** -6), central(2.0 ** -7)
    best = b + (b - a) / 3
    terms = float((y.abs() * out.abs()).sum())
    noise = 2 ** 7 * (40 + 24 + 30) * U * terms            # fp32 sums on both sides, divided by the step
    assert abs(best - slope) <= abs(b - a) / 3 + noise


def test_some_gradients_only():
    c = Case(60, 2, 3, 64, 96, BF16)
    x = torch.where(torch.from_numpy(c.used).to(DEV).unsqueeze(1), c.x, 0.0)
    y, saved = ffn.gated_ffn_saved(x, *c.w, c.route)
    all_of = ffn.gated_ffn_backward(y, saved, *c.w)
    for i in range(4):
        inputs = [t.detach().clone().requires_grad_(i == j) for j, t in enumerate((x, *c.w))]
        ffn.gated_ffn(*inputs, c.route).backward(y)
        for j, t in enumerate(inputs):
            assert (t.grad is None) == (i != j)
            if i == j:
                assert torch.equal(t.grad, all_of[i])


def test_refusals_on_the_device():
    c = Case(20, 2, 3, 64, 96, BF16)
    gate, up, down = c.w
    for bad in (lambda: ffn.gated_ffn(c.x, gate, up, down), lambda: ffn.gated_ffn(c.x[:, :32], gate, up, down, c.route),
                lambda: ffn.gated_ffn(c.x, gate, up, up, c.route), lambda: ffn.gated_ffn(c.x, gate.float(), up, down, c.route),
                lambda: ffn.gated_ffn(c.x.half(), gate.half(), up.half(), down.half(), c.route),
                lambda: ffn.gated_ffn(c.x[:-1], gate, up, down, c.route), lambda: ffn.gated_ffn(c.x, gate[:2], up[:2], down[:2], c.route),
                lambda: ffn.gated_ffn(c.x, gate, up, down, c.route, activation="relu"),
                lambda: ffn.gated_ffn(c.x, gate, up, down, c.route, saved_bits=4),
                lambda: ffn.gated_ffn(c.x, gate.cpu(), up, down, c.route)):
        with pytest.raises(ValueError):
            bad()
    y, saved = ffn.gated_ffn_saved(c.x, *c.w, c.route)
    for bad in (lambda: ffn.gated_ffn_backward(c.dy.float(), saved, *c.w), lambda: ffn.gated_ffn_backward(c.dy[1:], saved, *c.w),
                lambda: ffn.gated_ffn_backward(c.dy, saved, gate[:, :64], up[:, :64], down[:, :, :64])):
        with pytest.raises(ValueError):
            bad()
    with fwAD.dual_level():
        dual = fwAD.make_dual(c.x, c.x)
        for bad in (lambda: ffn.gated_ffn(dual, *c.w, c.route), lambda: ffn.gated_ffn_saved(dual, *c.w, c.route),
                    lambda: ffn.gated_ffn_backward(dual, saved, *c.w)):
            with pytest.raises(RuntimeError, match="forward-mode"):
                bad()


@pytest.mark.parametrize("T, K, E, H, F", [(1, 2, 4, 256, 512), (8, 1, 0, 64, 96), (7, 2, 3, 72, 200), (16, 1, 0, 136, 1040), (5, 1, 2, 65, 129)])
def test_a_few_rows_round_once(T, K, E, H, F):
    """Up to 16 rows in bf16: h is a sum of two bf16 terms, off by 2^-8 of 2^-8 of itself, and y alone is rounded."""
    for act in ("silu", "gelu"):
        c = Case(T, K, E, H, F, BF16)
        gate, up, down = c.w64
        g, u, mg, mu = L.ffn_pre(c.x64, gate, up, c.parts)
        eg, eu = (H + 2) * U * mg, (H + 2) * U * mu
        a, _ = L.act(g, act)
        h = a * u
        eh = (1.13 * eg + C * np.maximum(1, np.abs(g))) * (np.abs(u) + eu) + np.abs(a) * eu + 2.0 ** -16 * np.abs(h)
        want = L.ffn_rows(h, down, c.parts, H)
        # twice as many terms
        bound = L.ffn_rows(eh, np.abs(down), c.parts, H) + (2 * F + 4) * U * L.ffn_rows(np.abs(h) + eh, np.abs(down), c.parts, H)
        y = host(ffn.gated_ffn(c.x, *c.w, c.route, activation=act))
        assert (np.abs(y - want) <= bound + 2.0 ** -8 * (np.abs(want) + bound)).all()


def test_a_few_rows_that_are_not_finite():
    """An h beyond bf16's range is infinite, as in more rows, and leaves no NaN of its own."""
    n = 64
    x, gate, up, down = (torch.zeros(s, n, dtype=BF16, device=DEV) for s in (2, n, n, n))
    x[:, 0], gate[0, 0], up[0, 0], down[3, 0] = 1.0, 3e38, 3e38, 0.5
    x[1, 0] = -1.0                           # silu(-3e38) is 0, and 0 times -3e38
    y = ffn.gated_ffn(x, gate, up, down)
    many = ffn.gated_ffn(x.repeat(20, 1), gate, up, down)
    assert y[0, 3] == many[0, 3] == float("inf") and torch.isfinite(y[1]).all() and torch.equal(y[1], many[1])


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows", [2, 40])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_the_activation_s_tail(act, rows, dtype):
    """Each element of y and of dup is one act(g) by itself, for g from -12 to 12: x is 1 in its first column, gate holds g there,
    up 1, and down is the identity.  In bf16 one rounding (h; what follows are sums of one term that are exact) and exponentials
    within 2^-14 of themselves; in fp32 g^2 / 2 enters an exponential with four roundings, and four more factors."""
    n = 256
    g = torch.linspace(-12, 12, n).to(dtype)
    x, gate, up = torch.zeros(rows, 8, dtype=dtype), torch.zeros(n, 8, dtype=dtype), torch.zeros(n, 8, dtype=dtype)
    x[:, 0], gate[:, 0], up[:, 0] = 1, g, 1
    down = torch.eye(n, dtype=dtype)
    pad = torch.zeros(n, n, dtype=dtype)                 # hidden is n wide: x, gate and up have zeros behind
    wide = [torch.cat([t, pad[: t.shape[0], 8:]], 1).to(DEV) for t in (x, gate, up)]
    w = [*wide[1:], down.to(DEV)]
    want, _ = L.act(host(g), act)
    rel = 2.0 ** -8 + 2.0 ** -14 if dtype == BF16 else (4 * host(g) ** 2 + 16) * U
    tiny = 2.0 ** -126
    y = host(ffn.gated_ffn(wide[0], *w, activation=act))
    assert (np.abs(y - want) <= rel * np.abs(want) + tiny).all(), float((np.abs(y - want) / np.abs(want)).max())
    _, saved = ffn.gated_ffn_saved(wide[0], *w, activation=act)
    dy = torch.zeros(rows, n, dtype=dtype, device=DEV)
    dy[1] = 1                                            # dh is 1 in one row: dup is du times 1
    dup = host(ffn.gated_ffn_backward(dy, saved, *w)[2])[:, 0]
    assert (np.abs(dup - want) <= rel * np.abs(want) + tiny).all(), float((np.abs(dup - want) / np.abs(want)).max())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T, E, H, F", [(60, 2, 40, 333), (60, 0, 24, 300), (1, 0, 33, 1), (3000, 0, 72, 1700), (50, 3, 64, 130)])
def test_what_is_kept_holds_no_stale_memory(T, E, H, F, dtype):
    """Whoever reads what is kept as a tensor (a hook that packs it, by blocks that reach over the width) sees zeros behind it,
    whatever the memory held before."""
    c = Case(T, 1, E, H, F, dtype)
    for junk in (1e30, float("nan")):
        stale = [torch.full((c.rows * n,), junk, device=DEV) for n in (128, 384, 768, 2048, 4096) for _ in range(3)]
        torch.cuda.synchronize()
        del stale
        _, saved = ffn.gated_ffn_saved(c.x, *c.w, c.route)
        used = torch.from_numpy(c.used).to(DEV)
        assert saved.kept[0].shape[-1] % 128 == 0 and saved.kept[-1].shape[-1] % 128 == 0
        assert (saved.kept[0][:, used, F:] == 0).all() and (saved.kept[-1][used, F:] == 0).all()


def test_gradients_inside_saved_in_8_bits_do_not_depend_on_stale_memory():
    """300 rows of an odd width in fp32, all of them tokens."""
    c = Case(300, 1, 0, 201, 333, F32)
    out = []
    for junk in (1e30, 0.0):
        stale = [torch.full((n,), junk, device=DEV) for n in (300 * 384, 2 * 300 * 384, 300 * 201, 300 * 1000) for _ in range(3)]
        torch.cuda.synchronize()
        del stale
        leaves = [t.clone().requires_grad_() for t in (c.x, *c.w)]
        with checkpoint.saved_in_8_bits(min_elements=1):
            y = ffn.gated_ffn(leaves[0] * 1.0, *leaves[1:])
        y.backward(c.dy)
        out.append([t.grad for t in leaves])
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_a_changed_input_is_noticed():
    c = Case(20, 2, 3, 64, 96, BF16)
    x = torch.where(torch.from_numpy(c.used).to(DEV).unsqueeze(1), c.x, 0.0)
    w = [t.clone().requires_grad_() for t in c.w]
    y = ffn.gated_ffn(x, *w, c.route)
    with torch.no_grad():
        w[1].add_(1)
    with pytest.raises(RuntimeError, match="modified"):
        y.sum().backward()


@pytest.mark.parametrize("bits", [None, 8])
def test_a_changed_route_is_noticed(bits):
    """A route's tensors are the caller's: the backward pass needs them as the forward pass had them."""
    c = Case(20, 2, 3, 64, 96, BF16)
    x = torch.where(torch.from_numpy(c.used).to(DEV).unsqueeze(1), c.x, 0.0)
    for name in ("offsets", "counts"):
        route = moe.Route(c.route.row.clone(), c.route.offsets.clone(), c.route.counts.clone())
        w = [t.clone().requires_grad_() for t in c.w]
        y = ffn.gated_ffn(x, *w, route, saved_bits=bits)
        _, saved = ffn.gated_ffn_saved(x, *c.w, route, saved_bits=bits)
        getattr(route, name).mul_(1)
        with pytest.raises(RuntimeError, match="modified"):
            y.sum().backward()
        with pytest.raises(RuntimeError, match="modified"):
            ffn.gated_ffn_backward(c.dy, saved, *c.w)


def test_a_changed_input_of_a_saved_pass_is_noticed():
    c = Case(20, 1, 0, 64, 96, BF16)
    for bits in (None, 8):
        x = c.x.clone()
        _, saved = ffn.gated_ffn_saved(x, *c.w, saved_bits=bits)
        want = ffn.gated_ffn_backward(c.dy, saved, *c.w)
        x.mul_(2)
        if bits == 8:                            # x itself is not kept
            assert all(torch.equal(a, b) for a, b in zip(want, ffn.gated_ffn_backward(c.dy, saved, *c.w)))
        else:
            with pytest.raises(RuntimeError, match="modified"):
                ffn.gated_ffn_backward(c.dy, saved, *c.w)
    with torch.inference_mode():
        y, saved = ffn.gated_ffn_saved(c.x.clone(), *c.w)
        assert all(torch.isfinite(t).all() for t in ffn.gated_ffn_backward(c.dy, saved, *c.w))


def test_routes_that_name_rows_outside_the_buffer():
    """Such rows are left out, as the token operators do."""
    for dtype in (F32, BF16):
        c = Case(64, 1, 2, 64, 64, dtype, skew=0.0)
        n = c.rows
        counts = torch.tensor([n - 8, 500], dtype=torch.int32, device=DEV)
        offsets = torch.tensor([0, n - 8, n], dtype=torch.int32, device=DEV)
        r = moe.Route(c.route.row, offsets, counts)
        y, saved = ffn.gated_ffn_saved(c.x, *c.w, r)
        right = moe.Route(c.route.row, offsets, torch.tensor([n - 8, 8], dtype=torch.int32, device=DEV))
        assert torch.equal(y, ffn.gated_ffn(c.x, *c.w, right))
        got = ffn.gated_ffn_backward(c.dy, saved, *c.w)
        _, saved = ffn.gated_ffn_saved(c.x, *c.w, right)
        assert all(torch.equal(a, b) for a, b in zip(got, ffn.gated_ffn_backward(c.dy, saved, *c.w)))


def test_captured_and_replayed():
    c = Case(200, 2, 4, 128, 192, BF16)
    x = torch.where(torch.from_numpy(c.used).to(DEV).unsqueeze(1), c.x, 0.0)
    dy = torch.where(torch.from_numpy(c.used).to(DEV).unsqueeze(1), c.dy, 0.0)

    def step():
        y, saved = ffn.gated_ffn_saved(x, *c.w, c.route)
        y8, saved8 = ffn.gated_ffn_saved(x, *c.w, c.route, saved_bits=8)
        return (ffn.gated_ffn(x, *c.w, c.route), y, y8, *ffn.gated_ffn_backward(dy, saved, *c.w), *ffn.gated_ffn_backward(dy, saved8, *c.w))

    step()
    torch.cuda.synchronize()
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    with torch.cuda.graph(other, pool=graph.pool()):
        out2 = step()
    for seed in range(3):
        x.mul_(0.9)
        dy.mul_(1.1)
        graph.replay()
        want = [t.clone() for t in out]
        other.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, out2))
        assert all(torch.equal(a, b) for a, b in zip(want, step()))


@pytest.mark.parametrize("T, E, H, F, bits", [(539, 5, 201, 333, None), (900, 0, 520, 24, None), (60, 3, 24, 700, 8), (2000, 4, 256, 512, None)])
def test_a_chain_in_fp32(T, E, H, F, bits):
    """Each call reads what the one before it wrote last, or writes what it read, with nothing between them."""
    c = Case(T, min(2, max(E, 1)) if E else 1, E, H, F, F32)

    def chain(pause):
        x, out = c.x, []
        for _ in range(4):
            y, saved = ffn.gated_ffn_saved(x, *c.w, c.route, saved_bits=bits)
            pause()
            first = ffn.gated_ffn_backward(c.dy, saved, *c.w)
            pause()
            second = ffn.gated_ffn_backward(first[0], saved, *c.w)
            pause()
            out += [y, *first, *second]
            x = second[0]
        return out

    want = [t.clone() for t in chain(torch.cuda.synchronize)]
    assert all(torch.equal(a, b) for a, b in zip(chain(lambda: None), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(lambda: None)
    for _ in range(3):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# tiles of 64 or 128 for the input's gradient and for the weights', and depths that are shared by some CTAs or by none
@pytest.mark.parametrize("T, E, H, F", [(3000, 0, 1000, 1100), (4000, 0, 640, 640), (300, 8, 640, 640), (40, 2, 24, 2000), (1500, 1, 70, 40)])
def test_gradients_of_the_input_and_the_weights_together_and_alone(T, E, H, F):
    c = Case(T, 1, E, H, F, F32, align=16 if E else 1)
    _, saved = ffn.gated_ffn_saved(c.x, *c.w, c.route)
    got = ffn.gated_ffn_backward(c.dy, saved, *c.w)
    check_backward(c, "silu", saved, None, got)
    for which in ((0,), (1, 2, 3)):     # how a sum is cut up goes by the tiles of the weights that are asked for
        want = ffn._backward(c.dy, saved.x, *c.w, saved.kept, c.route, "silu", 32, sum(1 << i for i in which))
        assert all((t is not None) == (i in which) for i, t in enumerate(want)) and all(torch.equal(want[i], got[i]) for i in which)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = ffn.gated_ffn_backward(c.dy, ffn.gated_ffn_saved(c.x, *c.w, c.route)[1], *c.w)
    for _ in range(3):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_threads_and_streams():
    c = Case(300, 2, 4, 128, 192, BF16)
    y, saved = ffn.gated_ffn_saved(c.x, *c.w, c.route)
    want = (y, *ffn.gated_ffn_backward(c.dy, saved, *c.w))
    torch.cuda.synchronize()
    bad = []

    def work():
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    y, s = ffn.gated_ffn_saved(c.x, *c.w, c.route)
                    got = (y, *ffn.gated_ffn_backward(c.dy, s, *c.w))
                    if not all(torch.equal(a, b) for a, b in zip(got, want)):
                        bad.append("differs")
        except Exception as e:  # pragma: no cover
            bad.append(repr(e))

    threads = [threading.Thread(target=work) for _ in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad


def test_a_block_between_dispatch_and_combine():
    """Tokens through experts and back, against the sum over each token's choices in float64."""
    T, K, E, H, F = 90, 2, 4, 64, 96
    g = torch.Generator().manual_seed(11)
    ids = torch.randn(T, E, generator=g).topk(K, 1).indices
    ids[::9] = -1
    x = torch.randn(T, H, generator=g).to(BF16)
    weights = torch.softmax(torch.randn(T, K, generator=g), 1)
    w = [(torch.randn(E, a, b, generator=g) * b ** -0.5).to(BF16) for a, b in ((F, H), (F, H), (H, F))]
    for capacity, bits in ((0, None), (30, 8)):
        leaves = [t.to(DEV).requires_grad_() for t in (x, weights, *w)]
        route = moe.sort_tokens(ids.to(DEV), E, capacity=capacity)
        rows = ffn.gated_ffn(moe.dispatch(leaves[0], route), *leaves[2:], route, saved_bits=bits)
        out = moe.combine(rows, leaves[1], route)
        row = route.row.cpu().numpy()
        want = np.zeros((T, H))
        for t in range(T):
            for k in range(K):
                if row[t, k] < 0:
                    continue
                gate, up, down = (host(m)[ids[t, k]] for m in w)
                a, _ = L.act(gate @ host(x)[t], "silu")
                want[t] += float(weights[t, k]) * (down @ (a * (up @ host(x)[t])))
        # three roundings in a row (h, y and the sum), independent of each other: 2 * 2^-8 in the norm
        assert np.linalg.norm(host(out) - want) <= 2 * 2.0 ** -8 * np.linalg.norm(want)
        out.float().square().sum().backward()
        assert all(t.grad is not None and torch.isfinite(t.grad).all() and t.grad.abs().sum() > 0 for t in leaves)
