"""Plain numpy definitions of the operators of a model's layers, for the tests:
embedding rows and their gradient, activations in 8 bits.  float64 throughout;
8-bit codes are reproduced bit for bit."""
from __future__ import annotations

import numpy as np

from oracle.train_oracle import E4M3

BLOCK = 32


# ---- embedding

def embed(ids, table, scale):
    out = np.zeros((ids.size, table.shape[1]))
    for t, v in enumerate(ids.reshape(-1).tolist()):
        if 0 <= v < table.shape[0]:
            out[t] = table[v].astype(np.float64) * scale
    return out.reshape(*ids.shape, table.shape[1])


def embed_backward(dout, ids, vocab, scale):
    """float64 gradient, and the sums of the terms' magnitudes (for error bounds)."""
    h = dout.shape[-1]
    grad, mag = np.zeros((vocab, h)), np.zeros((vocab, h))
    flat = ids.reshape(-1)
    keep = np.flatnonzero((flat >= 0) & (flat < vocab))
    d = dout.reshape(-1, h).astype(np.float64)[keep] * scale
    np.add.at(grad, flat[keep], d)
    np.add.at(mag, flat[keep], np.abs(d))
    return grad, mag


# ---- activations in 8 bits

def _blocks(x):
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    pad = np.zeros((rows, nb * BLOCK))
    pad[:, :cols] = x
    return pad.reshape(rows, nb, BLOCK)


def scales8(x):
    """Scale bytes, rows x ceil(cols / 32), of fp32 or narrower values x."""
    a = np.abs(_blocks(np.asarray(x, np.float64)))
    most = np.where(np.isfinite(a), a, 0).max(2).astype(np.float32)
    return np.maximum((most.view(np.uint32) >> 23).astype(np.int64) - 7, 1).astype(np.uint8)


def pack8(x):
    """(codes, scale bytes) by the definition in include/muon.h: nearest code, the even one of two as near."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    scale = scales8(x)
    up = np.repeat(np.exp2(127.0 - scale), BLOCK, axis=1)[:, :cols]
    finite = np.isfinite(x)
    y = np.where(finite, np.abs(x), 0) * up
    values = E4M3[:127]                                    # ascending
    above = np.clip(np.searchsorted(values, y), 0, 126)    # the first code at or above y
    below = np.maximum(above - 1, 0)
    d_above, d_below = values[above] - y, y - values[below]
    code = np.where((d_below < d_above) | ((d_below == d_above) & (below % 2 == 0)), below, above)
    code = np.where(np.signbit(x), code | 128, code)
    sign_of_nan = np.where(finite, code, 127)
    return sign_of_nan.astype(np.uint8), scale


def unpack8(codes, scale):
    """float64 values."""
    rows, cols = codes.shape
    down = np.repeat(np.exp2(scale.astype(np.float64) - 127), BLOCK, axis=1)[:, :cols]
    v = E4M3[codes & 127]
    return np.where(codes & 128, -v, v) * down


def small_blocks(most):
    """fp32 rows of three blocks whose largest magnitude is 2^most, with smaller ones down to the smallest denormal."""
    g = np.random.default_rng(1000 + most)
    e = np.maximum(most - g.integers(0, 24, (8, 96)), -149)
    x = np.ldexp(np.where(e > -149, 1 + g.random((8, 96)), 1.0), np.minimum(e, most - 1)) * g.choice([-1.0, 1.0], (8, 96))
    x[:, ::32] = 2.0 ** most
    return x.astype(np.float32)


# ---- gated feed-forward block of experts

def _phi(g):
    from math import erfc
    return 0.5 * np.vectorize(erfc, otypes=[np.float64])(-g / np.sqrt(2.0)) if g.size else g


def act(g, name):
    """(activation, derivative)."""
    if name == "silu":
        s = 0.5 * (1 + np.tanh(0.5 * g))
        return g * s, s * (1 + g * (1 - s))
    cdf = _phi(g)
    return g * cdf, cdf + g * np.exp(-0.5 * g * g) / np.sqrt(2 * np.pi)


def ranges(offsets, counts, rows):
    """(expert, first row, end) of the rows that hold a token."""
    return [(e, int(o), int(o) + int(n)) for e, (o, n) in enumerate(zip(offsets, counts)) if n > 0]


def ffn_pre(x, gate, up, parts):
    """g, u, and the sums of their terms' magnitudes; zero in rows without a token."""
    rows, f = x.shape[0], gate.shape[1]
    g, u, mg, mu = (np.zeros((rows, f)) for _ in range(4))
    for e, a, b in parts:
        g[a:b], u[a:b] = x[a:b] @ gate[e].T, x[a:b] @ up[e].T
        mg[a:b], mu[a:b] = np.abs(x[a:b]) @ np.abs(gate[e]).T, np.abs(x[a:b]) @ np.abs(up[e]).T
    return g, u, mg, mu


def ffn_rows(a_, w, parts, cols):
    """Rows of a_ times the transposed matrix of their expert, zero elsewhere."""
    out = np.zeros((a_.shape[0], cols))
    for e, a, b in parts:
        out[a:b] = a_[a:b] @ w[e].T
    return out


def ffn_weight(p, q, parts, experts):
    """p^T q over each expert's rows."""
    out = np.zeros((experts, p.shape[1], q.shape[1]))
    for e, a, b in parts:
        out[e] = p[a:b].T @ q[a:b]
    return out
