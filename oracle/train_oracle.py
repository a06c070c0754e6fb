"""Plain numpy definitions of the training-step operators around the Muon
step, for the tests.  float64 throughout, except the 8-bit states, whose codes
are defined on fp32 arithmetic (every product and sum rounded by itself) and
are reproduced here bit for bit."""
from __future__ import annotations

import numpy as np

BLOCK = 256
M32 = np.uint64(0xFFFFFFFF)


# ---- AdamW

def adamw(p, g, m, v, lr, beta1, beta2, eps, weight_decay, step):
    """float64 (p, m, v) after one step."""
    p, g, m, v = (np.asarray(x, np.float64) for x in (p, g, m, v))
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    mhat = m / (1 - beta1 ** step)
    vhat = v / (1 - beta2 ** step)
    return p - lr * weight_decay * p - lr * mhat / (np.sqrt(vhat) + eps), m, v


def splitmix64(x: int) -> int:
    mask = (1 << 64) - 1
    x = (x + 0x9E3779B97F4A7C15) & mask
    x = ((x ^ (x >> 30)) * 0xBF58476D1CE4E5B9) & mask
    x = ((x ^ (x >> 27)) * 0x94D049BB133111EB) & mask
    return x ^ (x >> 31)


def mix32(x: np.ndarray) -> np.ndarray:
    x = x & M32
    x ^= x >> np.uint64(16)
    x = (x * np.uint64(0x6A09E667)) & M32
    x ^= x >> np.uint64(15)
    x = (x * np.uint64(0xBB67AE85)) & M32
    return x ^ (x >> np.uint64(16))


def random16(n: int, seed: int, step: int, first: int = 0):
    """The 16-bit random numbers of elements first .. first + n - 1, for m and v."""
    key = splitmix64((seed + step * 0x9E3779B97F4A7C15) & ((1 << 64) - 1))
    i = np.arange(first, first + n, dtype=np.uint64)
    block = mix32((i >> np.uint64(8)) + np.uint64(key & 0xFFFFFFFF)) ^ np.uint64(key >> 32)
    h = mix32(block + (i & np.uint64(255)) * np.uint64(0x9E3779B9))
    return (h & np.uint64(0xFFFF)).astype(np.uint32), (h >> np.uint64(16)).astype(np.uint32)


# the values of the codes 0 .. 127 (sign clear)
def code_values(mantissa: int, bias: int, special) -> np.ndarray:
    out = np.empty(128)
    for c in range(128):
        e, f = c >> mantissa, c & ((1 << mantissa) - 1)
        if special(c):
            out[c] = np.nan
        elif e == 0:
            out[c] = f * 2.0 ** (1 - bias - mantissa)
        else:
            out[c] = (1 + f / (1 << mantissa)) * 2.0 ** (e - bias)
    return out


E4M3 = code_values(3, 7, lambda c: c == 127)
E5M2 = code_values(2, 15, lambda c: c >= 124)


def decode8(codes, table):
    c = np.asarray(codes, np.uint8)
    x = table[c & 127]
    return np.where(c & 128, -x, x)


def per_element(scale_bytes, n):
    """Powers of two of one column of scale bytes, for each element."""
    s = np.exp2(np.asarray(scale_bytes, np.float64) - 127)
    return np.repeat(s, BLOCK)[:n]


def load8(m_codes, v_codes, scales):
    """float32 m and v of 8-bit states (the products are exact in fp32)."""
    n = len(m_codes)
    return ((decode8(m_codes, E4M3) * per_element(scales[:, 0], n)).astype(np.float32),
            (decode8(v_codes, E5M2) * per_element(scales[:, 1], n)).astype(np.float32))


def moments_f32(m, v, g, beta1, beta2):
    """New m and v in fp32, every product and sum rounded by itself."""
    f = np.float32
    g = np.asarray(g, f)
    with np.errstate(all="ignore"):
        m = f(beta1) * np.asarray(m, f) + f(1 - beta1) * g
        v = f(beta2) * np.asarray(v, f) + f(1 - beta2) * (g * g)
    return m, v


def store8(x, random, table, top, mantissa, least, never_zero):
    """(codes, scale bytes) of fp32 values x, from the definition in include/muon.h
    on exact numbers: blocks of 256, power-of-two scales, stochastic rounding."""
    x = np.asarray(x, np.float32)
    n = len(x)
    nb = -(-n // BLOCK)
    pad = np.zeros(nb * BLOCK, np.float32)
    pad[:n] = x
    a = np.abs(pad.astype(np.float64))
    finite = np.isfinite(a)
    most = np.where(finite, a, 0).reshape(nb, BLOCK).max(1).astype(np.float32)
    exponent = (most.view(np.uint32) >> 23).astype(np.int64)
    scale = np.maximum(exponent - top, 1)
    up = np.repeat(np.exp2(127.0 - scale), BLOCK)
    y = np.where(finite, a, 0) * up
    # the spacing of codes at y
    e = np.maximum(np.floor(np.log2(np.maximum(y, 2.0 ** -140))), least)
    ulp = np.exp2(e - mantissa)
    r = np.zeros(nb * BLOCK)
    r[:n] = random
    # numbers below the smallest spacing keep 23 bits after kLow is added to them
    low = 2.0 ** least
    y32 = np.where(y < low, ((y + low).astype(np.float32).astype(np.float64) - low), y)
    q = np.floor(y32 / ulp + r / 65536) * ulp
    if never_zero:
        q = np.where((a > 0) & (q == 0), 2.0 ** (least - mantissa), q)
    order = np.argsort(table[~np.isnan(table)])
    values = table[~np.isnan(table)][order]
    at = np.searchsorted(values, q)
    assert np.array_equal(values[at], q)
    codes = np.flatnonzero(~np.isnan(table))[order][at].astype(np.uint8)
    codes = np.where(np.signbit(pad), codes | 128, codes)
    codes = np.where(finite, codes, 127).astype(np.uint8)
    return codes[:n], scale.astype(np.uint8)


def store8_m(m, random):
    return store8(m, random, E4M3, 7, 3, -6, False)


def store8_v(v, random):
    return store8(v, random, E5M2, 14, 2, -14, True)


# ---- clipping

def clip(grads, max_norm):
    norm = np.sqrt(sum(float(np.sum(np.asarray(g, np.float64) ** 2)) for g in grads))
    c = min(1.0, max_norm / (norm + 1e-6))
    return norm, [np.asarray(g, np.float64) * c for g in grads]


# ---- tokens by expert

def sort(ids, experts, capacity=0, align=1):
    """(row, offsets, counts), one slot after another."""
    ids = np.asarray(ids)
    seen = np.zeros(experts, np.int64)
    rank = np.full(ids.shape, -1, np.int64)
    for t in range(ids.shape[0]):
        for k in range(ids.shape[1]):
            e = ids[t, k]
            if 0 <= e < experts:
                if capacity == 0 or seen[e] < capacity:
                    rank[t, k] = seen[e]
                seen[e] += 1
    counts = np.minimum(seen, capacity) if capacity else seen
    room = np.full(experts, capacity) if capacity else -(-seen // align) * align
    offsets = np.concatenate([[0], np.cumsum(room)])
    row = np.where(rank >= 0, offsets[np.clip(ids, 0, experts - 1)] + rank, -1)
    return row.astype(np.int32), offsets.astype(np.int32), counts.astype(np.int32)


def dispatch(x, row, rows):
    xs = np.zeros((rows, x.shape[1]))
    for t, k in zip(*np.nonzero(row >= 0)):
        xs[row[t, k]] = x[t]
    return xs


def combine(y, w, row):
    """float64 sums, and the sums of the terms' magnitudes (for error bounds)."""
    out = np.zeros((row.shape[0], y.shape[1]))
    mag = np.zeros_like(out)
    for t, k in zip(*np.nonzero(row >= 0)):
        term = (1.0 if w is None else float(w[t, k])) * y[row[t, k]].astype(np.float64)
        out[t] += term
        mag[t] += np.abs(term)
    return out, mag


def combine_backward(dout, y, w, row):
    dy = np.zeros(y.shape)
    dw = np.zeros(row.shape)
    mag = np.zeros(row.shape)
    for t, k in zip(*np.nonzero(row >= 0)):
        r = row[t, k]
        d = dout[t].astype(np.float64)
        dy[r] = float(w[t, k]) * d
        dw[t, k] = d @ y[r].astype(np.float64)
        mag[t, k] = np.abs(d) @ np.abs(y[r].astype(np.float64))
    return dy, dw, mag
