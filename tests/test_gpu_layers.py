"""Embedding rows and their gradient, and activations in 8 bits, against the
float64 definitions.

Bounds (u = 2^-24): an embedding row has one product in fp32 with a scale
rounded to it, 2 u, and its rounding to bf16, 2^-8 of the value.  A gradient sums
at most 64 terms of a chunk one after another, then the chunks' sums (in eight
parts of at most chunks / 8 + 1, joined one after another), then the scale: at most
(min(n, 64) + n / (8 chunk) + 12 + 2) u of the terms' magnitudes for n tokens.
Codes and scales are exact to the bit."""
import threading

import numpy as np
import pytest
import torch
import torch.autograd.forward_ad as fwAD

import oracle.layer_oracle as L
from muon_newton_schulz_gb300 import binding as B
from muon_newton_schulz_gb300 import checkpoint, embedding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def host(t):
    return t.detach().double().cpu().numpy()


def make_ids(n, vocab, seed, how):
    g = torch.Generator().manual_seed(seed)
    if how == "uniform":
        ids = torch.randint(0, max(vocab, 1), (n,), generator=g)
    elif how == "skewed":
        ids = ((vocab + 1.0) ** torch.rand(n, generator=g, dtype=torch.float64)).long().sub_(1).clamp_(0, vocab - 1)
    elif how == "same":
        ids = torch.full((n,), vocab // 2)
    else:                                   # some outside, also such as look valid in their low words
        ids = torch.randint(-vocab, 2 * vocab, (n,), generator=g)
        ids[::7] = 2 ** 40 + 1
    return ids


def grad_bound(mag, n):
    rounds = 608 * max(1, -(-n // (608 * 64)))               # four CTAs on each of 152 SMs, at most 64 tokens each
    chunk = min(64, max(8, -(-n // rounds)))
    return (min(n, 64) + n / (8 * chunk) + 14) * U * mag


CASES = [(1, 1, 1, "uniform"), (1, 65536, 2048, "uniform"), (0, 7, 12, "uniform"), (5, 3, 2, "outside"), (511, 100, 33, "skewed"),
         (513, 1000, 64, "outside"), (1003, 1001, 1003, "skewed"), (2049, 50, 130, "uniform"), (2048, 3000, 8, "same"),
         (5000, 70000, 40, "skewed"), (20000, 1 << 20, 16, "uniform"), (9001, 2, 264, "uniform"), (20000, 300, 2056, "skewed"),
         (40000, 5, 24, "same"), (160000, 30000, 9, "skewed")]


@pytest.mark.parametrize("n, vocab, hidden, how", CASES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_embed_and_gradient(n, vocab, hidden, how, dtype):
    ids = make_ids(n, vocab, n + vocab, how)
    kind = torch.int64 if how == "outside" or n % 2 else torch.int32
    dev_ids = ids.to(kind).to(DEV)
    g = torch.Generator().manual_seed(n + hidden)
    wide = 2.0 ** -8 if dtype == BF16 else 0.0
    scale = 3.7
    if vocab * hidden <= 1 << 24:
        table = torch.randn(vocab, hidden, generator=g).to(dtype)
        out = embedding.embed(dev_ids, table.to(DEV), scale=scale)
        want = L.embed(ids.numpy(), host(table), scale)
        assert out.shape == (n, hidden) and out.dtype == dtype
        assert (np.abs(host(out) - want) <= (2 * U + wide * (1 + 2 * U)) * np.abs(want)).all()
    dout = torch.randn(n, hidden, generator=g).to(dtype)
    got = embedding.embed_backward(dout.to(DEV), dev_ids, vocab, scale=scale)
    want, mag = L.embed_backward(host(dout), ids.numpy(), vocab, scale)
    assert got.shape == (vocab, hidden) and got.dtype == dtype
    bound = grad_bound(mag, n)
    assert (np.abs(host(got) - want) <= bound + wide * (np.abs(want) + bound)).all()
    assert (host(got)[mag == 0] == 0).all()
    again = embedding.embed_backward(dout.to(DEV), dev_ids, vocab, scale=scale)
    assert torch.equal(got, again)


def test_sum_of_whole_numbers_is_exact():
    """Runs of equal ids that begin, end and go on at every place in a chunk."""
    for n in (700, 2500, 30000):
        ids = torch.arange(n).mul(0.37).sin().mul(n / 40).abs().long()
        ids = ids.sort().values[torch.randperm(n, generator=torch.Generator().manual_seed(n))]
        dout = torch.randint(-8, 9, (n, 20), generator=torch.Generator().manual_seed(1)).float()
        got = embedding.embed_backward(dout.to(DEV), ids.to(DEV), n)
        want, _ = L.embed_backward(dout.numpy(), ids.numpy(), n, 1.0)
        np.testing.assert_array_equal(host(got), want)


@pytest.mark.parametrize("n, vocab, hidden", [(700_001, 3000, 3), (34_000_003, 70_000, 1)])
def test_sums_over_many_tokens(n, vocab, hidden):
    """More tokens than the sort's CTAs keep in registers, and more chunks than a grid's second dimension has places; whole
    numbers, and sums below 2^24, are exact."""
    g = torch.Generator(device=DEV).manual_seed(n)
    ids = (torch.rand(n, generator=g, device=DEV) ** 4 * vocab).int()         # the first ids have runs of many chunks
    dout = torch.randint(-1, 2, (n, hidden), generator=g, device=DEV).float()
    got = embedding.embed_backward(dout, ids, vocab)
    want = torch.zeros(vocab, hidden, dtype=torch.float64, device=DEV).index_add_(0, ids.long(), dout.double())
    assert want.abs().max() < 2 ** 24 and torch.equal(got.double(), want)


def test_strides_and_shapes():
    g = torch.Generator().manual_seed(2)
    table = torch.randn(50, 96, generator=g).to(DEV)
    ids = torch.randint(0, 50, (6, 4, 5), generator=g).to(DEV)
    for t in (table[:, 8:72], table[::2], table.t()[:50], table[:, 1:60]):
        i = ids % t.shape[0]
        assert torch.equal(embedding.embed(i, t), t[i])
    turned = ids.permute(2, 0, 1)
    assert torch.equal(embedding.embed(turned, table), table[turned])
    dout = torch.randint(-3, 4, (6, 4, 5, 40), generator=g).float().to(DEV)
    want, _ = L.embed_backward(host(dout), ids.cpu().numpy(), 50, 2.0)
    np.testing.assert_array_equal(host(embedding.embed_backward(dout, ids, 50, scale=2.0)), want)
    wide = torch.randint(-3, 4, (6, 4, 5, 80), generator=g).float().to(DEV)
    for d in (wide[..., 3:43], wide[..., 1:], wide[..., ::2]):
        want, _ = L.embed_backward(host(d), ids.cpu().numpy(), 50, 1.0)
        np.testing.assert_array_equal(host(embedding.embed_backward(d, ids, 50)), want)
    assert embedding.embed(ids[:0], table).shape == (0, 4, 5, 96)
    assert embedding.embed(ids[0, 0, 0], table).shape == (96,)
    assert embedding.embed(ids, table[:, :0]).shape == (6, 4, 5, 0)


def test_values_that_are_not_finite_stay_in_their_rows():
    table = torch.ones(8, 40, device=DEV)
    table[3, 5], table[4, 6] = float("nan"), float("inf")
    ids = torch.tensor([0, 3, 4, -1, 8], device=DEV)
    out = embedding.embed(ids, table, scale=2.0)
    assert torch.isnan(out[1, 5]) and out[2, 6] == float("inf") and (out[[0]] == 2).all() and (out[3:] == 0).all()
    dout = torch.ones(5, 40, device=DEV)
    dout[3:] = float("nan")                  # of ids outside the table
    dout[1, 7] = float("nan")
    got = embedding.embed_backward(dout, ids, 8)
    assert torch.isnan(got[3, 7]) and torch.isnan(got).sum() == 1 and (got[0] == 1).all() and (got[5:] == 0).all()


def test_embed_autograd_against_formula_and_differences():
    g = torch.Generator().manual_seed(8)
    table = torch.randn(12, 10, generator=g).to(DEV).requires_grad_()
    ids = torch.tensor([[1, 5, 1], [11, -1, 5]], device=DEV)
    c = torch.randn(2, 3, 10, generator=g).to(DEV)

    def f(t):
        return (embedding.embed(ids, t, scale=1.5).sin() * c).sum()

    f(table).backward()
    want = torch.zeros(12, 10, dtype=torch.float64)
    for a in range(2):
        for b in range(3):
            if ids[a, b] >= 0:
                row = table[ids[a, b]].detach().double().cpu()
                want[ids[a, b]] += 1.5 * (1.5 * row).cos() * c[a, b].double().cpu()
    assert (table.grad.double().cpu() - want).abs().max() <= 64 * U * want.abs().max()
    # central differences: the third derivative is at most 1.5^3, fp32 sums of 60 terms of size <= |c|
    d = torch.randn(12, 10, generator=g).to(DEV)
    step = 2.0 ** -7
    with torch.no_grad():
        slope = float(f(table + step * d) - f(table - step * d)) / (2 * step)
    third = 1.5 ** 3 * float((embedding.embed(ids, d).abs() ** 3 * c.abs()).sum()) / 6 * step ** 2
    noise = 2 * 64 * U * float(c.abs().sum()) / (2 * step)
    assert abs(slope - float((table.grad * d).sum())) <= third + noise + 64 * U * float((table.grad * d).abs().sum())
    # forward mode
    with fwAD.dual_level():
        dual = fwAD.make_dual(table.detach(), d)
        tangent = fwAD.unpack_dual(embedding.embed(ids, dual, scale=1.5)).tangent
    assert torch.equal(tangent, embedding.embed(ids, d, scale=1.5))
    with fwAD.dual_level(), pytest.raises(RuntimeError, match="forward-mode"):
        embedding.embed_backward(fwAD.make_dual(c, c), ids, 12)


# ---- activations in 8 bits

def bytes_of(t):
    return t.view(torch.uint8).cpu().numpy()


@pytest.mark.parametrize("rows, cols", [(1, 1), (1, 31), (3, 33), (7, 32), (1003, 1001), (64, 4096), (5, 8), (300, 96), (0, 5), (4, 0)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_pack_and_unpack(rows, cols, dtype):
    g = torch.Generator().manual_seed(rows + cols)
    x = (torch.randn(rows, cols, generator=g) * torch.randn(rows, 1, generator=g).mul(20).exp()).to(dtype)
    if cols > 4 and rows > 1:
        x[0, :5] = torch.tensor([float("inf"), -float("inf"), float("nan"), -0.0, 1e-42])
        x[1] = 0
    p = checkpoint.pack(x.to(DEV))
    codes, scale = L.pack8(x.double().numpy()) if rows * cols else (np.zeros((rows, cols), np.uint8), np.zeros((rows, -(-cols // 32)), np.uint8))
    assert p.codes.shape == (rows, cols) and p.scales.shape == scale.shape and p.dtype == dtype and p.shape == x.shape
    np.testing.assert_array_equal(bytes_of(p.scales), scale)
    got = bytes_of(p.codes)
    nan = (codes & 127) == 127
    np.testing.assert_array_equal(got[~nan], codes[~nan])
    assert ((got[nan] & 127) == 127).all()
    for to in (None, F32, BF16):
        back = checkpoint.unpack(p, to)
        assert back.dtype == (to or dtype) and back.shape == x.shape
        want = torch.from_numpy(L.unpack8(codes, scale)).float().to(back.dtype) if rows * cols else back.cpu()
        np.testing.assert_array_equal(host(back), host(want))


@pytest.mark.parametrize("most", [-100, -118, -119, -120, -125, -137, -149])
def test_small_blocks(most):
    """Codes are the definition's down to the smallest denormal, and within its bound."""
    x = L.small_blocks(most)
    p = checkpoint.pack(torch.from_numpy(x).to(DEV))
    codes, scale = L.pack8(x)
    np.testing.assert_array_equal(bytes_of(p.codes), codes)
    np.testing.assert_array_equal(bytes_of(p.scales), scale)
    off = np.abs(host(checkpoint.unpack(p)) - x)
    assert (off <= np.maximum(2.0 ** -4 * np.abs(x), max(2.0 ** (most - 17), 2.0 ** -136))).all()


def test_the_largest_values():
    """From 1.9375 * 2^127 on the nearest code stands for 2^128."""
    top = 2.0 ** 127
    x = torch.tensor([[1.9 * top, 1.93 * top, -1.95 * top, 2.0 ** 126]], dtype=torch.float64).float().to(DEV)
    back = checkpoint.unpack(checkpoint.pack(x))
    assert back.tolist() == [[1.875 * top, 1.875 * top, float("-inf"), 2.0 ** 126]]


def test_pack_strides_and_shapes():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(40, 6, 128, generator=g).to(DEV)
    for t in (x, x[:, 0], x[:, :, :96], x[:, 1, 3:70], x.transpose(0, 2), x[::3, 2, 32:], x[0, 0], x[0, 0, 1:], x[:, 0, ::2], x[:, 0, 1:33]):
        for kind in (F32, BF16):
            a = t.to(kind) if kind == BF16 else t
            p = checkpoint.pack(a)
            q = checkpoint.pack(a.contiguous())
            assert torch.equal(p.codes.view(torch.uint8), q.codes.view(torch.uint8)) and torch.equal(p.scales.view(torch.uint8), q.scales.view(torch.uint8))
            flat = a.contiguous().view(-1, a.shape[-1])
            codes, scale = L.pack8(host(flat))
            np.testing.assert_array_equal(bytes_of(p.codes).reshape(codes.shape), codes)
            np.testing.assert_array_equal(host(checkpoint.unpack(p)).reshape(codes.shape), L.unpack8(codes, scale))


def test_unpack_takes_any_scale_byte():
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).to(DEV)
    for s in (0, 1, 127, 254, 255):
        scales = torch.full((8,), s, dtype=torch.uint8).view(torch.float8_e8m0fnu).to(DEV)
        back = checkpoint.unpack(checkpoint.Packed(codes, scales, F32))
        want = codes.float().cpu() * scales.float().cpu().repeat_interleave(32)
        np.testing.assert_array_equal(host(back), host(want))


def test_saved_in_8_bits():
    """The gradient of x^3: 2 x^2 and x are saved through 8 bits (each off by at most 2^-4 of itself), parameters are not."""
    g = torch.Generator().manual_seed(4)
    x = (torch.randn(64, 256, generator=g).abs() + 0.5).to(DEV)
    w = torch.randn(256, 32, generator=g).to(DEV).requires_grad_()
    x.requires_grad_()
    h = x * 1.0                                              # not a leaf
    with checkpoint.saved_in_8_bits(min_elements=1000):
        y = (h * h) @ w
    c = torch.randn(64, 32, generator=g).to(DEV)
    y.backward(c)
    kept = checkpoint.unpack(checkpoint.pack(h.detach()))
    square = checkpoint.unpack(checkpoint.pack((h * h).detach()))
    assert torch.equal(x.grad, 2 * kept * (c @ w.detach().t())) or torch.allclose(x.grad, 2 * kept * (c @ w.detach().t()), rtol=1e-6, atol=0)
    assert torch.allclose(w.grad, square.t() @ c, rtol=1e-5, atol=1e-4)
    assert not torch.equal(kept, h.detach())


@pytest.mark.parametrize("rows, cols", [(1, 1), (3, 33), (64, 4096), (300, 97), (40, 64)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_infinities_stay_what_they_are(rows, cols, dtype):
    g = torch.Generator().manual_seed(rows * cols)
    x = (torch.randn(rows, cols, generator=g) * torch.randn(rows, 1, generator=g).mul(20).exp()).to(dtype)
    what = torch.randint(0, 6, (rows, cols), generator=g)
    for i, v in enumerate((float("inf"), -float("inf"), float("nan"))):
        x[what == i] = v
    x = x.to(DEV)
    p, q = checkpoint.pack(x, special=True), checkpoint.pack(x)
    assert torch.equal(p.scales.view(torch.uint8), q.scales.view(torch.uint8))
    for to in (F32, BF16):
        back, plain = checkpoint.unpack(p, to), checkpoint.unpack(q, to)
        assert torch.equal(torch.isinf(back), torch.isinf(x)) and torch.equal(torch.isnan(back), torch.isnan(x))
        inf = torch.isinf(x)
        assert torch.equal(back[inf].float(), x[inf].float())
        assert torch.isnan(plain[inf]).all() and torch.equal(back[~inf].nan_to_num(7), plain[~inf].nan_to_num(7))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols", [32, 45, 256])
def test_every_element_stays_of_its_kind(cols, dtype):
    """Elements of all sizes below their block's largest, down to the smallest, and the largest there are."""
    g = torch.Generator().manual_seed(cols)
    x = torch.randn(40, cols, generator=g, dtype=torch.float64).sign() * 2 ** (-160 * torch.rand(40, cols, generator=g, dtype=torch.float64))
    x[:, ::32] = 1
    x[:20] *= 2.0 ** torch.randint(-120, 120, (20, 1), generator=g)
    x[5, :] = 0
    x[6, 0], x[7, 0] = torch.finfo(dtype).max, -torch.finfo(dtype).max
    x = x.to(dtype).to(DEV)
    back = checkpoint.unpack(checkpoint.pack(x, special=True), F32)
    assert torch.isfinite(back).all() and torch.equal(back == 0, x == 0) and torch.equal(back.sign(), x.float().sign())
    v, b = host(x), host(back)
    blocks = np.pad(np.abs(v), ((0, 0), (0, -cols % 32))).reshape(40, -1, 32).max(2).repeat(32, 1)[:, :cols]
    assert (np.abs(b - v) <= np.maximum(np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -16 * blocks), 2.0 ** -135)).all()


def test_gradients_that_divide_by_what_was_saved():
    """Denominators, square roots and signs of elements far below their block's largest stay finite and what they are."""
    x = torch.full((64, 64), 1.0, device=DEV)
    x[:, 1::2] = 2.0 ** -30
    for f in (lambda h: h.log(), lambda h: h.sqrt(), lambda h: 1 / h, lambda h: torch.relu(h)):
        leaf = x.clone().requires_grad_()
        h = leaf * 1.0
        with checkpoint.saved_in_8_bits(min_elements=1):
            y = f(h)
        y.sum().backward()
        assert torch.isfinite(leaf.grad).all() and (leaf.grad != 0).all()
        if f(torch.ones(1, device=DEV)) == 1 and f(2 * torch.ones(1, device=DEV)) == 2:     # relu: no value is needed, but its sign
            assert (leaf.grad == 1).all()


def test_masked_logits_inside_saved_in_8_bits():
    """Words that are masked with -inf have a probability of 0: every gradient is finite, and the logits' is what it is
    without the context, because log-probabilities are not rounded."""
    g = torch.Generator().manual_seed(9)
    h0 = torch.randn(256, 64, generator=g).to(DEV)
    w0 = torch.randn(512, 64, generator=g).mul_(0.2).to(DEV)
    masked = torch.arange(512, device=DEV) >= 500
    target = torch.randint(0, 500, (256,), generator=g).to(DEV)

    def run(inside):
        h, w = h0.clone().requires_grad_(), w0.clone().requires_grad_()
        x = h * 1.0
        with inside:
            logits = (x @ w.t()).masked_fill(masked, float("-inf"))
            loss = torch.nn.functional.cross_entropy(logits, target)
        logits.retain_grad()
        loss.backward()
        return h.grad, logits.grad, w.grad, x.detach()

    dh, dl, dw, x = run(checkpoint.saved_in_8_bits(min_elements=1))
    want_h, want_l, want_w, _ = run(torch.enable_grad())
    assert torch.isfinite(dw).all() and torch.equal(dl, want_l) and torch.equal(dh, want_h)
    kept = checkpoint.unpack(checkpoint.pack(x))
    # fp32 products of 256 terms; each element that was kept is off by 2^-4 of itself
    want = dl.double().t() @ kept.double()
    assert ((dw - want).abs() <= 260 * U * (dl.abs().double().t() @ kept.abs().double())).all()
    assert not torch.equal(dw, want_w) and (dw[500:] == 0).all()


def test_scores_that_are_masked_keep_their_infinities():
    """logsumexp saves its argument: -inf of a masked score is kept, its gradient is 0 there and exp(kept - result) elsewhere."""
    g = torch.Generator().manual_seed(10)
    s = torch.randn(64, 96, generator=g).to(DEV).requires_grad_()
    hidden = torch.rand(64, 96, generator=g).to(DEV) < 0.3
    with checkpoint.saved_in_8_bits(min_elements=1):
        z = s.masked_fill(hidden, float("-inf"))
        y = z.logsumexp(1)
    y.sum().backward()
    kept = checkpoint.unpack(checkpoint.pack(z.detach(), special=True))
    want = torch.where(hidden, 0.0, (kept.double() - y.detach().double().unsqueeze(1)).exp())
    assert torch.isfinite(s.grad).all() and (s.grad[hidden] == 0).all()
    assert ((s.grad - want).abs() <= 2.0 ** -18 * want).all()


def test_what_saved_in_8_bits_leaves_alone(monkeypatch):
    """Attention's normalizers, a norm's statistics, masks and what `which` says no to are not packed."""
    F = torch.nn.functional
    packed = []
    pack = checkpoint.pack
    monkeypatch.setattr(checkpoint, "pack", lambda t, **kw: packed.append((tuple(t.shape), t.dtype)) or pack(t, **kw))
    x = torch.randn(2, 4, 64, 64, device=DEV, dtype=BF16).requires_grad_() * 1.0
    with checkpoint.saved_in_8_bits(min_elements=1):
        F.scaled_dot_product_attention(x, x, x).float().sum().backward()
    assert packed and {s for s, _ in packed} == {(2, 4, 64, 64)} and {d for _, d in packed} == {BF16}
    for f, want in ((lambda h: F.layer_norm(h, (64,)), {(32, 64)}), (lambda h: h * h.square().mean(1, keepdim=True).rsqrt(), {(32, 64)}),
                    (lambda h: h * torch.ones(32, 64, device=DEV), set())):
        h = torch.randn(32, 64, device=DEV).requires_grad_() * 1.0
        packed.clear()
        with checkpoint.saved_in_8_bits(min_elements=1):
            y = f(h)
        assert set(s for s, _ in packed) == want
        y.sum().backward()
    h = torch.randn(32, 64, device=DEV).requires_grad_() * 1.0
    packed.clear()
    with checkpoint.saved_in_8_bits(min_elements=1, which=lambda t: t.dtype == BF16):
        (h.sin().to(BF16).square().sum()).backward()
    assert packed == [((32, 64), BF16)]


# ---- streams, graphs, threads

def test_captured_and_replayed():
    """Each operator in a graph, replayed on new inputs, beside an eager call on another stream."""
    g = torch.Generator().manual_seed(5)
    ids = torch.randint(0, 300, (3000,), generator=g).to(DEV)
    table = torch.randn(300, 72, generator=g).to(DEV)
    dout = torch.randint(-3, 4, (3000, 72), generator=g).float().to(DEV)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        embedding.embed(ids, table), embedding.embed_backward(dout, ids, 300), checkpoint.unpack(checkpoint.pack(dout))
    torch.cuda.current_stream().wait_stream(stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = embedding.embed(ids, table, scale=2.0)
        grad = embedding.embed_backward(dout, ids, 300)
        back = checkpoint.unpack(checkpoint.pack(dout))
    for seed in range(3):
        g = torch.Generator().manual_seed(seed)
        ids.copy_(torch.randint(-5, 310, (3000,), generator=g))
        dout.copy_(torch.randint(-3, 4, (3000, 72), generator=g).float())
        graph.replay()
        with torch.cuda.stream(stream):
            eager = embedding.embed_backward(torch.ones(3000, 72, device=DEV), torch.zeros(3000, dtype=torch.int32, device=DEV), 2)
        torch.cuda.synchronize()
        want, _ = L.embed_backward(host(dout), ids.cpu().numpy(), 300, 1.0)
        np.testing.assert_array_equal(host(grad), want)
        assert (eager[0] == 3000).all() and (eager[1] == 0).all()
        known = (ids >= 0) & (ids < 300)
        assert torch.equal(out, torch.where(known.unsqueeze(1), table[ids.clamp(0, 299)] * 2, 0.0))
        assert torch.equal(back, dout)


def test_threads():
    """Threads that call at once, each on a stream of its own."""
    g = torch.Generator().manual_seed(6)
    ids = torch.randint(0, 500, (4000,), generator=g).to(DEV)
    dout = torch.randint(-3, 4, (4000, 64), generator=g).float().to(DEV)
    want, _ = L.embed_backward(host(dout), ids.cpu().numpy(), 500, 1.0)
    torch.cuda.synchronize()
    bad = []

    def work():
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    if not np.array_equal(host(embedding.embed_backward(dout, ids, 500)), want):
                        bad.append("sums")
                    if not torch.equal(checkpoint.unpack(checkpoint.pack(dout)), dout):
                        bad.append("codes")
        except Exception as e:  # pragma: no cover
            bad.append(repr(e))

    threads = [threading.Thread(target=work) for _ in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad


def test_other_threads_run_while_the_library_is_called():
    """The library's functions replaced by one whose status says whether the caller holds Python's lock: 0 is no, and the
    call's tensors come back."""
    import ctypes
    calls = B.torch_calls()
    check = ctypes.cast(ctypes.pythonapi.PyGILState_Check, ctypes.c_void_p).value
    x, ids = torch.zeros(8, 64, device=DEV), torch.zeros(8, dtype=torch.int64, device=DEV)
    w, d = torch.zeros(32, 64, device=DEV), torch.zeros(64, 32, device=DEV)
    calls.bind_layers(*[check] * 8)
    try:
        codes, scales = calls.pack8(x, 0, 0)
        assert isinstance(calls.unpack8(codes, scales, False, 0, 0), torch.Tensor)
        assert isinstance(calls.embed(ids, x, 1.0, 0, 0), torch.Tensor)
        assert isinstance(calls.embed_backward(x, ids, 5, 1.0, 0, 0), torch.Tensor)
        assert isinstance(calls.ffn_forward(x, w, w, d, None, None, 0, 0, 0, 0), torch.Tensor)
        y, *kept = calls.ffn_forward(x, w, w, d, None, None, 0, 32, 0, 0)
        assert len(calls.ffn_backward(y, x, w, w, d, None, None, kept, 0, 32, 15, 0, 0)) == 4
    finally:
        B._calls = None
        B.torch_calls()          # binds the library again


def test_long_tables_pass_32_bits():
    """Rows whose place in the table is beyond 2^32 bytes and elements."""
    vocab, hidden = (1 << 22) + 9, 1032
    table = torch.zeros(vocab, hidden, dtype=BF16, device=DEV)
    at = torch.tensor([0, (1 << 21) + 3, vocab - 1], device=DEV)
    table[at] = torch.arange(1, 4, device=DEV, dtype=BF16).unsqueeze(1)
    assert torch.equal(embedding.embed(at, table)[:, 0].cpu(), torch.tensor([1, 2, 3], dtype=BF16))
    del table
    got = embedding.embed_backward(torch.ones(3, hidden, device=DEV, dtype=BF16), at, vocab)
    assert float(got.sum(dtype=torch.float32)) == 3 * hidden and (got[at] == 1).all()


def test_refusals_on_the_device():
    ids = torch.zeros(3, dtype=torch.int64, device=DEV)
    table = torch.zeros(4, 8, device=DEV)
    for bad in (lambda: embedding.embed(ids, table.half()), lambda: embedding.embed(ids, table[0]), lambda: embedding.embed(ids, table.cpu()),
                lambda: embedding.embed(ids.float(), table), lambda: embedding.embed_backward(table, ids, 4),
                lambda: embedding.embed_backward(torch.zeros(3, 8, device=DEV), ids, -1), lambda: checkpoint.pack(table.double()),
                lambda: checkpoint.unpack(checkpoint.Packed(table, table, F32))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises((B.MuonError, ValueError)):
        embedding.embed_backward(torch.zeros(3, 8, device=DEV), ids, 1 << 40)
    torch.cuda.synchronize()
