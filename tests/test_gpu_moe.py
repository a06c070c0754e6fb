"""Tokens sorted by expert, dispatched, combined, and both gradients, against
the float64 definitions.

Bounds (u = 2^-24): a combined value has one product and one sum per choice,
(topk + 1) u of the terms' magnitudes; dw sums over a row: at most
hidden / 32 + 24 terms one after another; a bf16 result is rounded once more
(2^-8 of it).  Rows that are copied, and w * dout, are exact to the bit."""
import threading

import numpy as np
import pytest
import torch
import torch.autograd.forward_ad as fwAD

import oracle.train_oracle as O
from muon_newton_schulz_gb300 import binding as B
from muon_newton_schulz_gb300 import moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def make_ids(T, K, E, seed, masked=0.0, kind=torch.int64, skew=1.0):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(T, E, generator=g) + skew * torch.randn(E, generator=g)
    if K <= E:
        ids = logits.topk(K, 1).indices
    else:
        ids = torch.randint(0, E, (T, K), generator=g)
    if masked and T:
        ids[torch.rand(T, generator=g) < masked] = -1
        ids[torch.rand(T, K, generator=g) < masked / 4] = E       # beyond the last expert
    return ids.to(kind)


def host(t):
    return t.detach().double().cpu().numpy()


def route_of(ids, E, capacity=0, align=1):
    r = moe.sort_tokens(ids.to(DEV), E, capacity=capacity, align=align)
    row, offsets, counts = O.sort(ids.numpy(), E, capacity, align)
    np.testing.assert_array_equal(r.row.cpu().numpy(), row)
    np.testing.assert_array_equal(r.offsets.cpu().numpy(), offsets)
    np.testing.assert_array_equal(r.counts.cpu().numpy(), counts)
    assert r.offsets[-1] <= r.rows
    return r, row


@pytest.mark.parametrize("T, K, E", [(0, 2, 4), (1, 1, 1), (1, 8, 128), (3, 2, 5), (31, 3, 7), (33, 1, 1024), (257, 8, 16),
                                     (1000, 2, 33), (2048, 8, 128), (2049, 8, 100), (16385, 1, 16), (9000, 6, 64),
                                     (40000, 2, 1000), (70001, 3, 3), (200, 10, 4), (500, 64, 100)])
@pytest.mark.parametrize("masked, capacity, align", [(0.0, 0, 1), (0.3, 0, 16), (0.2, 1, 1), (0.0, 100, 1), (1.0, 0, 8)])
def test_sort(T, K, E, masked, capacity, align):
    if E * capacity > 2 ** 31:
        pytest.skip("too large")
    ids = make_ids(T, K, E, T + K, masked, torch.int32 if T % 2 else torch.int64)
    if masked == 1.0:
        ids[:] = -1
    route_of(ids, E, capacity, align)


def test_sort_odd_ids():
    big = torch.tensor([[2 ** 40, 1], [-(2 ** 35), 0], [2 ** 32 + 1, 2], [1, 1]])      # low words that look valid
    route_of(big, 3)
    same = torch.full((5000, 4), 2)                                                  # one expert takes all, twice a token
    route_of(same, 9)
    route_of(same, 9, capacity=77)
    t = make_ids(60, 4, 10, 1)
    r = moe.sort_tokens(t.to(DEV).t().contiguous().t(), 10)                              # strided ids
    np.testing.assert_array_equal(r.row.cpu().numpy(), O.sort(t.numpy(), 10)[0])


CASES = [(1, 2, 16, 2048, 0.0, 0, 1), (1, 1, 1, 1, 0.0, 0, 1), (5, 8, 128, 6144, 0.0, 0, 1), (7, 3, 9, 1001, 0.4, 0, 16),
         (130, 2, 16, 264, 0.2, 15, 1), (301, 6, 64, 100, 0.1, 0, 128), (64, 1, 4, 8, 0.0, 5, 1), (33, 12, 30, 40, 0.1, 0, 1),
         (20, 64, 100, 72, 0.0, 0, 1), (600, 8, 128, 512, 0.0, 30, 1), (0, 2, 4, 64, 0.0, 0, 8), (50, 4, 8, 3, 1.0, 0, 4)]


@pytest.mark.parametrize("T, K, E, H, masked, capacity, align", CASES)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("w_dtype", [F32, BF16])
def test_dispatch_combine_and_gradients(T, K, E, H, masked, capacity, align, dtype, w_dtype):
    ids = make_ids(T, K, E, 7 * T + K, masked)
    if masked == 1.0:
        ids[:] = -1
    r, row = route_of(ids, E, capacity, align)
    g = torch.Generator().manual_seed(T + H)
    x = torch.randn(T, H, generator=g).to(dtype).to(DEV)
    w = torch.softmax(torch.randn(T, K, generator=g), 1).to(w_dtype).to(DEV) if T else torch.empty(0, K, dtype=w_dtype, device=DEV)
    xs = moe.dispatch(x, r)
    assert xs.shape == (r.rows, H) and xs.dtype == dtype
    np.testing.assert_array_equal(host(xs), O.dispatch(host(x), row, r.rows))

    # rows without a token hold NaN, and so do the weights of dropped choices: neither may show
    y = torch.full((r.rows, H), float("nan"), dtype=dtype)
    used = torch.from_numpy(row[row >= 0].astype(np.int64))
    y[used] = torch.randn(len(used), H, generator=g).to(dtype)
    y = y.to(DEV)
    w = torch.where(torch.from_numpy(row >= 0).to(DEV), w, float("nan"))
    wide = 2.0 ** -8 if dtype == BF16 else 0.0
    for weights in (w, None):
        out = moe.combine(y, weights, r)
        want, mag = O.combine(host(y), None if weights is None else host(w), row)
        assert out.shape == (T, H) and out.dtype == dtype
        assert (np.abs(host(out) - want) <= (K + 1) * U * mag + wide * (np.abs(want) + (K + 1) * U * mag)).all()

    dout = torch.randn(T, H, generator=g).to(dtype).to(DEV)
    dy, dw = moe.combine_backward(dout, y, w, r)
    want_dy, want_dw, mag = O.combine_backward(host(dout), host(y), host(w), row)
    assert dy.dtype == dtype and dw.dtype == w_dtype and dy.shape == y.shape and dw.shape == w.shape
    # an fp32 product, rounded once more to bf16
    exact = torch.zeros(r.rows, H, dtype=dtype)
    t, k = np.nonzero(row >= 0)
    exact[torch.from_numpy(row[t, k].astype(np.int64))] = (w[t, k].float().unsqueeze(1) * dout[t].float()).to(dtype).cpu()
    assert torch.equal(dy.cpu(), exact)
    bound = (H / 32 + 24) * U * mag
    if w_dtype == BF16:
        bound = bound + 2.0 ** -8 * (np.abs(want_dw) + bound)
    assert (np.abs(host(dw) - want_dw) <= bound).all()

    dxs = torch.where(torch.from_numpy(np.isin(np.arange(r.rows), row)).to(DEV).unsqueeze(1),
                      torch.randn(r.rows, H, generator=g).to(dtype).to(DEV), float("nan"))
    dx = moe.dispatch_backward(dxs, r)
    want, mag = O.combine(host(dxs), None, row)
    assert (np.abs(host(dx) - want) <= (K + 1) * U * mag + wide * (np.abs(want) + (K + 1) * U * mag)).all()


@pytest.mark.parametrize("capacity, align", [(0, 16), (9, 1)])
def test_autograd_against_the_formula_and_differences(capacity, align):
    T, K, E, H = 40, 2, 6, 24
    ids = make_ids(T, K, E, 3, 0.1)
    r, row = route_of(ids, E, capacity, align)
    g = torch.Generator().manual_seed(8)
    x = torch.randn(T, H, generator=g).to(DEV).requires_grad_()
    w = torch.rand(T, K, generator=g).to(DEV).requires_grad_()
    a = torch.randn(r.rows, H, generator=g).to(DEV)             # the "experts": each row times its own numbers
    c = torch.randn(T, H, generator=g).to(DEV)

    def loss(x, w):
        return (moe.combine(a * moe.dispatch(x, r), w, r).double() * c).sum()

    loss(x, w).backward()
    # formula, in float64
    xd, wd = x.detach().double().cpu().requires_grad_(), w.detach().double().cpu().requires_grad_()
    keep = torch.from_numpy(row >= 0)
    at = torch.from_numpy(np.maximum(row, 0).astype(np.int64))
    ref = ((wd * keep).unsqueeze(2) * a.double().cpu()[at] * xd.unsqueeze(1)).sum(1)
    (ref * c.double().cpu()).sum().backward()
    np.testing.assert_allclose(host(x.grad), xd.grad.numpy(), rtol=0, atol=16 * U * float(xd.grad.abs().max()))
    np.testing.assert_allclose(host(w.grad), wd.grad.numpy(), rtol=0, atol=64 * U * H * float((a.abs().max() * x.detach().abs().max() * c.abs().max())))
    # central differences: the loss is linear in x and in w, so they are exact up to the fp32 rounding of `out`,
    # whose sums over T * H values of size |c| |out| grow no faster than their number
    step = 0.25
    for t in (x, w):
        d = torch.randn(t.shape, generator=g).to(DEV)
        with torch.no_grad():
            hi = loss(x + step * d, w) if t is x else loss(x, w + step * d)
            lo = loss(x - step * d, w) if t is x else loss(x, w - step * d)
        size = float((ref.detach().abs() * c.double().cpu().abs()).sum()) + float((t.grad.double() * d).abs().sum())
        assert abs(float(hi - lo) / (2 * step) - float((t.grad.double() * d).sum())) <= 16 * U * size / step


def test_combine_without_weights_has_a_gradient():
    ids = make_ids(12, 2, 4, 5)
    r, row = route_of(ids, 4)
    y = torch.randn(r.rows, 16, device=DEV, requires_grad=True)
    c = torch.randn(12, 16, device=DEV)
    (moe.combine(y, None, r) * c).sum().backward()
    np.testing.assert_array_equal(host(y.grad), O.dispatch(host(c), row, r.rows))


def test_strides_and_odd_addresses():
    T, K, E, H = 37, 2, 5, 96
    ids = make_ids(T, K, E, 2)
    r, row = route_of(ids, E)
    for dtype in (F32, BF16):
        buf = torch.randn(T + 1, H + 9, device=DEV).to(dtype)
        ys = torch.randn(r.rows + 1, H + 24, device=DEV).to(dtype)
        w = torch.rand(K, T, device=DEV).t()                               # strided weights
        for x in (buf[:T, :H], buf[:T, 1:H + 1], buf[1:, 3:H + 3], buf[:1].expand(T + 1, H + 9)[:T, :H],
                  torch.randn(H, T, device=DEV).to(dtype).t()):
            np.testing.assert_array_equal(host(moe.dispatch(x, r)), O.dispatch(host(x), row, r.rows))
        for y in (ys[:r.rows, :H], ys[:r.rows, 8:H + 8], ys[1:, 1:H + 1]):
            same = y.contiguous()
            assert torch.equal(moe.combine(y, w, r), moe.combine(same, w.contiguous(), r))
            d = buf[:T, 5:H + 5]
            for p, q in zip(moe.combine_backward(d, y, w, r), moe.combine_backward(d.contiguous(), same, w.contiguous(), r)):
                # the same products; a dot product may be summed in another order
                assert torch.equal(p, q) if p.shape[0] == r.rows else torch.allclose(p, q, rtol=0, atol=64 * U * H * 9)


def test_a_route_that_points_outside_is_not_followed():
    """Rows beyond the buffer count as dropped; offsets beyond it clear nothing outside."""
    T, K, E, H = 6, 2, 3, 32
    row = torch.tensor([[0, 12], [1, 2 ** 31 - 1], [-5, 2], [3, 4], [5, 6], [7, 8]], dtype=torch.int32, device=DEV)
    offsets = torch.tensor([0, -4, 100, 2 ** 30], dtype=torch.int32, device=DEV)
    counts = torch.tensor([2, 2 ** 31 - 1, -7], dtype=torch.int32, device=DEV)
    r = moe.Route(row, offsets, counts)
    assert r.rows == 12
    x = torch.randn(T, H, device=DEV)
    w = torch.rand(T, K, device=DEV)
    ok = np.array([[0, -1], [1, -1], [-1, 2], [3, 4], [5, 6], [7, 8]])
    xs = moe.dispatch(x, r)
    np.testing.assert_array_equal(host(xs)[:9], O.dispatch(host(x), ok, 12)[:9])
    y = torch.randn(12, H, device=DEV)
    want, mag = O.combine(host(y), host(w), ok)
    assert (np.abs(host(moe.combine(y, w, r)) - want) <= 3 * U * mag).all()
    _, dw = moe.combine_backward(x, y, w, r)
    assert not dw[0, 1] and not dw[1, 1] and not dw[2, 0]


def test_offsets_beyond_2_31_elements():
    T, K, E, H = 150_000, 2, 4, 8192
    ids = torch.arange(T * K).reshape(T, K) % E
    r = moe.sort_tokens(ids.to(DEV), E)
    row, _, _ = (t for t in O.sort(ids[:8].numpy(), E))
    y = torch.zeros(r.rows, H, dtype=BF16, device=DEV)
    assert y.numel() > 2 ** 31
    last = r.row[-1].tolist()
    assert max(last) == r.rows - 1 and min(last) * H > 2 ** 30
    y[last[0]] = 1.5
    y[last[1]] = 2.0
    w = torch.ones(T, K, device=DEV)
    out = moe.combine(y, w, r)
    assert (out[-1] == 3.5).all() and not out[:-1].any()
    x = torch.zeros(T, H, dtype=BF16, device=DEV)
    x[-1] = 3.0
    xs = moe.dispatch(x, r)
    assert (xs[last[0]] == 3).all() and (xs[last[1]] == 3).all()
    assert int((xs[:, 0] != 0).sum()) == 2
    dy, dw = moe.combine_backward(x, y, w * 0.5, r)
    assert (dy[last] == 1.5).all() and int((dy[:, 5] != 0).sum()) == 2
    assert dw[-1].tolist() == [3 * 1.5 * H, 3 * 2.0 * H] and not dw[:-1].any()


def test_streams_and_determinism():
    T, K, E, H = 5000, 4, 32, 256
    ids = make_ids(T, K, E, 4).to(DEV)
    x, w = torch.randn(T, H, device=DEV).to(BF16), torch.rand(T, K, device=DEV)

    def all_of():
        r = moe.sort_tokens(ids, E, align=8)
        xs = moe.dispatch(x, r)
        out = moe.combine(xs, w, r)
        return [r.row, r.offsets, r.counts, xs, out, *moe.combine_backward(out, xs, w, r), moe.dispatch_backward(xs, r)]

    first = all_of()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        second = all_of()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = all_of()
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_refusals():
    ids = make_ids(10, 2, 4, 1).to(DEV)
    r = moe.sort_tokens(ids, 4)
    x, y, w = torch.randn(10, 8, device=DEV), torch.randn(r.rows, 8, device=DEV), torch.rand(10, 2, device=DEV)
    for call, why in ((lambda: moe.dispatch(x[:9], r), "rows"), (lambda: moe.dispatch(x.half(), r), "bf16 or fp32"),
                      (lambda: moe.dispatch(x.cpu(), r), "cpu"), (lambda: moe.combine(y[:-1], w, r), "rows"),
                      (lambda: moe.combine(y, w[:, :1], r), "shape"), (lambda: moe.combine(y, w.half(), r), "bf16 or fp32"),
                      (lambda: moe.combine(y, w.cpu(), r), "cpu"),
                      (lambda: moe.combine_backward(x.to(BF16), y, w, r), "one row length and type"),
                      (lambda: moe.combine_backward(x[:, :4], y, w, r), "one row length and type"),
                      (lambda: moe.Route(r.row.long(), r.offsets, r.counts), "int32"),
                      (lambda: moe.Route(r.row, r.offsets[:-1], r.counts), "offsets")):
        with pytest.raises(ValueError, match=why):
            call()
    for kw in (dict(experts=0), dict(experts=1025), dict(experts=4, capacity=-1), dict(experts=4, align=0),
               dict(experts=4, capacity=4, align=4)):
        with pytest.raises(B.MuonError):
            moe.sort_tokens(ids, **kw)
    with pytest.raises(B.MuonError):
        moe.sort_tokens(torch.zeros(3, 65, dtype=torch.int64, device=DEV), 100)


def test_sort_of_more_slots_than_stay_in_registers():
    T, K, E = 320_000, 8, 40
    g = torch.Generator().manual_seed(3)
    ids = torch.randint(-1, E + 1, (T, K), generator=g, dtype=torch.int32)
    flat = ids.flatten().long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.argsort(key, stable=True)
    for capacity, align in ((0, 32), (70_000, 1)):
        r = moe.sort_tokens(ids.to(DEV), E, capacity=capacity, align=align)
        counts = torch.bincount(key, minlength=E + 1)
        room = torch.full((E,), capacity) if capacity else -(-counts[:E] // align) * align
        first = torch.cat([torch.zeros(1, dtype=torch.long), room.cumsum(0)])
        rank = torch.empty_like(key)
        rank[order] = torch.arange(len(key)) - (counts.cumsum(0) - counts)[key[order]]
        row = torch.where((key < E) & ((rank < capacity) | (capacity == 0)), first[key.clamp(max=E - 1)] + rank, -1)
        assert torch.equal(r.row.cpu().flatten().long(), row)
        assert torch.equal(r.offsets.cpu().long(), first)
        assert torch.equal(r.counts.cpu().long(), counts[:E].clamp(max=capacity) if capacity else counts[:E])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("masked, capacity", [(0.0, 0), (0.3, 9)])
def test_forward_mode_derivatives(dtype, masked, capacity):
    """Tangents go through dispatch and combine as the formulas say, with and without recording for a backward pass; a
    combined tangent is the sum of two combined values: their bounds, and one more rounding to the type."""
    T, K, E, H = 40, 2, 6, 24
    ids = make_ids(T, K, E, 3, masked)
    r, row = route_of(ids, E, capacity)
    g = torch.Generator().manual_seed(4)

    def rand(*shape, kind=dtype):
        return torch.randn(*shape, generator=g).to(kind).to(DEV)

    x, tx, y, ty = rand(T, H), rand(T, H), rand(r.rows, H), rand(r.rows, H)
    w, tw = rand(T, K, kind=F32), rand(T, K, kind=F32)
    wide = 2.0 ** -8 if dtype == BF16 else 0.0
    for recorded in (True, False):
        with fwAD.dual_level(), torch.set_grad_enabled(recorded):
            xs = moe.dispatch(fwAD.make_dual(x, tx), r)
            got = fwAD.unpack_dual(xs)
            assert torch.equal(got.primal, moe.dispatch(x, r)) and torch.equal(got.tangent, moe.dispatch(tx, r))
            assert fwAD.unpack_dual(moe.dispatch(x, r)).tangent is None
            for dy, dw in ((ty, tw), (ty, None), (None, tw)):
                out = moe.combine(y if dy is None else fwAD.make_dual(y, dy), w if dw is None else fwAD.make_dual(w, dw), r)
                got = fwAD.unpack_dual(out)
                assert torch.equal(got.primal, moe.combine(y, w, r)) and got.tangent.dtype == dtype
                want = mag = 0
                for a, b in ((dy, w), (y, dw)):
                    if a is not None and b is not None:
                        s, m = O.combine(host(a), host(b), row)
                        want, mag = want + s, mag + m
                assert (np.abs(host(got.tangent) - want) <= (K + 2) * U * mag + 2 * wide * (1 + wide) * mag).all()
            got = fwAD.unpack_dual(moe.combine(fwAD.make_dual(y, ty), None, r))
            assert torch.equal(got.tangent, moe.combine(ty, None, r))
            assert torch.equal(fwAD.unpack_dual(moe.dispatch_backward(fwAD.make_dual(y, ty), r)).tangent, got.tangent)
            with pytest.raises(RuntimeError, match="forward"):
                moe.combine_backward(x, fwAD.make_dual(y, ty), w, r)


def test_forward_mode_through_a_backward_pass():
    """The gradient of sum(dispatch(x)^2) is 2 x for each kept choice, and so is its tangent; that of combine's gradient
    is refused."""
    T, K, E, H = 30, 2, 5, 8
    r, row = route_of(make_ids(T, K, E, 2), E)
    x, tx = torch.randn(T, H, device=DEV, requires_grad=True), torch.randn(T, H, device=DEV)
    y = torch.randn(r.rows, H, device=DEV, requires_grad=True)
    w = torch.rand(T, K, device=DEV)
    with fwAD.dual_level():
        d = fwAD.make_dual(x, tx)
        grad, = torch.autograd.grad(moe.dispatch(d, r).square().sum(), d)
        assert torch.equal(fwAD.unpack_dual(grad).tangent, 2 * K * tx)
        out = moe.combine(fwAD.make_dual(y, torch.randn_like(y)), w.requires_grad_(), r)
        with pytest.raises(RuntimeError, match="forward"):
            torch.autograd.grad(out.square().sum(), w)


def test_tracing_is_refused():
    """A tracer would record the result's allocation and not the kernel that fills it."""
    from torch.fx.experimental.proxy_tensor import make_fx

    from muon_newton_schulz_gb300 import adamw
    ids = make_ids(10, 2, 4, 1).to(DEV)
    r = moe.sort_tokens(ids, 4)
    x, y, w = torch.randn(10, 8, device=DEV), torch.randn(r.rows, 8, device=DEV), torch.rand(10, 2, device=DEV)
    for f, args in ((lambda a: moe.sort_tokens(a, 4).row, (ids,)), (lambda a: moe.dispatch(a, r), (x,)),
                    (lambda a, b: moe.combine(a, b, r), (y, w)), (lambda a, b: moe.combine_backward(a, b, w, r), (x, y)),
                    (lambda a: moe.dispatch_backward(a, r), (y,)),
                    (lambda a: adamw.clip_grads([a], 1.0), (x,)),
                    (lambda a: adamw.adamw_step([a], [x], [torch.zeros_like(x)], [torch.zeros_like(x)], lr=1.0, step=1), (x + 0,))):
        with pytest.raises(RuntimeError, match="cannot be traced"):
            make_fx(f)(*args)
        f(*args)
    with pytest.raises(RuntimeError, match="traced"):
        torch.jit.trace(lambda a: moe.dispatch(a, r), (x,), check_trace=False)


def test_two_threads_sort_for_different_numbers_of_experts():
    """Each with its own handle and stream, through the C interface, which leaves the threads to run at the same time; both
    need more shared memory than a launch gets unasked."""
    results = {}

    def work(E, calls):
        st, h = B.muon_create(None, 0)
        assert st == B.MUON_OK
        stream = torch.cuda.Stream()
        ids = make_ids(300, 2, E, E, kind=torch.int32)
        with torch.cuda.stream(stream):
            d = ids.to(DEV)
            row, offsets, counts = (torch.empty(n, dtype=torch.int32, device=DEV) for n in (600, E + 1, E))
        stream.synchronize()
        shape = B.muon_moe_shape(300, 2, E, 0, 1)
        seen = set()
        for i in range(calls):
            seen.add(B.muon_moe_sort(h, shape, d.data_ptr(), 32, row.data_ptr(), offsets.data_ptr(), counts.data_ptr(),
                                     None, 0, stream.cuda_stream))
            if i % 256 == 0:
                stream.synchronize()
        stream.synchronize()
        B.muon_destroy(h)
        results[E] = (seen, np.array_equal(row.cpu().numpy().reshape(300, 2), O.sort(ids.numpy(), E)[0]))

    threads = [threading.Thread(target=work, args=(E, 20000)) for E in (400, 1024)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert results == {400: ({B.MUON_OK}, True), 1024: ({B.MUON_OK}, True)}


def test_memory_that_cannot_be_had():
    """An allocation that the device refuses arrives as torch's own error."""
    r = moe.sort_tokens(torch.zeros(1, 1, dtype=torch.int64, device=DEV), 1024, capacity=1 << 20)
    with pytest.raises(torch.OutOfMemoryError):
        moe.dispatch(torch.zeros(1, 4096, device=DEV), r)          # 16 TB


def test_other_threads_run_while_the_library_is_called():
    from test_train_host import _with_gil_check

    from muon_newton_schulz_gb300 import adamw
    r = moe.sort_tokens(make_ids(10, 2, 4, 1).to(DEV), 4)
    ids, x, y, w = r.row + 0, torch.randn(10, 8, device=DEV), torch.randn(r.rows, 8, device=DEV), torch.rand(10, 2, device=DEV)

    def each(_):
        # a status other than 0, which a caller that holds the lock gets, raises
        adamw.clip_grads([x], 1.0)
        adamw.adamw_step([x], [x], [x], [x], lr=1.0, step=1)
        moe.sort_tokens(ids, 4)
        moe.dispatch(x, r)
        moe.combine(y, w, r)
        moe.combine_backward(x, y, w, r)
        return True

    assert _with_gil_check(each)


def test_numbers_that_32_bits_do_not_hold_are_refused():
    ids = make_ids(10, 2, 4, 1).to(DEV)
    for kw in (dict(experts=4, capacity=1 << 32), dict(experts=(1 << 32) + 4), dict(experts=4, align=(1 << 32) + 1)):
        with pytest.raises(ValueError, match="2\\^31"):
            moe.sort_tokens(ids, **kw)


def test_gradients_of_a_combine_without_weights_are_refused():
    r = moe.sort_tokens(make_ids(10, 2, 4, 1).to(DEV), 4)
    with pytest.raises(ValueError, match="weights"):
        moe.combine_backward(torch.zeros(10, 8, device=DEV), torch.zeros(r.rows, 8, device=DEV), None, r)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("which", ["y", "weights", "both"])
def test_gradients_of_some_inputs(dtype, which):
    """Frozen experts or a frozen router: the other gradient is the one of both."""
    T, K, E, H = 50, 3, 6, 40
    r, row = route_of(make_ids(T, K, E, 9, 0.1), E, 0, 4)
    g = torch.Generator().manual_seed(1)
    y = torch.randn(r.rows, H, generator=g).to(dtype).to(DEV).requires_grad_(which != "weights")
    w = torch.rand(T, K, generator=g).to(DEV).requires_grad_(which != "y")
    c = torch.randn(T, H, generator=g).to(dtype).to(DEV)
    (moe.combine(y, w, r) * c).sum().backward()
    dy, dw = moe.combine_backward(c, y.detach(), w.detach(), r)
    assert (y.grad is None) == (which == "weights") and (w.grad is None) == (which == "y")
    assert y.grad is None or torch.equal(y.grad, dy)
    assert w.grad is None or torch.equal(w.grad, dw)
