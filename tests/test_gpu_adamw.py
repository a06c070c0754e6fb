"""AdamW and gradient clipping on the GPU against the float64 definitions.

Bounds, from the kernels' arithmetic (u = 2^-24, an fp32 rounding):
  m, v   four and five roundings of terms whose magnitudes add up to
         b1 |m| + (1 - b1) |g| and b2 v + (1 - b2) g^2;
  p      the root is within 2^-23, the quotient within two units in the last
         place (2^-22), the constants and products a rounding each: together
         below 2^-20 of the update, plus what the error of m moves, plus three
         roundings of p; a bf16 p is rounded once more (half a unit: 2^-8 |p|);
  8 bits codes and scales equal bit for bit;
  norm   each thread sums the squares of 64 elements of a chunk in fp32, the
         rest in fp64: 65 u of the sum, half of that for the root."""
import ctypes

import numpy as np
import pytest
import torch

import oracle.train_oracle as O
from muon_newton_schulz_gb300 import adamw
from muon_newton_schulz_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
HP = dict(lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
F32, BF16 = torch.float32, torch.bfloat16


def f64(t):
    return t.detach().double().cpu().numpy().ravel()


def codes(t):
    return t.detach().contiguous().view(torch.uint8).cpu().numpy().ravel()


def make(n, p_dtype, g_dtype, bits, seed, lead=0):
    """Tensors that begin `lead` elements into their buffers."""
    g = torch.Generator().manual_seed(seed)

    def place(x):
        buf = torch.zeros(n + lead + 3, dtype=torch.uint8 if x.element_size() == 1 else x.dtype, device=DEV)
        buf = buf.view(x.dtype)
        view = buf[lead:lead + n]
        view.copy_(x)
        return view

    p = place(torch.randn(n, generator=g).mul_(0.05).to(p_dtype))
    grad = torch.randn(n, generator=g).mul_(1e-3)
    grad[torch.rand(n, generator=g) < 0.2] = 0
    grad = place(grad.to(g_dtype))
    m = torch.randn(n, generator=g) * 1e-3
    v = torch.rand(n, generator=g) * 1e-6
    v[::7] = 0
    if bits == 32:
        return p, grad, place(m), place(v), None
    nb = -(-n // 256)
    mc = torch.randint(0, 256, (n,), generator=g, dtype=torch.int16)
    mc[(mc & 127) == 127] = 0                       # no NaN
    vc = torch.randint(0, 124, (n,), generator=g, dtype=torch.int16)
    s = torch.randint(90, 110, (nb, 2), generator=g, dtype=torch.int16)
    s[0] = torch.tensor([1, 1])                     # the smallest scales
    return (p, grad, place(mc.to(torch.uint8).view(torch.float8_e4m3fn)), place(vc.to(torch.uint8).view(torch.float8_e5m2)),
            s.to(torch.uint8).to(DEV).view(torch.float8_e8m0fnu))


def check(before, after, step, seed):
    """after = the tensors of `before` (host copies) stepped once."""
    p0, g0, m0, v0, s0 = before
    p1, g1, m1, v1, s1 = after
    b1, b2 = HP["betas"]
    g = f64(g0)
    if s0 is None:
        m, v = f64(m0), f64(v0)
    else:
        m, v = O.load8(codes(m0), codes(v0), codes(s0).reshape(-1, 2))
    want_p, want_m, want_v = O.adamw(f64(p0), g, m, v, HP["lr"], b1, b2, HP["eps"], HP["weight_decay"], step)
    em = 4 * U * (b1 * np.abs(m) + (1 - b1) * np.abs(g))
    ev = 5 * U * (b2 * np.abs(v) + (1 - b2) * g * g)
    if s0 is None:
        assert (np.abs(f64(m1) - want_m) <= em + 1e-45).all()
        assert (np.abs(f64(v1) - want_v) <= ev + 1e-45).all()
    else:
        m32, v32 = O.moments_f32(m, v, g, b1, b2)
        rm, rv = O.random16(len(g), seed, step)
        mc, ms = O.store8_m(m32, rm)
        vc, vs = O.store8_v(v32, rv)
        np.testing.assert_array_equal(codes(s1).reshape(-1, 2), np.stack([ms, vs], 1))
        np.testing.assert_array_equal(codes(m1), mc)
        np.testing.assert_array_equal(codes(v1), vc)
    denom = np.sqrt(want_v / (1 - b2 ** step)) + HP["eps"]
    size = HP["lr"] / (1 - b1 ** step)
    bound = 2.0 ** -20 * size * np.abs(want_m) / denom + size * em / denom + 3 * U * np.abs(f64(p0))
    if p0.dtype == BF16:
        bound = bound + 2.0 ** -8 * (np.abs(want_p) + bound)
    assert (np.abs(f64(p1) - want_p) <= bound).all()
    assert torch.equal(g0.cpu(), g1.cpu())


def clone(ts):
    return tuple(None if t is None else t.clone() for t in ts)


def step_all(sets, step, seed, **kw):
    ps, gs, ms, vs, ss = (list(x) for x in zip(*sets))
    adamw.adamw_step(ps, gs, ms, vs, ss, step=step, seed=seed, **HP, **kw)
    torch.cuda.synchronize()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p_dtype, g_dtype", [(F32, F32), (BF16, BF16), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("n, lead", [(1, 0), (3, 1), (255, 0), (256, 0), (257, 2), (4095, 3), (4096, 0), (4100, 1),
                                     (12345, 0), (65537, 5), (70000, 8)])
def test_one_tensor(bits, p_dtype, g_dtype, n, lead):
    ts = make(n, p_dtype, g_dtype, bits, 100 + n, lead)
    before = clone(ts)
    step_all([ts], 3, 77)
    check(before, ts, 3, 77)
    step_all([ts], 4, 77)
    assert all(torch.isfinite(t.float()).all() for t in ts if t is not None)


def test_neighbours_in_memory_are_left_alone():
    """Tensors packed without gaps: each is stepped as if it were alone."""
    for bits in (32, 8):
        sizes = [1, 5, 257, 3, 1000, 4097, 2, 9000]
        n = sum(sizes)
        whole = make(n, BF16, BF16, bits, 9)
        flat = [t.clone() for t in whole[:4]]
        at, sets = 0, []
        scales = torch.full((sum(-(-k // 256) for k in sizes) + 1, 2), 100, dtype=torch.uint8, device=DEV)
        keep = scales[-1].clone()
        sa = 0
        for k in sizes:
            nb = -(-k // 256)
            sets.append(tuple(t[at:at + k] for t in flat) + ((scales[sa:sa + nb].view(torch.float8_e8m0fnu) if bits == 8 else None),))
            at += k
            sa += nb
        befores = [clone(s) for s in sets]
        step_all(sets, 2, 5)
        for i, (b, s) in enumerate(zip(befores, sets)):
            check(b, s, 2, 5 + i)
        assert torch.equal(scales[-1], keep)


def test_buffers_aligned_differently():
    n = 5000
    for bits in (32, 8):
        for i in range(4):
            ts = list(make(n, BF16, F32, bits, 40, 0))
            other = make(n, BF16, F32, bits, 40, 1)
            ts[i] = other[i]
            before = clone(ts)
            step_all([tuple(ts)], 2, 3)
            check(before, tuple(ts), 2, 3)


@pytest.mark.parametrize("bits", [32, 8])
def test_batch_order_and_size_do_not_matter(bits):
    """More tensors than one launch holds, both kinds of state among them."""
    sets = [make(10 + 37 * (i % 50), BF16, BF16, bits if i % 3 else 32, i) for i in range(900)]
    one = [clone(s) for s in sets]
    step_all(sets, 7, 1000)
    order = list(range(899, -1, -1))
    for part in (order[:123], order[123:]):
        ps, gs, ms, vs, ss = (list(x) for x in zip(*[one[i] for i in part]))
        descs = (B.muon_adamw_desc * len(part))()
        for d, i in zip(descs, part):
            p, g, m, v, s = one[i]
            d.n, d.P, d.G, d.M, d.V = p.numel(), p.data_ptr(), g.data_ptr(), m.data_ptr(), v.data_ptr()
            d.scales = s.data_ptr() if s is not None else None
            d.p_dtype = d.g_dtype = B.MUON_BF16
            d.state_bits, d.step, d.seed = 32 if s is None else 8, 7, 1000 + i
            d.lr, d.weight_decay = HP["lr"], HP["weight_decay"]
        cfg = B.muon_adamw_config(*HP["betas"], HP["eps"])
        assert B.muon_adamw_step(B.thread_handle(0), cfg, ctypes.addressof(descs), len(part),
                                 torch.cuda.current_stream().cuda_stream) == B.MUON_OK
    torch.cuda.synchronize()
    for a, b in zip(sets, one):
        for x, y in zip(a, b):
            assert x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_per_tensor_numbers_and_fresh_states():
    for bits in (32, 8):
        sets = []
        for i in range(3):
            p, g, _, _, _ = make(600, F32, F32, 32, i)
            if bits == 32:
                sets.append((p, g, torch.zeros_like(p), torch.zeros_like(p), None))
            else:
                sets.append((p, g) + adamw.state8_like(p))
        before = [clone(s) for s in sets]
        ps, gs, ms, vs, ss = (list(x) for x in zip(*sets))
        lrs, wds, steps = [1e-3, 0.0, 5e-2], [0.0, 0.5, 0.1], [1, 2, 1000]
        adamw.adamw_step(ps, gs, ms, vs, ss, lr=lrs, weight_decay=wds, step=steps, betas=(0.9, 0.95), eps=1e-8, seed=4)
        for i in range(3):
            saved = dict(HP)
            try:
                HP.update(lr=lrs[i], weight_decay=wds[i])
                check(before[i], sets[i], steps[i], 4 + i)
            finally:
                HP.update(saved)


def test_transposed_parameters_and_empty_ones():
    p = torch.randn(40, 70, device=DEV).t()
    g = (torch.randn(40, 70, device=DEV) * 1e-3).t()
    m, v = torch.zeros_like(p), torch.zeros_like(p)
    assert m.stride() == p.stride()
    q = torch.empty(0, 5, device=DEV)
    before = clone((p, g, m, v))
    adamw.adamw_step([q, p], [q.clone(), g], [q.clone(), m], [q.clone(), v], step=1, seed=0, **HP)
    check(tuple(t.t() for t in before) + (None,), (p.t(), g.t(), m.t(), v.t(), None), 1, 1)
    adamw.adamw_step([], [], [], [], step=1, lr=1.0)


def test_refusals():
    p, g, m, v, _ = make(64, F32, F32, 32, 1)
    _, _, m8, v8, s8 = make(64, F32, F32, 8, 1)

    def call(p=p, g=g, m=m, v=v, s=None, **kw):
        adamw.adamw_step([p], [g], [m], [v], None if s is None else [s], **{**HP, "step": 1, **kw})

    wide = torch.randn(64, 4, device=DEV)
    for bad, why in ((dict(g=g[:63]), "shape"), (dict(m=m.half()), "m must be"), (dict(v=v.to(BF16)), "v must be"),
                     (dict(g=g.half()), "bf16 or fp32"), (dict(p=p.half()), "bf16 or fp32"),
                     (dict(m=m8, v=v8), "m must be"), (dict(m=m8, v=v8, s=s8[:0]), "scales"),
                     (dict(s=s8), "m must be"), (dict(g=g.cpu()), "cpu"),
                     (dict(p=wide[:, 0], g=wide[:, 1], m=wide[:, 2], v=wide[:, 3]), "gaps")):
        with pytest.raises(ValueError, match=why):
            call(**bad)
    for bad in (dict(step=0), dict(lr=float("nan")), dict(betas=(1.0, 0.9)), dict(eps=-1.0), dict(g=p), dict(m=v)):
        keep = clone((p, m, v))
        if "g" in bad or "m" in bad:
            with pytest.raises(B.MuonError, match="overlap"):
                call(**bad)
        else:
            with pytest.raises(B.MuonError):
                call(**bad)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(keep, (p, m, v)))


def test_not_finite():
    """Infinities and NaN stay with their elements; a block's other elements are stored as without them."""
    for bits in (32, 8):
        n = 700
        ts = make(n, F32, F32, bits, 3)
        clean = clone(ts)
        bad = {5: float("nan"), 300: float("inf"), 301: float("-inf"), 699: float("nan"), 40: 1e30}
        for i, x in bad.items():
            ts[1][i] = x
            clean[1][i] = 0.0
            # alone in its value too: an element of 0 never is its block's largest
            for k in (2, 3):
                if bits == 32:
                    clean[k][i] = ts[k][i] = 0.0
                else:
                    clean[k].view(torch.uint8)[i] = ts[k].view(torch.uint8)[i] = 0
        step_all([ts], 2, 9)
        step_all([clean], 2, 9)
        fine = torch.ones(n, dtype=torch.bool, device=DEV)
        fine[list(bad)] = False
        assert torch.equal(ts[0][fine], clean[0][fine])
        for i in bad:
            if i == 40:       # g^2 overflows: v is infinite, the update finite
                assert torch.isfinite(ts[0][i])
            else:
                assert torch.isnan(ts[0][i])
        if bits == 32:
            assert torch.equal(ts[2][fine], clean[2][fine]) and torch.equal(ts[3][fine], clean[3][fine])
        else:
            assert (codes(ts[2])[list(bad)[:4]] & 127 == 127).all() and (codes(ts[3])[list(bad)] == 127).all()
            same = fine.cpu().numpy()
            same[:256] = False          # m of element 40 is finite and its block's largest
            np.testing.assert_array_equal(codes(ts[2])[same], codes(clean[2])[same])
            np.testing.assert_array_equal(codes(ts[3])[fine.cpu().numpy()], codes(clean[3])[fine.cpu().numpy()])
            assert np.array_equal(codes(ts[4]).reshape(-1, 2)[:, 1], codes(clean[4]).reshape(-1, 2)[:, 1])


@pytest.mark.parametrize("size", [1e-44, 1e-38, 1e-30, 1e-19, 1e-12, 1.0, 1e12, 1e17, 1e37])
@pytest.mark.parametrize("eps", [1e-8, 1e-20, 0.0])
@pytest.mark.parametrize("lead", [0, 1])
def test_codes_at_the_ends_of_the_range(size, eps, lead):
    """Subnormal and huge moments, blocks whose elements differ by up to 2^80, and the form for a tiny eps."""
    n = 256 * 9
    p, g, m, v, s = make(n, F32, F32, 8, 21, lead)
    gen = torch.Generator().manual_seed(4)
    x = torch.randn(n, generator=gen).double() * size
    x[256 * 3:] *= torch.exp2(-torch.randint(0, 40, (n - 256 * 3,), generator=gen).double())
    x[256 * 6:] *= torch.exp2(-torch.randint(0, 40, (n - 256 * 6,), generator=gen).double())
    g.copy_(x.to(F32))
    m.view(torch.uint8).zero_()
    v.view(torch.uint8)[: 256 * 8] = 0
    for step in (1, 2):
        m0, v0 = O.load8(codes(m), codes(v), codes(s).reshape(-1, 2))
        m32, v32 = O.moments_f32(m0, v0, f64(g), 0.9, 0.95)
        adamw.adamw_step([p], [g], [m], [v], [s], lr=1e-3, betas=(0.9, 0.95), eps=eps, step=step, seed=9)
        rm, rv = O.random16(n, 9, step)
        mc, ms = O.store8_m(m32, rm)
        vc, vs = O.store8_v(v32, rv)
        np.testing.assert_array_equal(codes(s).reshape(-1, 2), np.stack([ms, vs], 1))
        finite = np.isfinite(m32)
        np.testing.assert_array_equal(codes(m)[finite], mc[finite])
        np.testing.assert_array_equal(codes(v), vc)
        assert (codes(m)[~finite] & 127 == 127).all()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e-3, 1e-15, 0.0])
def test_other_eps(bits, eps):
    saved = dict(HP)
    try:
        HP["eps"] = eps
        ts = make(3000, F32, F32, bits, 77)
        ts[1].add_(1e-3)                 # every v > 0: with eps = 0 the update is finite
        before = clone(ts)
        step_all([ts], 5, 2)
        check(before, ts, 5, 2)
    finally:
        HP.update(saved)


def test_8_bit_states_follow_32_bit_ones():
    """Gradients of steady size: after many steps the stored v has the right mean (nearest rounding would have
    stopped at a fraction of it) and the parameters have moved as far."""
    n, steps = 1 << 16, 400
    g = torch.Generator(device=DEV).manual_seed(2)
    p = torch.zeros(n, device=DEV)
    m, v, s = adamw.state8_like(p)
    q, m2, v2 = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    kw = dict(lr=1e-3, betas=(0.9, 0.99), eps=1e-12, weight_decay=0.0)
    for t in range(1, steps + 1):
        grad = 1e-3 * (1 + 0.1 * torch.randn(n, generator=g, device=DEV))
        adamw.adamw_step([p, q], [grad, grad], [m, m2], [v, v2], [s, None], step=t, seed=1, **kw)
    mv, vv = adamw.state8_values(m, v, s)
    assert abs(float(vv.mean() / v2.mean()) - 1) < 0.02
    assert abs(float(mv.mean() / m2.mean()) - 1) < 0.02
    # a rounding's variance is p (1 - p) steps^2 of 2^-2 v, forgotten over 100 steps: a standard deviation of about
    # 0.3 v, which moves 1 / sqrt(v) by 3/8 of its square: a few per cent
    assert abs(float(p.mean() / q.mean()) - 1) < 0.1


def test_more_than_2_31_elements():
    n = (1 << 31) + 777
    p = torch.zeros(n, dtype=BF16, device=DEV)
    g = torch.zeros(n, dtype=BF16, device=DEV)
    m = torch.zeros(n, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    v = torch.zeros(n, dtype=torch.uint8, device=DEV).view(torch.float8_e5m2)
    s = torch.zeros(-(-n // 256), 2, dtype=torch.uint8, device=DEV).view(torch.float8_e8m0fnu)
    tail = 256 * 5 + 777 % 256
    first = n - tail
    assert first % 256 == 0
    g[first:] = torch.randn(tail, device=DEV).mul_(1e-3).to(BF16)
    before = clone((p[first:], g[first:], m[first:], v[first:], s[first // 256:]))
    adamw.adamw_step([p], [g], [m], [v], [s], step=1, seed=3, **HP)
    rm, rv = O.random16(tail, 3, 1, first)
    m32, v32 = O.moments_f32(np.zeros(tail), np.zeros(tail), f64(before[1]), *HP["betas"])
    np.testing.assert_array_equal(codes(m[first:]), O.store8_m(m32, rm)[0])
    np.testing.assert_array_equal(codes(v[first:]), O.store8_v(v32, rv)[0])
    assert not p[:first].any() and p[first:].any()
    del m, v, s
    m32 = torch.zeros(n, device=DEV)
    v32 = torch.zeros(n, device=DEV)
    p.zero_()
    adamw.adamw_step([p], [g], [m32], [v32], step=1, **HP)
    check((p[first:] * 0, g[first:], m32[first:] * 0, v32[first:] * 0, None),
          (p[first:], g[first:], m32[first:], v32[first:], None), 1, 0)
    assert not m32[:first].any()


def test_on_another_stream_and_captured():
    ts = make(20000, BF16, BF16, 8, 6)
    want = clone(ts)
    step_all([want], 2, 8)
    side = torch.cuda.Stream()
    got = clone(ts)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step_all([got], 2, 8)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(want, got))
    got = clone(ts)
    torch.cuda.synchronize()
    step_all([got], 2, 8, stream=side.cuda_stream)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(want, got))
    again = clone(ts)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        ps, gs, ms, vs, ss = ([x] for x in again)
        adamw.adamw_step(ps, gs, ms, vs, ss, step=2, seed=8, **HP)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(want, again))


# ---------------------------------------------------------------- clipping

def grads_of(shapes, dtype, seed, scale):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(s, generator=g) * scale).to(dtype).to(DEV) for s in shapes]


SHAPES = [(1,), (7,), (1024, 3), (33, 65), (16385,), (3, 20000), (2048, 96), (0, 4), ()]


@pytest.mark.parametrize("dtype, out_dtype", [(F32, F32), (BF16, F32), (F32, BF16), (BF16, BF16)])
@pytest.mark.parametrize("scale", [1e-6, 0.1, 1e15])
@pytest.mark.parametrize("in_place", [True, False])
def test_clip(dtype, out_dtype, scale, in_place):
    gs = grads_of(SHAPES, dtype, 5, scale)
    want_norm, want = O.clip([f64(g) for g in gs], 1.0)
    if in_place:
        outs, got = gs, adamw.clip_grads(gs, 1.0)
    else:
        keep = clone(gs)
        outs = [torch.full(g.shape, float("nan"), dtype=out_dtype, device=DEV) for g in gs]
        got = adamw.clip_grads(gs, 1.0, outs)
        assert all(torch.equal(a, b) for a, b in zip(keep, gs))
    assert got.dtype == F32 and got.dim() == 0
    assert abs(float(got) - want_norm) <= 34 * U * want_norm
    for w, o in zip(want, outs):
        tol = 38 * U + (2.0 ** -8 if o.dtype == BF16 else 0.0)
        assert (np.abs(f64(o) - w) <= tol * np.abs(w)).all()
    if want_norm < 1:
        assert in_place or all(torch.equal(o, g.to(out_dtype)) for o, g in zip(outs, gs))


def test_clip_strided_packed_and_many():
    g = torch.Generator(device=DEV).manual_seed(1)
    wide = torch.randn(50, 130, generator=g, device=DEV)
    out = torch.zeros(50, 140, device=DEV)
    flat = torch.randn(5000, generator=g, device=DEV).to(BF16)
    res = torch.zeros(5000, device=DEV)
    long = torch.randn(3, 40000, generator=g, device=DEV)
    tr = torch.randn(20, 30, generator=g, device=DEV)
    gs = [wide[:, 1:100], wide[:, 100:104], flat[3:1004], flat[1004:1005], flat[1006:4001], long[:, :39999], tr.t()]
    outs = [out[:, 2:101], out[:, 104:108], res[3:1004], res[1005:1006], res[1007:4002], torch.zeros(3, 39999, device=DEV),
            torch.zeros(20, 30, device=DEV).t()]
    gs += [torch.randn(9, generator=g, device=DEV) for _ in range(1000)]
    outs += [torch.zeros(9, device=DEV) for _ in range(1000)]
    want_norm, want = O.clip([x.double().cpu().numpy() for x in gs], 2.0)
    first = adamw.clip_grads(gs, 2.0, outs)
    assert abs(float(first) - want_norm) <= 34 * U * want_norm
    for w, o in zip(want, outs):
        assert (np.abs(o.double().cpu().numpy() - w) <= 38 * U * np.abs(w)).all()
    written = sum(int((o != 0).sum()) for o in outs)
    assert written == int((out != 0).sum() + (res != 0).sum()) + sum(int((o != 0).sum()) for o in outs[5:])
    again = [torch.zeros_like(o) for o in outs]
    assert torch.equal(adamw.clip_grads(gs, 2.0, again), first)          # the same bits on every call
    assert all(torch.equal(a, b) for a, b in zip(again, outs))


def test_clip_on_another_stream_and_captured():
    gs = grads_of([(100,), (3000, 7), (40000,)], BF16, 9, 1.0)
    want = [torch.zeros(g.shape, device=DEV) for g in gs]
    norm = adamw.clip_grads(gs, 1.0, want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = [torch.zeros_like(w) for w in want]
    torch.cuda.synchronize()
    got = adamw.clip_grads(gs, 1.0, outs, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(got, norm) and all(torch.equal(a, b) for a, b in zip(outs, want))
    outs = [torch.zeros_like(w) for w in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        twice = [g * 2 for g in gs]            # a kernel before, not the library's
        got = adamw.clip_grads(twice, 2.0, outs)
        after = outs[0] + 0
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, 2 * norm) and torch.equal(after, outs[0])
    assert all(torch.equal(a, 2 * b) for a, b in zip(outs, want))


def test_clip_norm_only_empty_and_not_finite():
    gs = grads_of([(1000,), (50, 3)], F32, 2, 1.0)
    keep = clone(gs)
    want, _ = O.clip([f64(g) for g in gs], 1.0)
    assert abs(float(adamw.clip_grads(gs, float("inf"))) - want) <= 34 * U * want
    outs = [torch.full_like(g, 7.0) for g in gs]
    adamw.clip_grads(gs, float("inf"), outs)
    assert all((o == 7).all() for o in outs) and all(torch.equal(a, b) for a, b in zip(keep, gs))
    assert float(adamw.clip_grads([torch.empty(0, device=DEV)], 1.0)) == 0.0
    assert float(adamw.clip_grads([], 1.0)) == 0.0
    z = torch.zeros(100, device=DEV)
    assert float(adamw.clip_grads([z], 1.0)) == 0.0 and not z.any()
    for x in (float("inf"), float("nan")):
        g = torch.ones(300, device=DEV)
        g[17] = x
        norm = adamw.clip_grads([g], 1.0)
        assert not torch.isfinite(norm)
        assert torch.isnan(g[17]) and (torch.isnan(g).all() if x != x else (g[:17] == 0).all())


def test_clip_refusals():
    g = torch.ones(64, device=DEV)
    for bad in (0.0, -1.0, float("nan")):
        with pytest.raises(B.MuonError):
            adamw.clip_grads([g], bad)
    with pytest.raises(ValueError, match="shape"):
        adamw.clip_grads([g], 1.0, [torch.ones(63, device=DEV)])
    with pytest.raises(ValueError, match="bf16 or fp32"):
        adamw.clip_grads([g.half()], 1.0)
    with pytest.raises(ValueError, match="gaps"):
        adamw.clip_grads([torch.ones(8, 8, device=DEV)[:, ::2]], 1.0)
    with pytest.raises(B.MuonError, match="overlap"):
        adamw.clip_grads([g, g], 1.0)
    assert (g == 1).all()


@pytest.mark.parametrize("dtype, out_dtype", [(F32, F32), (BF16, F32), (F32, BF16), (BF16, BF16)])
@pytest.mark.parametrize("scale", [1e-42, 1e-30, 1e-24, 1e-19, 1e-17, 1e18, 1e20, 1e25, 1e35])
def test_clip_where_squares_leave_the_range_of_fp32(dtype, out_dtype, scale):
    """Gradients whose squares overflow or vanish in fp32: the norm and the factor are those of the definition.  Whole
    chunks, parts of them, rows, and elements that are 0 or far smaller than others."""
    gs = grads_of(SHAPES + [(40000,), (5, 17000)], dtype, 6, scale)
    gs[4][::2] = 0
    gs[-2][100:30000] *= 1e-12
    gs[-1] = gs[-1][:, :16999]
    want_norm, _ = O.clip([f64(g) for g in gs], 1.0)
    for max_norm in (1.0, want_norm / 2 or 2.0, 0.5, 1e-4):
        _, want = O.clip([f64(g) for g in gs], max_norm)
        outs = [torch.full(g.shape, float("nan"), dtype=out_dtype, device=DEV) for g in gs]
        got = adamw.clip_grads(gs, max_norm, outs)
        assert abs(float(got) - want_norm) <= 34 * U * want_norm + 2.0 ** -149
        for w, o in zip(want, outs):
            # what lies below the normal numbers of the result's type is rounded to its smallest steps
            tol = (38 * U + (2.0 ** -8 if out_dtype == BF16 else 0.0)) * np.abs(w) + (2.0 ** -133 if out_dtype == BF16 else 2.0 ** -148)
            assert (np.abs(f64(o) - w) <= tol).all()
    assert float(adamw.clip_grads(gs, float("inf"))) == float(got)


def test_clip_of_a_norm_beyond_fp32():
    """The norm is then infinite in fp32; the factor is formed from its value all the same."""
    for dtype in (F32, BF16):
        for n in (300, 40000):
            g = torch.full((n,), 3e38, dtype=dtype, device=DEV)
            g[1::2] *= -1
            keep = g.clone()
            for max_norm in (1.0, 1e-3):
                out = torch.zeros(n, device=DEV)
                norm = adamw.clip_grads([g], max_norm, [out])
                assert norm == float("inf") and torch.equal(g, keep)
                _, (want,) = O.clip([f64(g)], max_norm)
                assert (np.abs(f64(out) - want) <= 38 * U * np.abs(want)).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_what_is_written_counts_as_changed(bits):
    """Autograd finds that a tensor it has saved was changed since."""
    p, g, m, v, s = make(1000, F32, F32, bits, 4)
    p.requires_grad_()
    loss = (p * p).sum()
    written = [p, m, v] + ([s] if bits == 8 else [])
    before = [t._version for t in written]
    read = g._version
    with pytest.raises(B.MuonError):
        step_all([(p.detach(), g, m, v, s)], 0, 1)       # step 0: refused, nothing written
    assert [t._version for t in written] == before
    with torch.no_grad():
        step_all([(p, g, m, v, s)], 1, 1)
    assert [t._version for t in written] == [b + 1 for b in before] and g._version == read
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_clipped_gradients_count_as_changed():
    g, out = torch.ones(100, device=DEV), torch.zeros(100, device=DEV)
    version = lambda: (g._version, out._version)  # noqa: E731
    a, b = version()
    adamw.clip_grads([g], 1.0, [out])
    assert version() == (a, b + 1)
    adamw.clip_grads([g], float("inf"))              # the norm alone
    assert version() == (a, b + 1)
    adamw.clip_grads([g], 1.0)
    assert version() == (a + 1, b + 1)
    with torch.inference_mode():
        t = torch.ones(100, device=DEV)              # has no version
        adamw.clip_grads([t], 1.0)
    adamw.clip_grads([t], 0.5)
    assert abs(float(t.norm()) - 0.5) < 1e-5


def test_the_norm_keeps_no_workspace():
    """Norms that a program collects for its log cost their own bytes."""
    norm = adamw.clip_grads([torch.ones(100, device=DEV)], 1.0)
    assert float(norm) == 10.0 and norm.untyped_storage().nbytes() <= 64
