"""The torch.optim front end of AdamW, clipping through it, and the small
mixture-of-experts training that uses every operator together."""
import copy
import io
import math

import pytest
import torch

from muon_newton_schulz_gb300 import adamw
from muon_newton_schulz_gb300.optim import AdamW, clip_grad_norm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def raw(t):
    return t.detach().reshape(-1).view(torch.uint8)


def params(dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    shapes = [(100, 64), (64,), (), (3, 5, 7), (5000,)]
    return [torch.nn.Parameter((torch.randn(s, generator=g) * 0.1).to(dtype).to(DEV)) for s in shapes]


def fill(ps, seed):
    g = torch.Generator().manual_seed(seed)
    for p in ps:
        p.grad = (torch.randn(p.shape, generator=g) * 1e-2).to(p.dtype).to(DEV)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_optimizer_equals_direct_steps(bits, dtype):
    ps = params(dtype)
    copies = [p.detach().clone() for p in ps]
    opt = AdamW([{"params": ps[:2], "lr": 1e-3}, {"params": ps[2:], "weight_decay": 0.0, "betas": (0.8, 0.9)}], lr=2e-3,
                state_bits=bits, min_8bit_size=100, seed=5)
    states = []
    for p in copies:
        s = adamw.state8_like(p) if bits == 8 and p.numel() >= 100 else None
        states.append(s or (torch.zeros_like(p, dtype=torch.float32), torch.zeros_like(p, dtype=torch.float32), None))
    for t in range(1, 4):
        fill(ps, t)
        if t == 2:
            ps[1].grad = None
        opt.step()
        for idx, lr, wd, betas in (([0, 1], 1e-3, 0.1, (0.9, 0.95)), ([2, 3, 4], 2e-3, 0.0, (0.8, 0.9))):
            idx = [i for i in idx if ps[i].grad is not None]
            adamw.adamw_step([copies[i] for i in idx], [ps[i].grad for i in idx], [states[i][0] for i in idx],
                             [states[i][1] for i in idx], [states[i][2] for i in idx], lr=lr, weight_decay=wd, betas=betas,
                             step=[t - 1 if i == 1 and t == 3 else t for i in idx], seed=[5 + i for i in idx])
    for p, c, (m, v, s) in zip(ps, copies, states):
        st = opt.state[p]
        assert torch.equal(p, c)
        assert torch.equal(raw(st["exp_avg"]), raw(m))
        assert torch.equal(raw(st["exp_avg_sq"]), raw(v))
        assert ("scales" in st) == (s is not None)


def test_agrees_with_torch_adamw():
    """The same formula as torch's AdamW: after ten steps the fp32 parameters agree to a few parts in 10^6 of their
    movement (both round an update of relative size 2^-22 or so ten times)."""
    ps, qs = params(torch.float32), params(torch.float32)
    start = [p.detach().clone() for p in ps]
    a = AdamW(ps, lr=1e-2, weight_decay=0.05)
    b = torch.optim.AdamW(qs, lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.05)
    for t in range(10):
        fill(ps, t)
        fill(qs, t)
        a.step()
        b.step()
    for p, q, s in zip(ps, qs, start):
        assert float((p - q).detach().abs().max()) <= 10 * (2.0 ** -20 * 1e-2 + 2.0 ** -23 * float(s.abs().max() + 0.1))


def test_state_dict_keeps_types_and_continues():
    for bits in (32, 8):
        ps = params(torch.bfloat16)
        opt = AdamW(ps, state_bits=bits, min_8bit_size=100)
        for t in range(2):
            fill(ps, t)
            opt.step()
        buf = io.BytesIO()
        torch.save(opt.state_dict(), buf)
        buf.seek(0)
        qs = [torch.nn.Parameter(p.detach().clone()) for p in ps]
        other = AdamW(qs, state_bits=bits, min_8bit_size=100)
        saved = torch.load(buf, weights_only=True)
        keep = copy.deepcopy(saved)
        other.load_state_dict(saved)
        for p, q in zip(ps, qs):
            assert {k: v.dtype for k, v in opt.state[p].items() if k != "step"} == {
                k: v.dtype for k, v in other.state[q].items() if k != "step"}
        fill(ps, 7)
        fill(qs, 7)
        opt.step()
        other.step()
        for p, q in zip(ps, qs):
            assert torch.equal(p, q) and opt.state[p]["step"] == other.state[q]["step"] == 3
            assert torch.equal(raw(opt.state[p]["exp_avg"]), raw(other.state[q]["exp_avg"]))
        for i, st in saved["state"].items():      # the loaded dict was not stepped
            assert torch.equal(raw(st["exp_avg"]), raw(keep["state"][i]["exp_avg"]))


def test_gradients_of_another_layout_and_closures():
    p = torch.nn.Parameter(torch.randn(30, 40, device=DEV).t())
    q = torch.nn.Parameter(p.detach().clone())
    assert p.stride() != (30, 1)
    a, b = AdamW([p]), AdamW([q])
    g = torch.randn(40, 30, device=DEV)
    p.grad, q.grad = g.clone(), g.t().contiguous().t()
    assert a.step(lambda: 2.5) == 2.5
    b.step()
    assert torch.equal(p, q)
    AdamW([torch.nn.Parameter(torch.zeros(3, device=DEV))]).step()     # no gradient: nothing to do


def test_rejections():
    for bad, why in ((torch.zeros(4, dtype=torch.float16, device=DEV), "bf16 or fp32"), (torch.zeros(4), "CUDA"),
                     (torch.zeros(8, 8, device=DEV)[:, ::2], "gaps")):
        with pytest.raises(ValueError, match=why):
            AdamW([torch.nn.Parameter(bad)])
    p = [torch.nn.Parameter(torch.zeros(4, device=DEV))]
    for kw, why in ((dict(lr=-1.0), "learning rate"), (dict(betas=(1.0, 0.9)), "betas"), (dict(eps=-1.0), "eps"),
                    (dict(state_bits=16), "state_bits")):
        with pytest.raises(ValueError, match=why):
            AdamW(p, **kw)


def test_clip_grad_norm():
    ps = params(torch.float32)
    fill(ps, 1)
    ps[3].grad = None
    want = math.sqrt(sum(float(p.grad.double().square().sum()) for p in ps if p.grad is not None))
    norm = clip_grad_norm(ps, want / 2)
    assert abs(float(norm) - want) <= 1e-5 * want
    left = math.sqrt(sum(float(p.grad.double().square().sum()) for p in ps if p.grad is not None))
    assert abs(left - want / 2) <= 1e-5 * want


@pytest.mark.parametrize("bits", [32, 8])
def test_mixture_of_experts_training(bits):
    """The loss starts near log(512) and falls well towards the data's entropy (0.33 for the noise's choice and 0.1
    of log(512)): below a third of its start within 60 steps."""
    from muon_newton_schulz_gb300.train_moe import train
    losses = train(steps=60, state_bits=bits, seed=3)
    assert torch.isfinite(losses).all()
    assert losses[0] > 5.5 and losses[-5:].mean() < losses[0] / 3


def test_chains_of_dependent_launches():
    """The library's kernels are launched before those they depend on have finished.  Chains of them, of torch's kernels
    and of Muon steps give the same bits as with a wait after every call, at sizes where launches are short and long."""
    from muon_newton_schulz_gb300 import binding as B
    from muon_newton_schulz_gb300 import moe

    def chain(seed, T, H, wait):
        def done():
            if wait:
                torch.cuda.synchronize()

        g = torch.Generator(device=DEV).manual_seed(seed)
        E, K = 24, 3
        W = torch.randn(96, 160, generator=g, device=DEV)
        M = torch.zeros_like(W)
        muon = B.MuonStep(0)
        p = torch.zeros(T, H, device=DEV)
        m, v, s = adamw.state8_like(p)
        q, m32, v32 = torch.zeros(H, device=DEV), torch.zeros(H, device=DEV), torch.zeros(H, device=DEV)
        out = []
        for t in range(1, 13):
            x = torch.randn(T, H, generator=g, device=DEV)
            done()
            ids = torch.randn(T, E, generator=g, device=DEV).topk(K, 1).indices
            done()
            r = moe.sort_tokens(ids, E, align=4)
            done()
            xs = moe.dispatch(x, r)
            done()
            w = torch.rand(T, K, generator=g, device=DEV)
            done()
            y = moe.combine(xs, w, r)
            done()
            dy, dw = moe.combine_backward(y, xs, w, r)
            done()
            dx = moe.dispatch_backward(dy, r)
            done()
            col = dx.sum(0)
            done()
            norm = adamw.clip_grads([dx, col], 1.0)
            done()
            adamw.adamw_step([p, q], [dx, col], [m, m32], [v, v32], [s, None], lr=1e-2, step=t, seed=seed)
            done()
            G = (p[:1, :1] + torch.randn(96, 160, generator=g, device=DEV)) * (1 + norm)
            done()
            muon.step([W], [G], [M], [1e-2])
            done()
            x = x + W[0, 0]
            out += [r.row, dw, norm, x[0].clone()]
        torch.cuda.synchronize()
        assert muon.check_status() == B.MUON_OK
        muon.close()
        return out + [p, q, W, M, m.view(torch.uint8), v.view(torch.uint8)]

    for seed, T, H in ((1, 3, 8), (2, 900, 64), (3, 3000, 1031), (4, 20000, 256)):
        for a, b in zip(chain(seed, T, H, False), chain(seed, T, H, True)):
            assert torch.equal(a, b), (seed, T, H)


def test_inputs_from_another_stream_after_an_event():
    """A call whose inputs another stream writes, ordered by an event, while the call's own stream still runs a kernel of
    the library before it: it sees what the event promises."""
    from muon_newton_schulz_gb300 import moe
    T, K, E, H = 4096, 2, 16, 512
    other = torch.cuda.Stream()
    mine = torch.cuda.Stream()
    base = torch.randn(T, H, device=DEV)
    ids = torch.randint(0, E, (T, K), device=DEV)
    big = torch.randn(1 << 26, device=DEV)
    p, m, v = (torch.zeros(1 << 24, device=DEV) for _ in range(3))
    g = torch.randn(1 << 24, device=DEV)
    torch.cuda.synchronize()
    for i in range(20):
        x = torch.zeros(T, H, device=DEV)
        late = torch.full((T, K), -1, dtype=torch.int64, device=DEV)
        torch.cuda.synchronize()
        with torch.cuda.stream(other):
            for _ in range(1 + i % 4):
                big.mul_(1.0000001)                 # some hundred us
            x.copy_(base + i)
            late.copy_((ids + i) % E)
            ready = torch.cuda.Event()
            ready.record()
        with torch.cuda.stream(mine):
            adamw.adamw_step([p], [g], [m], [v], lr=1e-3, step=i + 1)     # still running when the next calls are made
            mine.wait_event(ready)
            r = moe.sort_tokens(late, E)
            xs = moe.dispatch(x, r)
            norm = adamw.clip_grads([x], 1e9)
        mine.synchronize()
        want = moe.sort_tokens((ids + i) % E, E)
        torch.cuda.synchronize()
        assert torch.equal(r.row, want.row) and torch.equal(r.counts, want.counts)
        assert torch.equal(xs, moe.dispatch(base + i, want))
        assert torch.equal(norm, adamw.clip_grads([base + i], 1e9))


@pytest.mark.parametrize("bits", [32, 8])
def test_capturing_a_step_is_refused(bits):
    """The step number lives on the host: a replay would repeat the captured step and its random bits."""
    ps, qs = params(torch.float32), params(torch.float32)
    a, b = (AdamW(x, state_bits=bits, min_8bit_size=100) for x in (ps, qs))
    fill(ps, 1)
    fill(qs, 1)
    for steps in (0, 1):         # before there is any state, and after
        keep = [p.detach().clone() for p in ps]
        with pytest.raises(RuntimeError, match="CUDA graph"):
            with torch.cuda.graph(torch.cuda.CUDAGraph()):
                a.step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, k) for p, k in zip(ps, keep))
        assert [a.state[p]["step"] for p in ps if a.state[p]] == [steps] * (len(ps) if steps else 0)
        a.step()
        b.step()
    for p, q in zip(ps, qs):
        assert torch.equal(p, q) and torch.equal(raw(a.state[p]["exp_avg"]), raw(b.state[q]["exp_avg"]))


def test_clip_grad_norm_of_one_tensor():
    p = torch.nn.Parameter(torch.zeros(30, 40, device=DEV))
    p.grad = torch.ones(30, 40, device=DEV)
    for x in (p, (q for q in [p])):
        p.grad.fill_(1.0)
        assert abs(float(clip_grad_norm(x, 1.0)) - 1200 ** 0.5) < 1e-4
        assert abs(float(p.grad.norm()) - 1.0) < 1e-5
    p.grad = None
    assert clip_grad_norm(p, 1.0).device == p.device and float(clip_grad_norm([p], 1.0)) == 0.0
