"""A training step from token ids to the optimizers: embedding, router, dispatch, gated experts (activations in their own type
or in 8 bits), combine, and their gradients, against the same model in elementary float64 operations."""
import numpy as np
import pytest
import torch
import torch.nn.functional as F

from muon_newton_schulz_gb300 import binding as B
from muon_newton_schulz_gb300 import checkpoint, embedding, ffn, moe
from muon_newton_schulz_gb300.train_moe import Model, main, train

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def kept8(x):
    return checkpoint.unpack(checkpoint.pack(x.float())).double()


class Rounded(torch.autograd.Function):
    """Values that count as x in the forward pass's later use alone: the gradient passes through."""
    @staticmethod
    def forward(ctx, x, to):
        return to

    @staticmethod
    def backward(ctx, d):
        return d, None


def plain(model, ids):
    """The model's logits in float64 for the routes that its own router takes, with the roundings to bf16 that the block documents
    (the dispatched rows, h, y and the combined rows)."""
    layer = model.layer
    p = {k: v.double() for k, v in model.named_parameters()}
    x = p["embedding"][ids] * 2.0
    h = x / (x.square().mean(1, keepdim=True) + torch.finfo(torch.float32).eps).sqrt() * p["layer.gain"]
    logits = h @ p["layer.router"].t()
    with torch.no_grad():        # the router's choices, and the rows that its capacity leaves
        x32 = model.embedding[ids] * 2.0
        h32 = F.rms_norm(x32, (x32.shape[1],)) * layer.gain
        top = (h32 @ layer.router.t()).topk(layer.topk, dim=1).indices
        capacity = int(layer.capacity_factor * len(ids) * layer.topk / layer.experts)
        route = moe.sort_tokens(top, layer.experts, capacity=max(8, -(-capacity // 8) * 8))
    weights = torch.softmax(logits.gather(1, top), 1)
    out = torch.zeros_like(x)
    row = route.row
    bf16 = lambda t: Rounded.apply(t, t.detach().to(torch.bfloat16).double())  # noqa: E731
    rows = bf16(h)
    for e in range(layer.experts):
        for k in range(layer.topk):
            t = torch.nonzero((top[:, k] == e) & (row[:, k] >= 0)).flatten()
            g, u = rows[t] @ p["layer.gate"][e].t(), rows[t] @ p["layer.up"][e].t()
            y = bf16(bf16(F.silu(g) * u) @ p["layer.down"][e].t())
            out = out.index_add(0, t, weights[t, k].unsqueeze(1) * y)
    z = x + bf16(out)
    return z / (z.square().mean(1, keepdim=True) + torch.finfo(torch.float32).eps).sqrt() @ p["head"].t()


@pytest.mark.parametrize("bits", [None, 8])
def test_gradients_of_a_model(bits):
    """Each rounding to bf16 is at most 2^-8 of its value, 2^-8 / sqrt(3) in the mean square, and their signs are independent.
    On the way to a gradient there are at most nine of them one after another (the rows, h, y, the sum; backward the same
    four and a gradient in bf16), so 3 * 2^-8 / sqrt(3) in the norm; twice that is allowed for.  With 8 bits three more, each
    2^-4 / sqrt(3) at most (the saved x, g and u): 2^-4, twice that."""
    torch.manual_seed(3)
    model = Model(vocab=200, hidden=128, ffn=192, experts=4, gated=True, saved_bits=bits).to(DEV)
    ids = torch.randint(0, 200, (300,), device=DEV)
    target = torch.randint(0, 200, (300,), device=DEV)
    loss = F.cross_entropy(model(ids), target)
    loss.backward()
    got = {k: v.grad.double() for k, v in model.named_parameters()}
    model.zero_grad()
    want = F.cross_entropy(plain(model, ids), target)
    want.backward()
    bound = 2 * 3 * 2.0 ** -8 / 3 ** 0.5 + (2 * 2.0 ** -4 if bits else 0.0)
    assert abs(loss.item() - want.item()) <= 2.0 ** -8 * want.item()
    for k, v in model.named_parameters():
        assert torch.isfinite(got[k]).all() and v.grad is not None
        w = v.grad.double()
        assert float((got[k] - w).norm()) <= bound * float(w.norm()), (k, float((got[k] - w).norm() / w.norm()))


@pytest.mark.parametrize("bits", [None, 8])
def test_training_runs(bits, capsys):
    losses = train(steps=3, tokens=512, gated=True, saved_bits=bits, seed=1)
    again = train(steps=3, tokens=512, gated=True, saved_bits=bits, seed=1)
    assert losses.shape == (3,) and torch.isfinite(losses).all()
    assert torch.equal(losses[:1], again[:1])
    main(["--steps", "2", "--tokens", "256", "--gated", *(["--saved-bits", "8"] if bits else [])])
    assert "loss" in capsys.readouterr().out


def test_saved_bits_go_with_gated(capsys):
    with pytest.raises(SystemExit):
        main(["--saved-bits", "8"])


def test_memory_that_is_kept():
    """8 bits: x, g and u in one byte an element and a scale byte for 32; 16 bits: g, u and h in two, x by reference."""
    torch.manual_seed(0)
    R, H, W = 4096, 512, 1024
    x = torch.randn(R, H, device=DEV, dtype=torch.bfloat16)
    w = [torch.randn(*s, device=DEV, dtype=torch.bfloat16).mul_(0.05) for s in ((W, H), (W, H), (H, W))]
    size = lambda saved: sum(t.numel() * t.element_size() for t in saved.kept)  # noqa: E731
    _, own = ffn.gated_ffn_saved(x, *w)
    _, eight = ffn.gated_ffn_saved(x, *w, saved_bits=8)
    assert size(own) == R * (3 * W * 2 + 2 * W // 32) and own.x.data_ptr() == x.data_ptr()
    assert size(eight) == R * ((2 * W + H) + (2 * W + H) // 32) and eight.x is None


def test_a_wait_that_runs_out_is_reported(monkeypatch):
    """A handle made while the test hook is set issues no loads in the first product: its waits run out after a second, the
    kernels return, and the status says so; the next call on another handle is right."""
    torch.manual_seed(0)
    x = torch.randn(300, 128, device=DEV, dtype=torch.bfloat16)
    w = [torch.randn(*s, device=DEV, dtype=torch.bfloat16).mul_(0.1) for s in ((256, 128), (256, 128), (128, 256))]
    want = ffn.gated_ffn(x, *w)
    st, plain_handle = B.muon_create(None, 0)
    assert st == B.MUON_OK and B.muon_check_status(plain_handle, None, 0) == B.MUON_OK
    monkeypatch.setenv("MUON_GB300_TEST_WITHHOLD_LOADS", "1")
    st, h = B.muon_create(None, 0)
    monkeypatch.delenv("MUON_GB300_TEST_WITHHOLD_LOADS")
    assert st == B.MUON_OK
    shape = B.muon_ffn_shape(300, 128, 256, 1, B.MUON_BF16, B.MUON_SILU, 0)
    st, need = B.muon_ffn_workspace_size(shape, False)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    y = torch.empty_like(x)
    stack = lambda t: B.muon_stack(t.data_ptr(), (0, t.stride(0), 1))  # noqa: E731
    stacks = [stack(t) for t in w]
    torch.cuda.synchronize()
    run = lambda handle: B.muon_ffn_forward(handle, shape, None, None, x.data_ptr(), 128, *stacks, y.data_ptr(), 128, None,  # noqa: E731
                                            ws.data_ptr(), need, 0)
    assert run(h) == B.MUON_OK
    torch.cuda.synchronize()
    assert B.muon_check_status(h, None, 0) == B.MUON_ERR_TIMEOUT
    assert B.muon_check_status(h, None, 0) == B.MUON_OK                 # read and cleared
    assert run(plain_handle) == B.MUON_OK
    torch.cuda.synchronize()
    assert B.muon_check_status(plain_handle, None, 0) == B.MUON_OK
    assert torch.equal(y, want) and torch.equal(ffn.gated_ffn(x, *w), want)
    B.muon_destroy(h)
    B.muon_destroy(plain_handle)


def in_a_thread_that_withholds_loads(monkeypatch, f):
    """f in a new thread, whose handle's first feed-forward product issues no loads."""
    import threading
    out = []

    def work():
        monkeypatch.setenv("MUON_GB300_TEST_WITHHOLD_LOADS", "1")
        B.thread_handle(0)
        monkeypatch.delenv("MUON_GB300_TEST_WITHHOLD_LOADS")
        try:
            out.append(f())
        except Exception as e:
            out.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    return out[0]


def test_a_wait_that_runs_out_in_another_thread_is_reported(monkeypatch):
    torch.manual_seed(0)
    x = torch.randn(300, 128, device=DEV, dtype=torch.bfloat16)
    w = [torch.randn(*s, device=DEV, dtype=torch.bfloat16).mul_(0.1) for s in ((256, 128), (256, 128), (128, 256))]
    want = ffn.gated_ffn(x, *w)
    assert ffn.check_status() == ffn.check_status(DEV) == ffn.check_status(0) == B.MUON_OK
    torch.cuda.synchronize()
    assert isinstance(in_a_thread_that_withholds_loads(monkeypatch, lambda: ffn.gated_ffn(x, *w)), torch.Tensor)
    torch.cuda.synchronize()
    assert ffn.check_status(DEV) == B.MUON_ERR_TIMEOUT
    assert ffn.check_status(DEV) == B.MUON_OK                           # read and cleared
    assert torch.equal(ffn.gated_ffn(x, *w), want) and ffn.check_status() == B.MUON_OK
    with pytest.raises(ValueError, match="CUDA"):
        ffn.check_status("cpu")
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            y = ffn.gated_ffn(x, *w)
            with pytest.raises(RuntimeError, match="captured"):
                ffn.check_status()
    graph.replay()
    assert torch.equal(y, want)


def test_a_training_run_whose_block_gave_up_says_so(monkeypatch):
    e = in_a_thread_that_withholds_loads(monkeypatch, lambda: train(steps=1, tokens=256, gated=True))
    assert isinstance(e, B.MuonError) and e.status == B.MUON_ERR_TIMEOUT
    assert torch.isfinite(train(steps=1, tokens=256, gated=True)).all()


def test_a_handle_is_told_of_its_own_waits_alone(monkeypatch):
    monkeypatch.setenv("MUON_GB300_TEST_WITHHOLD_LOADS", "1")
    bad, other = B.muon_create(None, 0)[1], B.muon_create(None, 0)[1]
    monkeypatch.delenv("MUON_GB300_TEST_WITHHOLD_LOADS")
    good, third = B.muon_create(None, 0)[1], B.muon_create(None, 0)[1]
    x = torch.randn(300, 128, device=DEV, dtype=torch.bfloat16)
    w = [torch.randn(*s, device=DEV, dtype=torch.bfloat16).mul_(0.1) for s in ((256, 128), (256, 128), (128, 256))]
    shape = B.muon_ffn_shape(300, 128, 256, 1, B.MUON_BF16, B.MUON_SILU, 0)
    need = B.muon_ffn_workspace_size(shape, False)[1]
    ws, y = torch.empty(need, dtype=torch.uint8, device=DEV), torch.empty_like(x)
    stacks = [B.muon_stack(t.data_ptr(), (0, t.stride(0), 1)) for t in w]
    torch.cuda.synchronize()

    def run(h):
        assert B.muon_ffn_forward(h, shape, None, None, x.data_ptr(), 128, *stacks, y.data_ptr(), 128, None, ws.data_ptr(), need, 0) == B.MUON_OK

    run(bad), run(good)
    assert B.muon_ffn_check_status(good, 0) == B.muon_check_status(good, None, 0) == ffn.check_status() == B.MUON_OK
    assert B.muon_ffn_check_status(bad, 0) == B.MUON_ERR_TIMEOUT and B.muon_last_error_message(bad)
    assert B.muon_ffn_check_status(bad, 0) == B.MUON_OK
    # handles that share a word: each time-out is reported once, to either
    for h in (other, third):
        assert B.muon_ffn_share_status(h, 15) == B.MUON_OK
    run(other)
    assert B.muon_ffn_check_status(good, 0) == B.MUON_OK
    assert B.muon_ffn_check_status(third, 0) == B.MUON_ERR_TIMEOUT and B.muon_ffn_check_status(other, 0) == B.MUON_OK
    assert B.muon_ffn_share_status(third, 0) == B.MUON_OK
    run(other)
    assert B.muon_ffn_check_status(third, 0) == B.MUON_OK and B.muon_ffn_check_status(other, 0) == B.MUON_ERR_TIMEOUT
    for h in (bad, other, good, third):
        B.muon_destroy(h)


def test_a_captured_training_step():
    """Forward and backward passes through autograd in a graph, replayed on other inputs."""
    torch.manual_seed(0)
    table = torch.nn.Parameter(torch.randn(60, 128, device=DEV))
    w = [torch.nn.Parameter(torch.randn(3, *s, device=DEV, dtype=torch.bfloat16).mul_(0.1)) for s in ((192, 128), (192, 128), (128, 192))]
    leaves = [table, *w]
    ids = torch.randint(0, 60, (200,), device=DEV)
    top = torch.randint(0, 3, (200, 1), device=DEV)

    def step():
        x = embedding.embed(ids, table, scale=2.0)
        route = moe.sort_tokens(top, 3)
        y = ffn.gated_ffn(moe.dispatch(x.to(torch.bfloat16), route), *w, route, saved_bits=8)
        moe.combine(y, None, route).float().square().sum().backward()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            for p in leaves:
                p.grad = None
            step()
    torch.cuda.current_stream().wait_stream(side)
    for p in leaves:
        p.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    captured = [p.grad for p in leaves]
    for seed in range(2):
        g = torch.Generator().manual_seed(seed)
        ids.copy_(torch.randint(-3, 60, (200,), generator=g))
        top.copy_(torch.randint(-1, 3, (200, 1), generator=g))
        graph.replay()
        got = [t.clone() for t in captured]
        for p in leaves:
            p.grad = None
        step()
        assert all(torch.equal(a, p.grad) for a, p in zip(got, leaves))


def test_no_rows():
    for dtype in (torch.float32, torch.bfloat16):
        for h, f in ((64, 96), (33, 65)):
            x = torch.zeros(0, h, device=DEV, dtype=dtype, requires_grad=True)
            w = [torch.randn(*s, device=DEV, dtype=dtype).requires_grad_() for s in ((f, h), (f, h), (h, f))]
            for bits in (None, 8):
                y = ffn.gated_ffn(x, *w, saved_bits=bits)
                y.sum().backward()
                assert y.shape == (0, h) and x.grad.shape == (0, h) and all((t.grad == 0).all() for t in w)
