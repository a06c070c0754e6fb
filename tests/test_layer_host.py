"""Embedding rows and activations in 8 bits without a GPU: the C ABI validates on a host-only handle before anything could
be launched, the torch layer refuses what the library cannot take, and the oracle's codes agree with torch's float8 types."""
import os
import re

import numpy as np
import pytest
import torch

import oracle.layer_oracle as L
from muon_newton_schulz_gb300 import binding as B
from muon_newton_schulz_gb300 import checkpoint, embedding

BASE, MB = 1 << 30, 1 << 20
F32, BF16 = B.MUON_F32, B.MUON_BF16


@pytest.fixture(scope="module")
def h():
    B.load_library(build_if_missing=True)
    st, handle = B.muon_create(None, -1)
    assert st == B.MUON_OK
    yield handle
    B.muon_destroy(handle)


def _embed(h, ids=BASE, bits=64, tokens=10, table=BASE + MB, ldt=64, vocab=100, hidden=64, dtype=F32, scale=1.0,
           out=BASE + 2 * MB, ldo=64):
    return B.muon_embed(h, ids, bits, tokens, table, ldt, vocab, hidden, dtype, scale, out, ldo, 0)


def _grad(h, ids=BASE, bits=64, tokens=10, dout=BASE + MB, ldd=64, vocab=100, hidden=64, dtype=F32, scale=1.0,
          dtable=BASE + 2 * MB, ldt=64, ws=BASE + 3 * MB, ws_bytes=MB):
    return B.muon_embed_backward(h, ids, bits, tokens, dout, ldd, vocab, hidden, dtype, scale, dtable, ldt, ws, ws_bytes, 0)


def test_embed_refusals(h):
    assert _embed(h) == _embed(h, bits=32, ids=BASE + 4) == _embed(h, dtype=BF16, table=BASE + MB + 2) == B.MUON_ERR_UNSUPPORTED
    assert _embed(h, vocab=0, table=None) == B.MUON_ERR_UNSUPPORTED      # every id is outside: rows of zeros
    assert _embed(h, tokens=0, ids=None) == _embed(h, hidden=0) == B.MUON_OK
    for kw in (dict(ids=None), dict(ids=BASE + 4), dict(bits=16), dict(tokens=-1), dict(tokens=1 << 31), dict(table=None),
               dict(ldt=63), dict(vocab=-1), dict(vocab=(1 << 31) - 1), dict(hidden=-1), dict(dtype=2), dict(out=None),
               dict(ldo=63), dict(out=BASE + MB + 256), dict(out=BASE + 72), dict(table=BASE + MB + 2)):
        assert _embed(h, **kw) == B.MUON_ERR_INVALID_ARG, kw
        assert B.muon_last_error_message(h)


def test_embed_backward_refusals(h):
    assert _grad(h) == _grad(h, vocab=1 << 20, dtable=1 << 40) == B.MUON_ERR_UNSUPPORTED
    assert _grad(h, tokens=0, ids=None, dout=None, ws=None, ws_bytes=0) == B.MUON_ERR_UNSUPPORTED   # zeros are written
    assert _grad(h, vocab=0, dtable=None) == _grad(h, hidden=0) == B.MUON_OK
    need = B.muon_embed_backward_workspace_size(10, 100, 64)[1]
    assert 0 < need <= MB
    for kw in (dict(ws=None), dict(ws=BASE + 3 * MB + 8), dict(ws_bytes=need - 1)):
        assert _grad(h, **kw) == B.MUON_ERR_WORKSPACE, kw
    for kw in (dict(ids=None), dict(bits=8), dict(tokens=-1), dict(dout=None), dict(ldd=63), dict(vocab=-1), dict(hidden=-1),
               dict(dtype=7), dict(dtable=None), dict(ldt=3), dict(dtable=BASE + MB), dict(ws=BASE + MB), dict(dtable=BASE + 8)):
        assert _grad(h, **kw) == B.MUON_ERR_INVALID_ARG, kw


@pytest.mark.parametrize("tokens, vocab, hidden", [(0, 5, 7), (1, 1, 1), (512, 100, 64), (513, 100, 64), (2048, 1 << 30, 3),
                                                   (65536, 65536, 2048), ((1 << 31) - 1, (1 << 31) - 2, 16)])
def test_embed_workspace(h, tokens, vocab, hidden):
    st, need = B.muon_embed_backward_workspace_size(tokens, vocab, hidden)
    assert st == B.MUON_OK
    chunks = -(-tokens // 8)
    assert need <= 16 * tokens + 4 * 152 * 4096 + chunks * 2 * 4 * (hidden + 255) + 8 * 256
    assert need >= (8 * tokens if tokens else 0)


def test_embed_workspace_refusals(h):
    for bad in ((-1, 5, 5), (5, -1, 5), (5, 5, -1), (1 << 31, 5, 5), (5, (1 << 31) - 1, 5), ((1 << 31) - 1, 5, 1 << 40)):
        assert B.muon_embed_backward_workspace_size(*bad)[0] == B.MUON_ERR_INVALID_ARG, bad


@pytest.mark.parametrize("pack", [True, False])
def test_saved8_refusals(h, pack):
    def call(x=BASE, ldx=100, rows=10, cols=100, dtype=F32, codes=BASE + MB, scales=BASE + 2 * MB):
        if pack:
            return B.muon_pack8(h, x, ldx, rows, cols, dtype, codes, scales, 0)
        return B.muon_unpack8(h, codes, scales, rows, cols, x, ldx, dtype, 0)

    assert call() == call(ldx=101) == call(dtype=BF16, x=BASE + 2) == call(codes=BASE + MB + 1) == B.MUON_ERR_UNSUPPORTED
    assert call(rows=0) == call(cols=0) == B.MUON_OK
    for kw in (dict(x=None), dict(codes=None), dict(scales=None), dict(x=BASE + 2), dict(ldx=99), dict(rows=-1), dict(cols=-1),
               dict(dtype=3), dict(rows=1 << 40), dict(codes=BASE + 3996), dict(scales=BASE + 8)):
        assert call(**kw) == B.MUON_ERR_INVALID_ARG, kw
    # codes and scales are both written by pack, both only read by unpack
    assert call(scales=BASE + MB + 999) == (B.MUON_ERR_INVALID_ARG if pack else B.MUON_ERR_UNSUPPORTED)


def test_saved8_takes_a_flag_for_special_values(h):
    for call in (lambda d: B.muon_pack8(h, BASE, 100, 10, 100, d, BASE + MB, BASE + 2 * MB, 0),
                 lambda d: B.muon_unpack8(h, BASE + MB, BASE + 2 * MB, 10, 100, BASE, 100, d, 0)):
        assert call(F32 | B.MUON_SAVED8_SPECIAL) == call(BF16 | B.MUON_SAVED8_SPECIAL) == B.MUON_ERR_UNSUPPORTED
        assert call(3 | B.MUON_SAVED8_SPECIAL) == call(B.MUON_SAVED8_SPECIAL << 1) == B.MUON_ERR_INVALID_ARG


def test_torch_layer_refuses():
    i, t = torch.zeros(3, dtype=torch.int64), torch.zeros(5, 4)
    with pytest.raises(ValueError, match="CUDA"):
        embedding.embed(i, t)
    with pytest.raises(ValueError, match="int32 or int64"):
        embedding.embed(t, t)
    with pytest.raises(ValueError, match="CUDA"):
        embedding.embed_backward(torch.zeros(3, 4), i, 5)
    with pytest.raises(TypeError):
        embedding.embed_backward(torch.zeros(3, 4), i, 5.0)
    with pytest.raises(ValueError, match="CUDA"):
        checkpoint.pack(t)
    with pytest.raises(ValueError, match="bf16 or fp32"):
        checkpoint.pack(i)
    with pytest.raises(ValueError, match="dimension"):
        checkpoint.pack(torch.zeros(()))
    p = checkpoint.Packed(torch.zeros(2, 40).to(torch.float8_e4m3fn), torch.zeros(2, 2, dtype=torch.uint8).view(torch.float8_e8m0fnu), torch.float32)
    with pytest.raises(ValueError, match="CUDA"):
        checkpoint.unpack(p)
    with pytest.raises(ValueError, match="bf16 or fp32"):
        checkpoint.unpack(p, torch.float16)
    calls = B.torch_calls()
    assert calls.embed(i, t, 1.0, 0, 0) is None and calls.embed_backward(t, i, 5, 1.0, 0, 0) is None
    assert calls.pack8(t, 0, 0) is None and calls.unpack8(t, t, False, 0, 0) is None and calls.pack8(3, 0, 0) is None


def test_saved_in_8_bits_leaves_cpu_tensors_alone():
    x = torch.randn(400, 400, requires_grad=True)
    with checkpoint.saved_in_8_bits(min_elements=1):
        y = (x * x).sum()
    y.backward()
    assert torch.equal(x.grad, 2 * x)


def test_statistics_are_known():
    """What operations save beside their activations, through torch's own hooks."""
    F = torch.nn.functional
    seen = []

    def keep(t):
        if t.is_floating_point() and t.dim():
            seen.append((tuple(t.shape), checkpoint._is_statistic(t)))
        return t

    def saved(f):
        seen.clear()
        with torch.autograd.graph.saved_tensors_hooks(keep, lambda t: t):
            f()
        return set(seen)

    class Function(torch.autograd.Function):
        @staticmethod
        def forward(ctx, a):
            ctx.save_for_backward(a, a.exp()[:3])
            return a * 2

        @staticmethod
        def backward(ctx, g):
            raise AssertionError

    h = torch.randn(4, 8, requires_grad=True) * 1.0
    q = h.view(1, 2, 2, 8)
    assert saved(lambda: F.cross_entropy(h, torch.tensor([0, 1, 2, 3]))) == {((4, 8), True)}
    assert saved(lambda: h.logsumexp(1)) == {((4, 8), False), ((4,), True)}
    assert saved(lambda: F.softmax(h, 1)) == {((4, 8), False)}
    assert saved(lambda: Function.apply(h)) == {((4, 8), False), ((3, 8), True)}
    assert ((1, 2, 2), False) not in saved(lambda: F.scaled_dot_product_attention(q, q, q)) and ((1, 2, 2, 8), False) in set(seen)
    assert {s for s, stat in saved(lambda: F.layer_norm(h, (8,))) if not stat} == {(4, 8)}
    assert ((4, 1), True) in saved(lambda: h * h.square().mean(1, keepdim=True).rsqrt()) and ((4, 1), False) not in set(seen)
    assert saved(lambda: (lambda a, b: a * b)(*h.chunk(2, 1))) == {((4, 4), False)}
    assert saved(lambda: h * torch.ones(4, 8)) == {((4, 8), True)}          # a factor without a gradient


def test_parameters_and_their_views_are_known():
    w = torch.nn.Parameter(torch.zeros(4, 6))
    x = torch.zeros(4, 6)
    assert checkpoint._is_parameter(w) and checkpoint._is_parameter(w.t()) and checkpoint._is_parameter(w[1:].t())
    assert not checkpoint._is_parameter(x) and not checkpoint._is_parameter(w * 2) and not checkpoint._is_parameter((w * 2).t())


# ---- the oracle itself

def test_codes_match_torch():
    """Nearest e4m3 codes, ties to even, are torch's; powers of two scale exactly."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn(50, 96, generator=g) * torch.randn(50, 1, generator=g).mul(8).exp()
    x[:20] = x[:20].to(torch.bfloat16).float()            # ties
    codes, scale = L.pack8(x.numpy())
    up = torch.from_numpy(np.repeat(np.exp2(127.0 - scale), 32, axis=1)).float()
    want = (x * up).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(codes, want)
    back = L.unpack8(codes, scale)
    most = np.repeat(np.abs(x.numpy()).reshape(50, 3, 32).max(2), 32, axis=1)
    assert (np.abs(back - x.numpy()) <= np.maximum(2.0 ** -4 * np.abs(x.numpy()), 2.0 ** -17 * most)).all()


def test_codes_at_the_edges():
    x = np.zeros((1, 70), np.float32)
    x[0, :8] = [1.0, -0.0, np.inf, -np.inf, np.nan, 1.9999999, -2.0 ** -17, 2.0 ** -18]
    x[0, 32], x[0, 64] = 1e-45, 3.4e38
    codes, scale = L.pack8(x)
    assert scale.tolist() == [[120, 1, 247]]
    assert codes[0, :8].tolist() == [0x70, 0x80, 127, 127, 127, 0x78, 0x80, 0]      # 2^-10 of the scaled: half a code, to even
    assert codes[0, 32] == 0 and L.unpack8(codes, scale)[0, 64] == 2.0 ** 128


@pytest.mark.parametrize("most", [-100, -118, -119, -120, -125, -137, -149])
def test_bound_of_small_blocks(most):
    """2^-4 of the element, 2^-17 of the block's largest, or 2^-136: half of the smallest code, 2^-9, under the smallest scale."""
    x = L.small_blocks(most)
    codes, scale = L.pack8(x)
    off = np.abs(L.unpack8(codes, scale) - x)
    assert (off <= np.maximum(2.0 ** -4 * np.abs(x), max(2.0 ** (most - 17), 2.0 ** -136))).all()
    if most <= -137:
        assert ((codes & 127) == 0).all()


def test_kernels_wait_for_their_predecessor_before_they_touch_memory():
    """In every kernel that may be launched early, the wait for the grid before it stands before all that reads or writes
    global memory.  One may put it off: the weights' gradients in fp32 read nothing of the input's gradient, the launch
    before theirs, which began after the grids before it; they wait at their end, for the kernels behind them."""
    kernels = 0
    for name in ("k_embed.cu", "k_saved8.cu", "k_ffn.cu", "k_ffn_few.cu", "k_ffn_tc.cu", "k_ffn_lines.cu"):
        with open(os.path.join(os.path.dirname(B.__file__), "csrc", name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"__global__\b[^{;]*?\b(k_\w+)\s*\([^{]*\{", text):
            at, depth = m.end(), 1
            while depth:
                depth += {"{": 1, "}": -1}.get(text[at], 0)
                at += 1
            body = text[m.end(): at]
            wait = re.search(r"(?:^|[;{}])\s*grid_dependency_wait\(\);", body)
            if m.group(1) == "k_ffn_simt":
                wait = re.search(r"[;{}]\s*if \(!kWeight \|\| !p\.beside\) grid_dependency_wait\(\);", body)
                end = re.search(r"[;{}]\s*if \(kWeight && p\.beside\) grid_dependency_wait\(\);\s*\}$", body)
                assert end and re.findall(r"\breturn\b[^;]*;", body) == ["return;"]
                assert re.search(r"if constexpr \(kWeight\) \{[^}]*(?:\}[^}]*)?\} else \{.*find_tile.*\}\s*if \(!tile\) return;", body, re.S)
            assert wait, m.group(1)
            before = body[: wait.start() + 1]
            assert not re.search(r"key_of\(|row_of\(|clears_rows|ffn_clear_rows|ffn_expert|find_tile|find_chunk|fill_table|run_producer|run_mma|run_epilogue|load\(|store\(|\bp\.(ids|key|at|hist|key_in|at_in|part|table|out|x|codes|scales|dout|dtable)\b",
                                 before), m.group(1)
            kernels += 1
    assert kernels >= 13
    with open(os.path.join(os.path.dirname(B.__file__), "csrc", "ffn_api.cpp")) as f:
        text = f.read()
    assert re.findall(r"\bbeside = ([^;]*);", text) == ["c.dx != nullptr"]
    assert re.search(r"if \(c\.dx\) pass\.product\(\{FfnProduct::kInput[^;]*;\s*pass\.weights\(", text)


def test_no_grid_starts_early_and_reads_without_a_wait():
    """What an earlier grid wrote is visible to a grid that has waited for it, or that began when it was complete.  The weights'
    gradients in fp32 do not wait where they follow the input's: they are then one grid with it, which waits first, or a grid
    that is not launched early."""
    with open(os.path.join(os.path.dirname(B.__file__), "csrc", "k_ffn.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    one = text[text.index("k_ffn_grads(const"):]
    assert re.match(r"[^{]*\{\s*using S[^;]*;\s*extern __shared__ float4 smem\[\];\s*grid_dependency_wait\(\);", one)
    launch = text[text.index("int launch_tiles("): text.index("bool large_tiles(")]
    assert re.search(r"if \(kWhat == FfnProduct::kWeight && p\.beside\) pdl = false;\s*return launch_clusters\(", launch)
    # k_ffn_simt is launched there alone
    assert text.count("k_ffn_simt<") == launch.count("k_ffn_simt<")


# ---- gated feed-forward block

def _shape(rows=10, hidden=64, ffn=96, experts=3, dtype=F32, activation=B.MUON_SILU, saved_bits=0):
    return B.muon_ffn_shape(rows, hidden, ffn, experts, dtype, activation, saved_bits)


GB = 1 << 30


def _stack(p, a, b):
    return B.muon_stack(p, (a * b, b, 1))


def _saved(bits, base=20 * GB):
    names = {0: (), 32: ("gate", "up", "act"), 16: ("gate", "up", "act", "gate_scales", "up_scales"),
             8: ("gate", "up", "gate_scales", "up_scales", "x_codes", "x_scales")}.get(bits, ())
    return B.muon_ffn_saved(**{n: base + i * GB for i, n in enumerate(names)}) if bits else None


def _ffn_forward(h, shape=None, off=GB, cnt=GB + MB, x=2 * GB, ldx=64, gate=None, up=None, down=None, y=6 * GB, ldy=64, saved="own",
                 ws=7 * GB, ws_bytes=GB, **kw):
    s = shape or _shape(**kw)
    gate = gate or _stack(3 * GB, 96, 64)
    up = up or _stack(4 * GB, 96, 64)
    down = down or _stack(5 * GB, 64, 96)
    return B.muon_ffn_forward(h, s, off, cnt, x, ldx, gate, up, down, y, ldy, _saved(s.saved_bits) if saved == "own" else saved, ws, ws_bytes, 0)


def _ffn_backward(h, off=GB, cnt=GB + MB, dy=8 * GB, lddy=64, x="own", ldx=64, saved="own", dx=9 * GB, lddx=64, dgate="own", dup="own",
                  ddown="own", ws=7 * GB, ws_bytes=GB, **kw):
    s = _shape(**{**dict(saved_bits=32), **kw})
    x = (None if s.saved_bits == 8 else 2 * GB) if x == "own" else x
    own = lambda v, p, a, b: _stack(p, a, b) if v == "own" else v  # noqa: E731
    return B.muon_ffn_backward(h, s, off, cnt, dy, lddy, x, ldx, _stack(3 * GB, 96, 64), _stack(4 * GB, 96, 64), _stack(5 * GB, 64, 96),
                               _saved(s.saved_bits) if saved == "own" else saved, dx, lddx, own(dgate, 10 * GB, 96, 64),
                               own(dup, 11 * GB, 96, 64), own(ddown, 12 * GB, 64, 96), ws, ws_bytes, 0)


def test_ffn_struct_sizes():
    import ctypes
    assert ctypes.sizeof(B.muon_ffn_shape) == 3 * 8 + 4 * 4
    assert ctypes.sizeof(B.muon_stack) == 4 * 8
    assert ctypes.sizeof(B.muon_ffn_saved) == 7 * 8


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(rows=1 << 31), dict(hidden=-1), dict(hidden=(1 << 21) + 1), dict(ffn=(1 << 21) + 1),
                                 dict(experts=0), dict(experts=1025), dict(dtype=2), dict(activation=2), dict(saved_bits=16),
                                 dict(saved_bits=4), dict(dtype=BF16, saved_bits=32), dict(rows=(1 << 31) - 1, hidden=1 << 21)])
def test_ffn_shape_refusals(h, bad):
    assert B.muon_ffn_workspace_size(_shape(**bad), False)[0] == B.MUON_ERR_INVALID_ARG
    assert _ffn_forward(h, **bad) == B.MUON_ERR_INVALID_ARG and B.muon_last_error_message(h)


def test_ffn_workspace(h):
    for dtype, es in ((F32, 4), (BF16, 2)):
        for bits in (0, 8, 8 * es):
            s = _shape(rows=1000, ffn=200, dtype=dtype, saved_bits=bits)
            wide = 1000 * 256 * es
            assert B.muon_ffn_workspace_size(s, False) == (B.MUON_OK, 0 if bits == 8 * es else wide)
            back = B.muon_ffn_workspace_size(s, True)[1]
            assert back >= 2 * wide and back <= (3 if bits == 8 else 2) * wide + (1000 * 64 * es if bits == 8 else 0) + 3 * 5 * 128 + 256


def test_ffn_forward_refusals(h):
    for kw in (dict(), dict(dtype=BF16), dict(saved_bits=32), dict(saved_bits=8), dict(dtype=BF16, saved_bits=16), dict(ldx=72, ldy=65),
               dict(activation=B.MUON_GELU), dict(experts=1, off=None, cnt=None),
               # widths that are no multiples of 8 may begin anywhere
               dict(dtype=BF16, hidden=63, x=2 * GB + 2, ldx=67, y=6 * GB + 2, gate=B.muon_stack(3 * GB + 2, (96 * 65, 65, 1)),
                    up=_stack(4 * GB + 6, 96, 63), down=_stack(5 * GB, 63, 96)), dict(gate=B.muon_stack(3 * GB, (96 * 64, 1, 96))),
               dict(gate=B.muon_stack(3 * GB, (192 * 64, 64, 1)))):     # half of a stack of both
        assert _ffn_forward(h, **kw) == B.MUON_ERR_UNSUPPORTED, (kw, B.muon_last_error_message(h))
    assert _ffn_forward(h, rows=0, x=None, y=None, ws=None, ws_bytes=0) == B.MUON_OK
    for kw in (dict(off=None), dict(cnt=None), dict(off=None, cnt=None), dict(off=GB + 2), dict(x=None), dict(x=2 * GB + 2), dict(ldx=63), dict(y=None),
               dict(ldy=63), dict(y=2 * GB + 128), dict(y=GB + 4), dict(saved=_saved(32)), dict(saved_bits=32, saved=None),
               dict(saved_bits=8, saved=_saved(32)), dict(dtype=BF16, x=2 * GB + 2), dict(dtype=BF16, ldx=65),
               dict(gate=B.muon_stack(None, (96 * 64, 64, 1))), dict(gate=B.muon_stack(3 * GB, (96 * 64, 2, 2))),
               dict(gate=B.muon_stack(3 * GB, (96 * 64, 63, 1))), dict(gate=B.muon_stack(3 * GB, (96 * 64 - 1, 64, 1))),
               dict(gate=B.muon_stack(3 * GB, (64, 3 * 64, 1))),       # experts' rows between each other's
               dict(dtype=BF16, gate=B.muon_stack(3 * GB, (96 * 66, 66, 1))),
               dict(dtype=BF16, gate=B.muon_stack(3 * GB + 8, (96 * 64, 64, 1))),
               dict(dtype=BF16, gate=B.muon_stack(3 * GB, (96 * 64, 1, 96))),             # up runs the other way
               dict(saved_bits=32, saved=_saved(32, 2 * GB))):
        assert _ffn_forward(h, **kw) == B.MUON_ERR_INVALID_ARG, kw
        assert B.muon_last_error_message(h)
    for kw in (dict(ws=None), dict(ws=7 * GB + 16), dict(ws_bytes=100)):
        assert _ffn_forward(h, **kw) == B.MUON_ERR_WORKSPACE, kw


def test_ffn_backward_refusals(h):
    for kw in (dict(), dict(dtype=BF16, saved_bits=16), dict(saved_bits=8), dict(dx=None), dict(dgate=None, dup=None, ddown=None),
               dict(dgate=B.muon_stack(None, (0, 0, 0))), dict(rows=0, dy=None, x=None, dx=None)):
        assert _ffn_backward(h, **kw) == B.MUON_ERR_UNSUPPORTED, (kw, B.muon_last_error_message(h))
    assert _ffn_backward(h, dx=None, dgate=None, dup=None, ddown=None) == B.MUON_OK        # nothing is asked for
    for kw in (dict(saved_bits=0, saved=None), dict(saved=None), dict(x=None), dict(saved_bits=8, x=2 * GB), dict(dy=None), dict(lddy=63),
               dict(lddx=63), dict(dx=8 * GB), dict(dgate=B.muon_stack(10 * GB, (96 * 64, 1, 96))), dict(dgate=_stack(3 * GB, 96, 64)),
               dict(dup=_stack(10 * GB + 64, 96, 64)), dict(dtype=BF16, saved_bits=16, lddy=65)):
        assert _ffn_backward(h, **kw) == B.MUON_ERR_INVALID_ARG, kw
    for kw in (dict(ws=None), dict(ws=7 * GB + 16), dict(ws_bytes=100)):
        assert _ffn_backward(h, **kw) == B.MUON_ERR_WORKSPACE, kw


def test_ffn_status_refusals(h):
    assert B.muon_ffn_check_status(None, 0) == B.muon_ffn_share_status(None, 1) == B.MUON_ERR_INVALID_ARG
    assert B.muon_ffn_check_status(h, 0) == B.MUON_ERR_UNSUPPORTED
    assert B.muon_ffn_share_status(h, 1) == B.muon_ffn_share_status(h, 0) == B.MUON_OK
    for group in (-1, 16):
        assert B.muon_ffn_share_status(h, group) == B.MUON_ERR_INVALID_ARG and B.muon_last_error_message(h)


def test_ffn_torch_layer_refuses():
    from muon_newton_schulz_gb300 import ffn
    x, g, d = torch.zeros(5, 8), torch.zeros(16, 8), torch.zeros(8, 16)
    with pytest.raises(ValueError, match="CUDA"):
        ffn.gated_ffn(x, g, g, d)
    with pytest.raises(ValueError, match="rows x hidden"):
        ffn.gated_ffn(x[0], g, g, d)
    with pytest.raises(ValueError, match="activation"):
        ffn.gated_ffn(x, g, g, d, activation="relu")
    with pytest.raises(ValueError, match="saved_bits"):
        ffn.gated_ffn(x, g, g, d, saved_bits=16)
    calls = B.torch_calls()
    assert calls.ffn_forward(x, g, g, d, None, None, 0, 0, 0, 0) is None
    assert calls.ffn_backward(x, x, g, g, d, None, None, [], 0, 32, 15, 0, 0) is None
    assert calls.ffn_backward(x, x, g, g, d, None, None, [], 0, 7, 15, 0, 0) is None


def test_ffn_oracle_derivatives():
    g = np.linspace(-6, 6, 2001)
    for name in ("silu", "gelu"):
        a, s = L.act(g, name)
        step = 1e-5
        diff = (L.act(g + step, name)[0] - L.act(g - step, name)[0]) / (2 * step)
        assert np.abs(diff - s).max() < 1e-9
        want = (torch.nn.functional.silu if name == "silu" else torch.nn.functional.gelu)(torch.from_numpy(g)).numpy()
        assert np.abs(a - want).max() < 1e-14
        assert np.abs(s).max() < 1.13 and np.abs(np.gradient(s, g)).max() < 0.8
