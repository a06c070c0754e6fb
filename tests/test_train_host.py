"""AdamW, gradient clipping and tokens by expert without a GPU: the C ABI
validates on a host-only handle before anything could be launched, the torch
layer refuses what the library cannot take, and the oracle's 8-bit codes agree
with torch's float8 types."""
import ctypes
import os
import re
import sysconfig

import numpy as np
import pytest
import torch

import oracle.train_oracle as O
from muon_newton_schulz_gb300 import adamw, moe
from muon_newton_schulz_gb300 import binding as B


@pytest.fixture(scope="module")
def h():
    B.load_library(build_if_missing=True)
    st, handle = B.muon_create(None, -1)
    assert st == B.MUON_OK
    yield handle
    B.muon_destroy(handle)


BASE = 1 << 20
MB = 1 << 20


def _adam(**kw):
    d = B.muon_adamw_desc(1000, BASE, BASE + MB, BASE + 2 * MB, BASE + 3 * MB, None, B.MUON_F32, B.MUON_F32, 32, 0, 1,
                          0, 2e-4, 0.1)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def _adam_step(h, descs, cfg=None):
    arr = (B.muon_adamw_desc * max(1, len(descs)))(*descs)
    return B.muon_adamw_step(h, cfg, ctypes.addressof(arr), len(descs), 0)


def test_struct_sizes():
    assert ctypes.sizeof(B.muon_adamw_desc) == 8 * 6 + 4 * 4 + 8 * 4
    assert ctypes.sizeof(B.muon_adamw_config) == 24
    assert ctypes.sizeof(B.muon_clip_desc) == 8 * 6 + 4 * 2
    assert ctypes.sizeof(B.muon_moe_shape) == 8 + 4 * 4


def test_adamw_defaults():
    c = B.muon_adamw_config_default()
    assert (c.beta1, c.beta2, c.eps) == (0.9, 0.95, 1e-8)


def test_adamw_valid_reaches_the_device_check(h):
    assert _adam_step(h, [_adam()]) == B.MUON_ERR_UNSUPPORTED
    assert _adam_step(h, [_adam(state_bits=8, scales=BASE + 4 * MB)]) == B.MUON_ERR_UNSUPPORTED
    # addresses only need their element's alignment
    assert _adam_step(h, [_adam(P=BASE + 4, G=BASE + MB + 8)]) == B.MUON_ERR_UNSUPPORTED
    assert _adam_step(h, [_adam(state_bits=8, M=BASE + 2 * MB + 1, scales=BASE + 4 * MB)]) == B.MUON_ERR_UNSUPPORTED
    # one gradient may serve two parameters
    two = _adam(P=BASE + 5 * MB, M=BASE + 6 * MB, V=BASE + 7 * MB)
    assert _adam_step(h, [_adam(), two]) == B.MUON_ERR_UNSUPPORTED


def test_adamw_nothing_to_do(h):
    assert _adam_step(h, []) == B.MUON_OK
    assert _adam_step(h, [B.muon_adamw_desc()]) == B.MUON_OK
    assert B.muon_adamw_step(h, None, None, 1, 0) == B.MUON_ERR_INVALID_ARG
    assert B.muon_adamw_step(h, None, None, -1, 0) == B.MUON_ERR_INVALID_ARG
    assert B.muon_adamw_step(None, None, None, 0, 0) == B.MUON_ERR_INVALID_ARG


@pytest.mark.parametrize("bad, why", [
    (dict(n=-1), "2^40"),
    (dict(n=(1 << 40) + 1), "2^40"),
    (dict(P=None), "non-NULL"),
    (dict(G=None), "non-NULL"),
    (dict(M=None), "non-NULL"),
    (dict(V=None), "non-NULL"),
    (dict(P=BASE + 2), "P must be aligned"),
    (dict(G=BASE + MB + 1, g_dtype=B.MUON_BF16), "G must be aligned"),
    (dict(M=BASE + 2 * MB + 2), "M and V must be aligned"),
    (dict(p_dtype=2), "p_dtype"),
    (dict(g_dtype=-1), "g_dtype"),
    (dict(state_bits=16), "state_bits"),
    (dict(state_bits=8), "scales must be non-NULL"),
    (dict(state_bits=8, scales=BASE + 4 * MB + 1), "2-byte"),
    (dict(scales=BASE + 4 * MB), "NULL for 32-bit"),
    (dict(reserved=1), "reserved"),
    (dict(step=0), "step"),
    (dict(lr=float("nan")), "finite"),
    (dict(weight_decay=float("inf")), "finite"),
    (dict(M=BASE + 100), "overlap"),
    (dict(G=BASE + 3 * MB + 3996), "overlap"),
    (dict(state_bits=8, scales=BASE + 3 * MB + 998), "overlap"),
])
def test_adamw_refusals(h, bad, why):
    assert _adam_step(h, [_adam(**bad)]) == B.MUON_ERR_INVALID_ARG
    assert why in B.muon_last_error_message(h)


@pytest.mark.parametrize("cfg", [(1.0, 0.9, 0.0), (-0.1, 0.9, 0.0), (0.9, 1.0, 0.0), (0.9, 0.9, -1.0),
                                 (float("nan"), 0.9, 0.0), (0.9, 0.9, float("inf"))])
def test_adamw_config_refusals(h, cfg):
    assert _adam_step(h, [_adam()], B.muon_adamw_config(*cfg)) == B.MUON_ERR_INVALID_ARG


def test_overlap_is_found_behind_a_long_range(h):
    # G of desc 0 spans the P of desc 1, with other buffers starting between
    a = _adam(n=10 * MB, G=BASE + 256 * MB, P=BASE + 512 * MB, M=BASE + 1024 * MB, V=BASE + 2048 * MB)
    b = _adam(P=BASE + 256 * MB + 8 * MB, G=BASE + 256 * MB + 4 * MB, M=BASE + 4096 * MB, V=BASE + 4097 * MB)
    assert _adam_step(h, [a, b]) == B.MUON_ERR_INVALID_ARG
    assert "desc 0 G and desc 1 P" in B.muon_last_error_message(h)


def _clip(**kw):
    d = B.muon_clip_desc(100, 64, BASE, 64, BASE + MB, 64, B.MUON_F32, B.MUON_F32)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def _clip_call(h, descs, max_norm=1.0, norm=1 << 30, ws=1 << 31, ws_bytes=B.MUON_CLIP_WORKSPACE_BYTES):
    arr = (B.muon_clip_desc * max(1, len(descs)))(*descs)
    return B.muon_clip_grads(h, ctypes.addressof(arr), len(descs), max_norm, norm, ws, ws_bytes, 0)


def test_clip_valid_reaches_the_device_check(h):
    for d in (_clip(), _clip(out=None), _clip(out=BASE), _clip(ldg=65, ldo=70), _clip(out_dtype=B.MUON_BF16)):
        assert _clip_call(h, [d]) == B.MUON_ERR_UNSUPPORTED
    assert _clip_call(h, [_clip()], max_norm=float("inf")) == B.MUON_ERR_UNSUPPORTED


@pytest.mark.parametrize("bad, why", [
    (dict(rows=-1), "rows and cols"),
    (dict(cols=1 << 41), "2^40"),
    (dict(G=None), "non-NULL"),
    (dict(G=BASE + 2), "aligned"),
    (dict(g_dtype=5), "g_dtype"),
    (dict(out_dtype=5), "out_dtype"),
    (dict(ldg=63), "ldg and ldo"),
    (dict(ldo=63), "ldg and ldo"),
    (dict(out=BASE + 256), "overlap"),
])
def test_clip_refusals(h, bad, why):
    assert _clip_call(h, [_clip(**bad)]) == B.MUON_ERR_INVALID_ARG
    assert why in B.muon_last_error_message(h)


def test_column_ranges_of_one_buffer_do_not_overlap(h):
    one = _clip(cols=24, ldg=64, ldo=64)
    two = _clip(cols=40, ldg=64, ldo=64, G=BASE + 96, out=BASE + MB + 96)
    assert _clip_call(h, [one, two]) == B.MUON_ERR_UNSUPPORTED
    assert _clip_call(h, [two, one]) == B.MUON_ERR_UNSUPPORTED
    for bad in (dict(cols=25), dict(out=BASE + MB + 4), dict(ldo=65), dict(out=BASE + MB + 64 * 4 + 196)):
        a = _clip(**{**dict(cols=24, ldg=64, ldo=64), **bad})
        assert _clip_call(h, [a, two]) == B.MUON_ERR_INVALID_ARG, bad


def test_clip_call_refusals(h):
    for m in (0.0, -1.0, float("nan")):
        assert _clip_call(h, [_clip()], max_norm=m) == B.MUON_ERR_INVALID_ARG
    assert _clip_call(h, [_clip()], norm=None) == B.MUON_ERR_INVALID_ARG
    assert _clip_call(h, [_clip()], norm=BASE + 4) == B.MUON_ERR_INVALID_ARG      # inside G
    assert _clip_call(h, [_clip()], ws=None) == B.MUON_ERR_WORKSPACE
    assert _clip_call(h, [_clip()], ws=(1 << 31) + 8) == B.MUON_ERR_WORKSPACE
    assert _clip_call(h, [_clip()], ws_bytes=100) == B.MUON_ERR_WORKSPACE
    # the norm of one gradient held twice is fine; clipping it in place twice is not
    assert _clip_call(h, [_clip(out=None), _clip(out=None)]) == B.MUON_ERR_INVALID_ARG
    assert _clip_call(h, [_clip(out=None), _clip(out=None)], max_norm=float("inf")) == B.MUON_ERR_UNSUPPORTED


def _shape(tokens=10, topk=2, experts=4, capacity=0, align=1):
    return B.muon_moe_shape(tokens, topk, experts, capacity, align)


@pytest.mark.parametrize("kw, rows", [
    (dict(), 20), (dict(align=16), 80), (dict(capacity=7), 28), (dict(tokens=0), 0), (dict(tokens=0, align=8), 32),
    (dict(tokens=0, capacity=3), 12),
])
def test_moe_rows(h, kw, rows):
    assert B.muon_moe_rows(_shape(**kw)) == (B.MUON_OK, rows)


@pytest.mark.parametrize("kw", [dict(topk=0), dict(topk=65), dict(experts=0), dict(experts=1025), dict(tokens=-1),
                                dict(tokens=1 << 30, topk=2), dict(capacity=-1), dict(align=0),
                                dict(capacity=5, align=2), dict(capacity=1 << 30), dict(align=1 << 30)])
def test_moe_shape_refusals(h, kw):
    assert B.muon_moe_rows(_shape(**kw))[0] == B.MUON_ERR_INVALID_ARG
    assert B.muon_moe_sort_workspace_size(_shape(**kw))[0] == B.MUON_ERR_INVALID_ARG


def test_moe_sort_workspace(h):
    assert B.muon_moe_sort_workspace_size(_shape()) == (B.MUON_OK, 0)
    st, big = B.muon_moe_sort_workspace_size(_shape(tokens=100000, experts=128))
    assert st == B.MUON_OK and 0 < big <= 152 * 128 * 4
    s = _shape(tokens=100000, experts=128)
    args = (BASE, 64, 1 << 30, 2 << 30, 3 << 30)
    assert B.muon_moe_sort(h, s, *args, None, 0, 0) == B.MUON_ERR_WORKSPACE
    assert B.muon_moe_sort(h, s, *args, 4 << 30, big - 1, 0) == B.MUON_ERR_WORKSPACE
    assert B.muon_moe_sort(h, s, *args, (4 << 30) + 64, big, 0) == B.MUON_ERR_WORKSPACE
    assert B.muon_moe_sort(h, s, *args, 4 << 30, big, 0) == B.MUON_ERR_UNSUPPORTED


def test_moe_sort_refusals(h):
    s = _shape()
    ok = [BASE, 64, 1 << 30, 2 << 30, 3 << 30, None, 0, 0]
    assert B.muon_moe_sort(h, s, *ok) == B.MUON_ERR_UNSUPPORTED
    for at, value in ((0, None), (0, BASE + 4), (1, 16), (2, None), (3, None), (4, None), (2, (1 << 30) + 2),
                      (3, (1 << 30) + 8)):
        bad = list(ok)
        bad[at] = value
        assert B.muon_moe_sort(h, s, *bad) == B.MUON_ERR_INVALID_ARG, (at, value)


def test_moe_row_operator_refusals(h):
    s = _shape()                       # 10 tokens, 20 rows
    row, off, cnt = 1 << 30, (1 << 30) + MB, (1 << 30) + 2 * MB
    x, xs = 1 << 31, (1 << 31) + MB
    f32, bf16 = B.MUON_F32, B.MUON_BF16

    def disp(row=row, off=off, cnt=cnt, x=x, ldx=64, xs=xs, ldxs=64, hidden=64, dtype=f32):
        return B.muon_moe_dispatch(h, s, row, off, cnt, x, ldx, xs, ldxs, hidden, dtype, 0)

    assert disp() == disp(dtype=bf16, x=x + 2) == disp(ldx=65) == B.MUON_ERR_UNSUPPORTED
    assert disp(hidden=0) == B.MUON_OK
    for kw in (dict(row=None), dict(off=None), dict(cnt=None), dict(x=None), dict(xs=None), dict(ldx=63),
               dict(ldxs=63), dict(hidden=-1), dict(dtype=3), dict(x=x + 2), dict(xs=x + 64), dict(row=row + 1),
               dict(off=xs + 4)):
        assert disp(**kw) == B.MUON_ERR_INVALID_ARG, kw
        assert B.muon_last_error_message(h)

    w, dw = (1 << 30) + 3 * MB, (1 << 30) + 4 * MB

    def comb(row=row, y=xs, ldy=64, w=w, wd=f32, out=x, ldo=64, hidden=64, dtype=f32):
        return B.muon_moe_combine(h, s, row, y, ldy, w, wd, out, ldo, hidden, dtype, 0)

    assert comb() == comb(w=None) == comb(wd=bf16, w=w + 2) == B.MUON_ERR_UNSUPPORTED
    for kw in (dict(row=None), dict(y=None), dict(out=None), dict(ldy=63), dict(ldo=63), dict(wd=4), dict(w=w + 2),
               dict(out=xs + 256), dict(out=w, hidden=1), dict(dtype=9)):
        assert comb(**kw) == B.MUON_ERR_INVALID_ARG, kw

    def back(row=row, off=off, cnt=cnt, dout=x, ldd=64, y=xs, ldy=64, w=w, wd=f32, dy=xs + MB, lddy=64, dw=dw,
             hidden=64, dtype=f32):
        return B.muon_moe_combine_backward(h, s, row, off, cnt, dout, ldd, y, ldy, w, wd, dy, lddy, dw, hidden, dtype, 0)

    assert back() == B.MUON_ERR_UNSUPPORTED
    for kw in (dict(w=None), dict(dw=None), dict(dw=w), dict(dw=dw + 2), dict(dout=None), dict(y=None), dict(dy=None),
               dict(dy=xs), dict(lddy=1), dict(off=None), dict(wd=-1), dict(hidden=-3)):
        assert back(**kw) == B.MUON_ERR_INVALID_ARG, kw


def test_torch_layer_refuses_cpu_tensors():
    t = torch.zeros(8)
    with pytest.raises(ValueError, match="CUDA"):
        adamw.adamw_step([t], [t], [t], [t], lr=1e-3, step=1)
    with pytest.raises(ValueError, match="CUDA"):
        adamw.clip_grads([t], 1.0)
    with pytest.raises(ValueError, match="CUDA"):
        moe.sort_tokens(torch.zeros(3, 2, dtype=torch.int64), 4)
    i = torch.zeros(3, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        moe.Route(i, torch.zeros(5, dtype=torch.int32), torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="same length"):
        adamw.adamw_step([t], [t], [t], [], lr=1e-3, step=1)
    for kw in (dict(lr=[1e-3, 1e-3]), dict(lr=1e-3, weight_decay=[]), dict(lr=1e-3, step=[1, 2]), dict(lr=1e-3, seed=[])):
        with pytest.raises(ValueError, match="entry for each"):
            adamw.adamw_step([t], [t], [t], [t], **{"step": 1, **kw})
    with pytest.raises(ValueError, match="topk"):
        moe.sort_tokens(torch.zeros(3, dtype=torch.int64), 4)
    with pytest.raises(ValueError, match="int32 or int64"):
        moe.sort_tokens(torch.zeros(3, 2), 4)


def test_built_module_takes_only_lists_of_tensors():
    calls = B.torch_calls()
    t = torch.zeros(4)
    assert calls.clip([t], [t], 0, 1.0, 0, 0) is None            # not on the device: refused before any call
    assert calls.adamw([t], [t], [t], [t], None, 0, 1e-3, 0.0, 1, 0, 0.9, 0.95, 1e-8, 0, 0) is None
    assert calls.adamw([3], [t], [t], [t], None, 0, 1e-3, 0.0, 1, 0, 0.9, 0.95, 1e-8, 0, 0) is None
    with pytest.raises(TypeError):
        calls.clip(3, [t], 0, 1.0, 0, 0)


def test_is_dense():
    t = torch.zeros(4, 6, 5)
    assert adamw.is_dense(t) and adamw.is_dense(t.permute(2, 0, 1)) and adamw.is_dense(t[1])
    assert adamw.is_dense(torch.zeros(1, 5).expand(1, 5)) and adamw.is_dense(torch.zeros(()))
    assert not adamw.is_dense(t[:, :3]) and not adamw.is_dense(torch.zeros(1, 5).expand(3, 5))


# ---- the oracle itself

def test_code_tables_match_torch():
    codes = torch.arange(256, dtype=torch.int16).to(torch.uint8)
    for kind, table in ((torch.float8_e4m3fn, O.E4M3), (torch.float8_e5m2, O.E5M2)):
        want = codes.view(kind).float().numpy().astype(np.float64)
        got = O.decode8(codes.numpy(), table)
        fine = ~np.isnan(got)
        np.testing.assert_array_equal(got[fine], want[fine])
        assert not np.isfinite(want[~fine]).any()


def test_rounding_is_unbiased_and_stays_on_the_grid():
    """Every 16-bit random number once: the mean of the stored value is the value, to 2^-16 of a code step."""
    n = 1 << 16
    for value, store, table in ((1.3, O.store8_m, O.E4M3), (0.77e-3, O.store8_v, O.E5M2), (5e-9, O.store8_m, O.E4M3)):
        x = np.full(n, value, np.float32)
        # 255 values under one block maximum of 1.9 each, so that small values land among the small codes
        x[::256] = 1.9
        r = np.arange(n, dtype=np.uint32)
        codes, scale = store(x, r)
        got = O.decode8(codes, table) * O.per_element(scale, n)
        part = np.arange(n) % 256 != 0
        kinds = np.unique(got[part])
        assert len(kinds) <= 2
        step = kinds[-1] - kinds[0] if len(kinds) == 2 else 0.0
        assert abs(got[part].mean() - np.float64(np.float32(value))) <= step * 2 ** -7 + 1e-12
    z, _ = O.store8_v(np.array([1.0] + [1e-30] * 255, np.float32), np.zeros(256, np.uint32))
    assert (z > 0).all()


def test_random_numbers_are_uniform_and_uncorrelated():
    """Means, variances and neighbour correlations of 2^20 draws, within 5 standard errors; and two steps, two
    seeds and the two halves are uncorrelated."""
    n = 1 << 20
    rows = [x.astype(np.float64) / 65536 for s, t in ((1, 1), (1, 2), (2, 1), (0, 1)) for x in O.random16(n, s, t)]
    se = 1 / np.sqrt(n)
    for a in rows:
        assert abs(a.mean() - 0.5) < 5 * se * 0.2887
        assert abs(a.var() - 1 / 12) < 5 * se * 0.0745
        for lag in (1, 2, 8, 32, 256, 257):
            assert abs(np.corrcoef(a[:-lag], a[lag:])[0, 1]) < 5 * se
        counts = np.bincount((a * 256).astype(int), minlength=256)
        chi = ((counts - n / 256) ** 2 / (n / 256)).sum()
        assert abs(chi - 255) < 6 * np.sqrt(2 * 255)
    for i in range(len(rows)):
        for j in range(i):
            assert abs(np.corrcoef(rows[i], rows[j])[0, 1]) < 5 * se


def test_calls_are_not_traced():
    from torch.fx.experimental.proxy_tensor import make_fx

    def f(x):
        assert B.torch_calls().adamw([], [], [], [], None, 0, 1e-3, 0.0, 1, 0, 0.9, 0.95, 1e-8, 0, 0) != B.MUON_OK    # no handle
        return x + 1

    x = torch.zeros(3)
    f(x)
    with pytest.raises(RuntimeError, match="cannot be traced"):
        make_fx(f)(x)
    with pytest.raises(RuntimeError, match="cannot be traced"):
        torch.jit.trace(f, (x,), check_trace=False)
    f(x)


def test_clip_grad_norm_takes_a_tensor_and_gives_its_device():
    from muon_newton_schulz_gb300.optim import clip_grad_norm
    p = torch.nn.Parameter(torch.ones(3, 4))
    p.grad = torch.ones(3, 4)
    with pytest.raises(ValueError, match="CUDA"):       # its gradient is looked at, and not those of its rows
        clip_grad_norm(p, 1.0)
    q = torch.nn.Parameter(torch.zeros(3, device="meta"))
    for x in (q, [q], iter([q])):
        norm = clip_grad_norm(x, 1.0)
        assert norm.device.type == "meta" and norm.shape == () and norm.dtype == torch.float32
    assert float(clip_grad_norm([], 1.0)) == 0.0


def test_kernels_wait_for_their_predecessor_before_they_touch_memory():
    """What a kernel may see of the grid before it is promised only behind its own wait: in every kernel that may be launched
    early, that wait is a statement of its own and stands before all that reads or writes global memory."""
    kernels = 0
    for name in ("k_adamw.cu", "k_moe.cu"):
        with open(os.path.join(os.path.dirname(B.__file__), "csrc", name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"__global__\b[^{;]*?\b(k_\w+)\s*\([^{]*\{", text):
            at, depth = m.end(), 1
            while depth:
                depth += {"{": 1, "}": -1}.get(text[at], 0)
                at += 1
            body = text[m.end(): at]
            wait = re.search(r"(?:^|[;{}])\s*grid_dependency_wait\(\);", body)
            assert wait, m.group(1)
            before = body[: wait.start() + 1]
            assert not re.search(r"expert_of\(|stage\(|clear_rows|sum_squares|_blocks|adamw8_any|adamw32_body|load\d?\(|store\d?\(|"
                                 r"\bp\.(ids|row|offsets|counts|hist|w|x|y|out|dw|partial|norm)\b", before), m.group(1)
            kernels += 1
    assert kernels >= 9


def test_the_built_module_is_named_after_what_it_was_built_for():
    """One built for another Python or torch is not found, and not loaded."""
    from muon_newton_schulz_gb300 import build
    assert sysconfig.get_config_var("SOABI") in build.CALLS_NAME and torch.__version__ in build.CALLS_NAME
    assert B.torch_calls().__file__ == build.CALLS


def _with_gil_check(f):
    """What f returns while the library's functions are replaced by one whose status says whether the caller holds
    Python's lock."""
    calls = B.torch_calls()
    check = ctypes.cast(ctypes.pythonapi.PyGILState_Check, ctypes.c_void_p).value
    calls.bind(*[check] * 6)
    try:
        return f(calls)
    finally:
        B._calls = None
        B.torch_calls()          # binds the library again


def test_other_threads_run_while_the_library_is_called():
    assert _with_gil_check(lambda c: c.adamw([], [], [], [], None, 0, 1e-3, 0.0, 1, 0, 0.9, 0.95, 1e-8, 0, 0)) == 0


def test_moe_sizes_that_32_bits_do_not_hold_are_refused():
    assert moe._sizes(10, 2, 4, 0, 1)[1] == 20
    for bad in (dict(capacity=1 << 32), dict(capacity=(1 << 32) + 5), dict(experts=(1 << 32) + 4), dict(align=(1 << 32) + 1),
                dict(topk=(1 << 32) + 2), dict(tokens=1 << 64), dict(experts=-(1 << 32) + 4)):
        with pytest.raises(ValueError, match=next(iter(bad))):
            moe._sizes(**{**dict(tokens=10, topk=2, experts=4, capacity=0, align=1), **bad})
    for bad in (4.0, "4", None):
        with pytest.raises(TypeError):
            moe._sizes(10, 2, bad, 0, 1)
    assert moe._sizes(10, 2, np.int64(4), np.int32(7), 1)[1] == 28


def test_a_vector_between_the_rows_of_a_matrix_does_not_overlap(h):
    matrix = _clip(cols=24, ldg=64, out=None)
    row = dict(rows=1, ldg=40, out=None)
    for at, cols in ((24, 40), (5 * 64 + 24, 40), (5 * 64 + 30, 3), (98 * 64 + 24, 40), (99 * 64 + 24, 1000)):
        assert _clip_call(h, [matrix, _clip(**row, cols=cols, G=BASE + 4 * at)]) == B.MUON_ERR_UNSUPPORTED, at
    for at, cols in ((23, 2), (24, 41), (5 * 64 + 24, 41), (6 * 64, 1), (98 * 64 + 24, 41), (99 * 64 + 23, 1), (30, 70)):
        assert _clip_call(h, [matrix, _clip(**row, cols=cols, G=BASE + 4 * at)]) == B.MUON_ERR_INVALID_ARG, at
    assert _clip_call(h, [matrix, _clip(**row, cols=40, G=BASE - 8)]) == B.MUON_ERR_INVALID_ARG
