"""Cases of the training-step operators around the Muon step, their plain forms and their definition in 64 bits.

Operators: an AdamW step over many tensors with states in 32 or in 8 bits, gradient clipping by the global norm, and tokens
sorted by expert (dispatch), put back with their weights (combine), and both gradients (backward).
"""
import math

import torch

own = False

LR, BETA1, BETA2, EPS, DECAY = 2e-4, 0.9, 0.95, 1e-8, 0.1
BLOCK = 256  # elements of an 8-bit state that share a scale
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "int64": torch.int64, "int32": torch.int32}
BYTES = {"f32": 4, "bf16": 2, "none": 0, "int64": 8, "int32": 4}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the norm gains of a 24-layer model: 49 short vectors, where a step is all latency
        dict(name="adamw32_gains", op="adamw", bits=32, mats=0, rows=0, cols=2048, gains=49, p="f32", g="f32", packed=False),
        # embedding and output head of a bf16 model with its norm gains: bandwidth
        dict(name="adamw32_embeddings", op="adamw", bits=32, mats=2, rows=32768, cols=2048, gains=49, p="bf16", g="bf16", packed=False),
        # a router, gains and biases of odd sizes packed one after another, so that few begin on a 16-byte boundary
        dict(name="adamw8_packed_odd", op="adamw", bits=8, mats=1, rows=1001, cols=1003, gains=7, p="f32", g="f32", packed=True),
        # a large embedding and head with their states in 8 bits
        dict(name="adamw8_embeddings", op="adamw", bits=8, mats=2, rows=65536, cols=2048, gains=49, p="bf16", g="bf16", packed=False),
        # the gradients of the gains alone
        dict(name="clip_gains", op="clip", mats=0, rows=0, cols=2048, gains=49, g="f32", out="f32", packed=False),
        # the bf16 gradients of a layer's experts, clipped into the fp32 buffers that the Muon step reads
        dict(name="clip_experts", op="clip", mats=16, rows=2048, cols=8192, gains=0, g="bf16", out="f32", packed=False),
        # one token of a served model
        dict(name="dispatch_one_token", op="dispatch", tokens=1, topk=2, experts=16, hidden=2048, type="bf16", ids="int64", masked=0.0, capacity=0, align=1),
        # a training batch over 128 experts
        dict(name="dispatch_batch", op="dispatch", tokens=16384, topk=8, experts=128, hidden=2048, type="bf16", ids="int64", masked=0.0, capacity=0, align=1),
        # a few tokens of a served model of hidden size 6144
        dict(name="combine_few_tokens", op="combine", tokens=5, topk=8, experts=128, hidden=6144, type="bf16", weights="f32", masked=0.0, capacity=0, align=1),
        # a training batch, top 2 of 16
        dict(name="combine_batch", op="combine", tokens=16384, topk=2, experts=16, hidden=6144, type="bf16", weights="f32", masked=0.0, capacity=0, align=1),
        # odd sizes with padding tokens and experts that run over their capacity, in fp32
        dict(name="backward_ragged", op="backward", tokens=1003, topk=2, experts=16, hidden=1001, type="f32", weights="f32", masked=0.1, capacity=157, align=1),
        # the gradients of a training batch over 128 experts
        dict(name="backward_batch", op="backward", tokens=16384, topk=8, experts=128, hidden=2048, type="bf16", weights="f32", masked=0.0, capacity=0, align=1),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["adamw", "adamw", "clip", "dispatch", "combine", "backward"])
    if op in ("adamw", "clip"):
        cols = _spread(rng, 16, 8192)
        mats = rng.choice([0, 1, 1, 2, 3, 16])
        rows = _spread(rng, 1, max(1, min(65536, (1 << 27) // (cols * max(mats, 1)))))
        case = dict(op=op, mats=mats, rows=rows if mats else 0, cols=cols, gains=_spread(rng, 1, 200), g=rng.choice(["f32", "bf16"]), packed=rng.random() < 0.4)
        if op == "adamw":
            return dict(case, bits=rng.choice([32, 8]), p=rng.choice([case["g"], "bf16", "f32"]))
        return dict(case, out=rng.choice([case["g"], "f32"]))
    experts = _spread(rng, 4, 256)
    topk = rng.choice([k for k in (1, 2, 3, 4, 6, 8) if k <= experts])
    hidden = rng.choice([_spread(rng, 64, 8192), 8 * _spread(rng, 16, 1024), 2048, 6144])
    tokens = _spread(rng, 1, max(1, min(65536, (1 << 27) // (hidden * topk))))
    capacity = rng.choice([0, 0, max(1, int(1.25 * tokens * topk / experts))])
    case = dict(op=op, tokens=tokens, topk=topk, experts=experts, hidden=hidden, type=rng.choice(["bf16", "bf16", "f32"]),
                masked=rng.choice([0.0, 0.0, 0.15]), capacity=capacity, align=1 if capacity else rng.choice([1, 1, 16, 128]))
    if op == "dispatch":
        return dict(case, ids=rng.choice(["int64", "int32"]))
    return dict(case, weights=rng.choice(["f32", "f32", "bf16"] + (["none"] if op == "combine" else [])))


# ---------------------------------------------------------------- what a program has in hand

def _sizes(case):
    return [case["rows"] * case["cols"]] * case["mats"] + [case["cols"]] * case["gains"]


def _starts(case, sizes, unit):
    """Where each tensor begins in a flat buffer, and the buffer's length."""
    at, n = [], 0
    for s in sizes:
        at.append(n)
        n += s if case["packed"] else -(-s // unit) * unit
    return at, n


def _rows_of(case):
    """Rows of the buffer that holds the sorted tokens."""
    if case["capacity"]:
        return case["experts"] * case["capacity"]
    a = case["align"]
    return -(-(case["tokens"] * case["topk"] + case["experts"] * (a - 1)) // a) * a


def _grads(flat, case, gen):
    """Gradients of a mid-training step: small, of very different size from column to column, and zero for a part of the rows
    (the words that a batch does not hold)."""
    n = flat.numel()
    col = torch.rand(997, generator=gen, device="cuda").mul_(6).exp_()
    flat.copy_(torch.randn(n, generator=gen, device="cuda").mul_(1e-5 if case["mats"] else 1e-3))
    flat.mul_(col.repeat(-(-n // 997))[:n])
    if case["mats"] and case["rows"] > 1:
        w = case["cols"]
        m = n // w
        flat[: m * w].view(m, w).mul_((torch.rand(m, 1, generator=gen, device="cuda") > 0.4).to(flat.dtype))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case, "seed": seed}
    if case["op"] in ("adamw", "clip"):
        sizes = _sizes(case)
        at, n = _starts(case, sizes, 128)
        view = lambda flat: [flat[a: a + k] for a, k in zip(at, sizes)]  # noqa: E731
        s["flat_g"] = torch.empty(n, device="cuda", dtype=TYPES[case["g"]])
        _grads(s["flat_g"], case, gen)
        s["g"] = view(s["flat_g"])
        if case["op"] == "clip":
            s["flat_out"] = torch.zeros(n, device="cuda", dtype=TYPES[case["out"]])
            s["out"] = view(s["flat_out"])
            s["max_norm"] = 0.5
            return s
        s["flat_p"] = torch.randn(n, generator=gen, device="cuda").mul_(0.02).to(TYPES[case["p"]])
        s["p"] = view(s["flat_p"])
        m = s["flat_g"].float() * torch.randn(n, generator=gen, device="cuda").mul_(0.3)
        v = s["flat_g"].float().square() * torch.rand(n, generator=gen, device="cuda").mul_(0.5).add_(0.1)
        m[n // 2:] += 1e-6 * torch.randn(n - n // 2, generator=gen, device="cuda")
        v[n // 2:] += 1e-12
        if case["bits"] == 32:
            s["flat_m"], s["flat_v"] = m, v
            s["m"], s["v"], s["scales"] = view(m), view(v), None
        else:
            s["flat_m"] = torch.zeros(n, device="cuda", dtype=torch.float8_e4m3fn)
            s["flat_v"] = torch.zeros(n, device="cuda", dtype=torch.float8_e5m2)
            blocks = [-(-k // BLOCK) for k in sizes]
            s["flat_scales"] = torch.zeros(sum(blocks), 2, device="cuda", dtype=torch.uint8).view(torch.float8_e8m0fnu)
            s["m"], s["v"] = view(s["flat_m"]), view(s["flat_v"])
            s["scales"] = list(s["flat_scales"].split(blocks))
            for i, (x, y) in enumerate(zip(view(m), view(v))):
                _store8(x, y, s["m"][i], s["v"][i], s["scales"][i], seed + i, 0)
        s["step"] = 100
        return s
    T, K, E, H, R = case["tokens"], case["topk"], case["experts"], case["hidden"], _rows_of(case)
    logits = torch.randn(T, E, generator=gen, device="cuda") + torch.randn(E, generator=gen, device="cuda")
    top = logits.topk(K, dim=1)
    ids = top.indices
    if case["masked"]:  # tokens of padding go to no expert
        ids = torch.where(torch.rand(T, 1, generator=gen, device="cuda") < case["masked"], -1, ids)
    kind = TYPES[case["type"]]
    rand = lambda *shape: torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).to(kind)  # noqa: E731
    if case["op"] == "dispatch":
        s["ids"] = ids.to(TYPES[case["ids"]]).contiguous()
        s["x"] = rand(T, H)
        return s
    s["row"], s["offsets"], s["counts"] = _sort(ids, case)
    s["y"] = rand(R, H)
    s["w"] = None if case["weights"] == "none" else torch.softmax(top.values, 1).to(TYPES[case["weights"]])
    if case["op"] == "backward":
        s["dout"], s["dxs"] = rand(T, H), rand(R, H)
    return s


# ---------------------------------------------------------------- the operators

def run(s):
    return (_run_own if own else _run_plain)(s, s["case"])


def _run_own(s, case):
    from muon_newton_schulz_gb300 import adamw, moe

    if case["op"] == "adamw":
        s["step"] += 1
        adamw.adamw_step(s["p"], s["g"], s["m"], s["v"], s["scales"], lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY, step=s["step"], seed=s["seed"])
        return _adamw_outputs(s)
    if case["op"] == "clip":
        norm = adamw.clip_grads(s["g"], s["max_norm"], outs=s["out"])
        return {"norm": norm, "out": s["flat_out"]}
    if case["op"] == "dispatch":
        route = moe.sort_tokens(s["ids"], case["experts"], capacity=case["capacity"], align=case["align"])
        return {"row": route.row, "offsets": route.offsets, "counts": route.counts, "xs": moe.dispatch(s["x"], route)}
    route = moe.Route(s["row"], s["offsets"], s["counts"], capacity=case["capacity"], align=case["align"])
    if case["op"] == "combine":
        return {"out": moe.combine(s["y"], s["w"], route)}
    dy, dw = moe.combine_backward(s["dout"], s["y"], s["w"], route)
    return {"dy": dy, "dw": dw, "dx": moe.dispatch_backward(s["dxs"], route)}


def _run_plain(s, case):
    if case["op"] == "adamw":
        s["step"] += 1
        for i, (p, g, m, v) in enumerate(zip(s["p"], s["g"], s["m"], s["v"])):
            _adamw_plain(p, g, m, v, s["scales"][i] if s["scales"] else None, s["step"], s["seed"] + i)
        return _adamw_outputs(s)
    if case["op"] == "clip":
        norm = torch.stack([g.float().square().sum() for g in s["g"]]).sum().sqrt()
        scale = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
        for g, out in zip(s["g"], s["out"]):
            out.copy_(g.float() * scale)
        return {"norm": norm, "out": s["flat_out"]}
    if case["op"] == "dispatch":
        row, offsets, counts = _sort(s["ids"], case)
        return {"row": row, "offsets": offsets, "counts": counts, "xs": _scatter(s["x"].repeat_interleave(case["topk"], 0), row, _rows_of(case))}
    w = s["w"].float() if s["w"] is not None else torch.ones_like(s["row"], dtype=torch.float32)
    if case["op"] == "combine":
        return {"out": (_gather(s["y"], s["row"]).mul_(w.unsqueeze(2))).sum(1).to(s["y"].dtype)}
    dout = s["dout"].float().unsqueeze(1)
    dw = (_gather(s["y"], s["row"]).mul_(dout)).sum(2).to(s["w"].dtype)
    dy = _scatter((w.unsqueeze(2) * dout).flatten(0, 1).to(s["y"].dtype), s["row"], s["y"].shape[0])
    return {"dy": dy, "dw": dw, "dx": _gather(s["dxs"], s["row"]).sum(1).to(s["dxs"].dtype)}


def _adamw_outputs(s):
    out = {"p": s["flat_p"], "m": s["flat_m"], "v": s["flat_v"]}
    if s["scales"] is not None:
        out["scales"] = s["flat_scales"]
    return out


# ---------------------------------------------------------------- AdamW in its plain form

def _adamw_plain(p, g, m, v, scales, step, seed):
    g = g.float()
    if scales is None:
        m0, v0 = m, v
    else:
        m0, v0 = _load8(m, v, scales)
    m1 = BETA1 * m0 + (1 - BETA1) * g
    v1 = BETA2 * v0 + (1 - BETA2) * (g * g)
    denom = v1.sqrt() / math.sqrt(1 - BETA2 ** step) + EPS
    p.copy_(p.float() * (1 - LR * DECAY) - (LR / (1 - BETA1 ** step)) * (m1 / denom))
    if scales is None:
        m.copy_(m1)
        v.copy_(v1)
    else:
        _store8(m1, v1, m, v, scales, seed, step)


def _per_element(scales, n):
    return scales.float().repeat_interleave(BLOCK, 0)[:n]


def _load8(m, v, scales):
    each = _per_element(scales, m.numel())
    return m.float() * each[:, 0], v.float() * each[:, 1]


def _mix64(x):
    """A 64-bit mix of a whole number (SplitMix: Steele, Lea and Flood, 2014)."""
    x = (x + 0x9E3779B97F4A7C15) % 2 ** 64
    x = (x ^ (x >> 30)) * 0xBF58476D1CE4E5B9 % 2 ** 64
    x = (x ^ (x >> 27)) * 0x94D049BB133111EB % 2 ** 64
    return x ^ (x >> 31)


def _mix32(x):
    x = ((x ^ (x >> 16)) * 0x6A09E667) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0xBB67AE85) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _random16(n, seed, step):
    """The two 16-bit random numbers of each element of a tensor, for the rounding of its m and its v: an input, given by the
    tensor's seed and the step."""
    key = _mix64((seed + step * 0x9E3779B97F4A7C15) % 2 ** 64)
    i = torch.arange(n, device="cuda")
    block = _mix32(((i >> 8) + (key & 0xFFFFFFFF)) & 0xFFFFFFFF)
    h = _mix32(((block ^ (key >> 32)) + (i & 255) * 0x9E3779B9) & 0xFFFFFFFF)
    return h & 0xFFFF, h >> 16


def _store8(m1, v1, m, v, scales, seed, step):
    """Writes m1 and v1 in 8 bits: power-of-two scales for blocks of 256, stochastic rounding to e4m3 and e5m2."""
    n = m1.numel()
    rm, rv = _random16(n, seed, step)
    full = -(-n // BLOCK) * BLOCK
    for x, r, to, col, top, low, kept in ((m1, rm, m, 0, 7, 2.0 ** -6, 20), (v1, rv, v, 1, 14, 2.0 ** -14, 21)):
        bits = torch.zeros(full, device="cuda", dtype=torch.int32)
        bits[:n] = x.abs().view(torch.int32)
        code = ((bits.view(-1, BLOCK).amax(1) >> 23) - top).clamp(min=1)
        up = ((254 - code) << 23).view(torch.float32).repeat_interleave(BLOCK)[:n]
        y = x.abs() * up
        off = torch.where(y < low, low, 0.0)
        t = ((y + off).view(torch.int32) + (r.to(torch.int32) << (kept - 16))) & -(1 << kept)
        z = t.view(torch.float32) - off
        if col:
            z = torch.where((x > 0) & (z == 0), 2.0 ** -16, z)
        to.copy_(torch.copysign(z, x))
        scales.view(torch.uint8)[:, col] = code.to(torch.uint8)


# ---------------------------------------------------------------- tokens by expert in their plain form

def _sort(ids, case):
    """Row of each (token, choice), first row of each expert (and the end), kept tokens of each expert."""
    E, cap, a = case["experts"], case["capacity"], case["align"]
    flat = ids.reshape(-1).long()
    known = (flat >= 0) & (flat < E)
    key = torch.where(known, flat, E)
    order = torch.argsort(key, stable=True)
    counts = torch.zeros(E + 1, device="cuda", dtype=torch.int64).scatter_add_(0, key, torch.ones_like(key))
    begin = counts.cumsum(0) - counts
    rank = torch.empty_like(key).scatter_(0, order, torch.arange(key.numel(), device="cuda")) - begin[key]
    counts = counts[:E]
    if cap:
        known = known & (rank < cap)
        counts = counts.clamp(max=cap)
        offsets = torch.arange(E + 1, device="cuda") * cap
    else:
        offsets = torch.zeros(E + 1, device="cuda", dtype=torch.int64)
        offsets[1:] = ((counts + a - 1) // a * a).cumsum(0)
    row = torch.where(known, offsets[key.clamp(max=E - 1)] + rank, -1)
    return row.to(torch.int32).view(ids.shape), offsets.to(torch.int32), counts.to(torch.int32)


def _gather(y, row):
    """y's rows in fp32, zero where there is none: tokens x choices x hidden."""
    return torch.where((row >= 0).unsqueeze(2), y[row.clamp(min=0).long()].float(), 0.0)


def _scatter(x, row, rows):
    """One row of x for each (token, choice), at its place among `rows`, zero elsewhere."""
    out = torch.zeros(rows + 1, x.shape[1], device=x.device, dtype=x.dtype)
    flat = row.reshape(-1).long()
    out[torch.where(flat >= 0, flat, rows)] = x
    return out[:rows]


# ---------------------------------------------------------------- bytes and operations

def work(case):
    if case["op"] in ("adamw", "clip"):
        n = sum(_sizes(case))
        if case["op"] == "clip":
            return {"bytes": n * (BYTES[case["g"]] + BYTES[case["out"]]), "flops": 3 * n}
        state = 16 if case["bits"] == 32 else 4 + 4 / BLOCK
        return {"bytes": n * (2 * BYTES[case["p"]] + BYTES[case["g"]] + state), "flops": 15 * n}
    T, K, H, R, b = case["tokens"], case["topk"], case["hidden"], _rows_of(case), BYTES[case["type"]]
    kept = T * K * (1 - case["masked"])
    if case["capacity"]:
        kept = min(kept, R)
    if case["op"] == "dispatch":
        return {"bytes": T * K * (BYTES[case["ids"]] + 4) + (T + R) * H * b, "flops": 0}
    w = BYTES[case["weights"]]
    if case["op"] == "combine":
        return {"bytes": T * K * (4 + w) + (kept + T) * H * b, "flops": 2 * kept * H}
    return {"bytes": T * K * (4 + 2 * w) + (T + kept + R) * H * b + T * K * 4 + (kept + T) * H * b, "flops": 4 * kept * H}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adamw":
        return _adamw_exact(s, case)
    if case["op"] == "clip":
        total = sum(float(torch.dot(g.double(), g.double())) for g in s["g"])
        norm = math.sqrt(total)
        out = s["flat_out"].double()
        at, _ = _starts(case, _sizes(case), 128)
        for a, g in zip(at, s["g"]):
            out[a: a + g.numel()] = g.double() * min(1.0, s["max_norm"] / (norm + 1e-6))
        return {"norm": torch.tensor(norm, dtype=torch.float64), "out": out}
    T, K, H, R = case["tokens"], case["topk"], case["hidden"], _rows_of(case)
    zeros = lambda n: torch.zeros(n, H, device="cuda", dtype=torch.float64)  # noqa: E731
    if case["op"] == "dispatch":
        row, _, _ = _sort(s["ids"], case)
        xs = zeros(R)
        for k in range(K):
            t = torch.nonzero(row[:, k] >= 0).flatten()
            xs.index_copy_(0, row[t, k].long(), s["x"][t].double())
        return {"row": None, "offsets": None, "counts": None, "xs": xs}
    row = s["row"]
    if case["op"] == "combine":
        out = zeros(T)
        for k in range(K):
            t = torch.nonzero(row[:, k] >= 0).flatten()
            y = s["y"][row[t, k].long()].double()
            out.index_add_(0, t, y if s["w"] is None else y * s["w"][t, k].double().unsqueeze(1))
        return {"out": out}
    dy, dx = zeros(R), zeros(T)
    dw = torch.zeros(T, K, device="cuda", dtype=torch.float64)
    for k in range(K):
        t = torch.nonzero(row[:, k] >= 0).flatten()
        r = row[t, k].long()
        d = s["dout"][t].double()
        dy.index_copy_(0, r, d * s["w"][t, k].double().unsqueeze(1))
        dw[t, k] = torch.einsum("th,th->t", d, s["y"][r].double())
        dx.index_add_(0, t, s["dxs"][r].double())
    return {"dy": dy, "dw": dw, "dx": dx}


def _adamw_exact(s, case):
    t = s["step"] + 1
    out = {k: s["flat_" + k].double() for k in ("p", "m", "v")}
    at, _ = _starts(case, _sizes(case), 128)
    codes = []
    for i, a in enumerate(at):
        n = s["p"][i].numel()
        g, p, m, v = s["g"][i].double(), s["p"][i].double(), s["m"][i].double(), s["v"][i].double()
        if s["scales"] is not None:
            b = torch.arange(n, device="cuda") // BLOCK
            m, v = m * s["scales"][i][:, 0].double()[b], v * s["scales"][i][:, 1].double()[b]
        m, v = m * BETA1 + g * (1 - BETA1), v * BETA2 + g ** 2 * (1 - BETA2)
        step = LR * (m / (1 - BETA1 ** t)) / (torch.sqrt(v / (1 - BETA2 ** t)) + EPS)
        out["p"][a: a + n] = p - LR * DECAY * p - step
        if s["scales"] is not None:
            rm, rv = _random16(n, s["seed"] + i, t)
            pair = []
            for x, r, name, top, mantissa, least in ((m, rm, "m", 7, 3, -6), (v, rv, "v", 14, 2, -14)):
                most = torch.zeros(-(-n // BLOCK), device="cuda", dtype=torch.float64).scatter_reduce_(0, b, x.abs(), "amax")
                e = torch.where(most > 0, torch.frexp(most)[1] - 1 - top, -126).clamp(min=-126)
                y = torch.ldexp(x.abs(), -e[b])
                ulp = torch.ldexp(torch.ones_like(y), (torch.frexp(y)[1] - 1).clamp(min=least) - mantissa)
                q = torch.floor(y / ulp + r.double() / 65536) * ulp
                if name == "v":
                    q = torch.where((x > 0) & (q == 0), 2.0 ** -16, q)
                out[name][a: a + n] = q * torch.sign(x)
                pair.append(torch.ldexp(torch.ones_like(most), e))
            codes.append(torch.stack(pair, 1))
        else:
            out["m"][a: a + n], out["v"][a: a + n] = m, v
    if s["scales"] is not None:
        out["scales"] = torch.cat(codes)
    return out
