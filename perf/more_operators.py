"""Cases of the operators between a training step's token ids and its optimizers, their plain forms and their definition in 64 bits.

Operators: embedding rows with scaling and their gradient, activations kept in 8 bits (e4m3 codes with a power of two for 32
elements), and the gated feed-forward block of experts over tokens sorted by expert (or of one dense layer), forward, and forward
and backward with its activations kept in the inputs' type or in 8 bits.
"""
import math

import torch

own = False

BLOCK = 32  # elements of a row that share a scale
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "int64": torch.int64, "int32": torch.int32}
BYTES = {"f32": 4, "bf16": 2, "int64": 8, "int32": 4}
MOST_WORK = 16384 * 2048 * 8192  # rows x hidden x ffn of a training step


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the token that a served model has just drawn
        dict(name="embed_one_token", op="embed", tokens=1, vocab=65536, hidden=2048, type="bf16", ids="int64", masked=0.0),
        # the words of a training batch
        dict(name="embed_batch", op="embed", tokens=65536, vocab=65536, hidden=2048, type="bf16", ids="int64", masked=0.0),
        # the gradient of a small table of odd sizes, with padding tokens, in fp32
        dict(name="embed_grad_odd", op="embed_grad", tokens=1003, vocab=1001, hidden=1003, type="f32", ids="int32", masked=0.1),
        # the gradient of a training batch, whose words are as uneven as in text
        dict(name="embed_grad_batch", op="embed_grad", tokens=65536, vocab=65536, hidden=2048, type="bf16", ids="int64", masked=0.0),
        # the activations of a small layer of odd width
        dict(name="saved8_odd", op="saved8", rows=1003, cols=1001, type="f32"),
        # both projections of a batch through experts 8192 wide
        dict(name="saved8_batch", op="saved8", rows=16384, cols=16384, type="bf16"),
        # one token of a served model: the weights of two experts are read
        dict(name="ffn_one_token", op="ffn", tokens=1, topk=2, experts=16, hidden=2048, ffn=8192, type="bf16", act="silu", masked=0.0, capacity=0, align=1),
        # a few tokens of a served model: most experts are read, each for a few rows
        dict(name="ffn_few_tokens", op="ffn", tokens=24, topk=2, experts=16, hidden=2048, ffn=8192, type="bf16", act="silu", masked=0.0, capacity=0, align=1),
        # a batch without gradients (prompts, evaluation)
        dict(name="ffn_batch", op="ffn", tokens=16384, topk=2, experts=16, hidden=2048, ffn=8192, type="bf16", act="silu", masked=0.0, capacity=0, align=1),
        # a training step in fp32 with odd sizes, padding tokens and experts that run over their capacity
        dict(name="ffn_train_odd", op="ffn_train", tokens=301, topk=2, experts=5, hidden=201, ffn=333, type="f32", act="gelu", saved=0, masked=0.1, capacity=100, align=1),
        # a training step of a layer of experts
        dict(name="ffn_train_batch", op="ffn_train", tokens=8192, topk=2, experts=16, hidden=2048, ffn=8192, type="bf16", act="silu", saved=0, masked=0.0, capacity=0, align=1),
        # the same with a capacity factor of 1.25 and the activations in 8 bits
        dict(name="ffn_train_saved8", op="ffn_train", tokens=8192, topk=2, experts=16, hidden=2048, ffn=8192, type="bf16", act="silu", saved=8, masked=0.0, capacity=1280, align=1),
    ]


def _spread(rng, lo, hi):
    hi = max(lo, hi)
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "saved8", "ffn", "ffn", "ffn_train", "ffn_train"])
    if op in ("embed", "embed_grad"):
        hidden = rng.choice([_spread(rng, 16, 8192), 8 * _spread(rng, 4, 1024), 2048, 6144])
        vocab = _spread(rng, 32, min(262144, (1 << 27) // hidden))
        tokens = _spread(rng, 1, min(262144, (1 << 27) // hidden))
        return dict(op=op, tokens=tokens, vocab=vocab, hidden=hidden, type=rng.choice(["bf16", "bf16", "f32"]), ids=rng.choice(["int64", "int32"]), masked=rng.choice([0.0, 0.0, 0.2]))
    if op == "saved8":
        cols = rng.choice([_spread(rng, 1, 16384), 8 * _spread(rng, 2, 2048), 2048, 8192])
        return dict(op=op, rows=_spread(rng, 1, min(65536, (1 << 28) // cols)), cols=cols, type=rng.choice(["bf16", "bf16", "f32"]))
    kind = rng.choice(["bf16", "bf16", "bf16", "f32"])
    odd = kind == "f32" or rng.random() < 0.25
    width = lambda: _spread(rng, 64, 2048) if odd else rng.choice([8 * _spread(rng, 8, 512), 128 * _spread(rng, 1, 32), 2048])  # noqa: E731
    hidden, ffn = width(), rng.choice([width(), 8192] if not odd else [width()])
    experts = rng.choice([0, _spread(rng, 2, 64), _spread(rng, 2, 64), 16])  # 0: one dense layer
    while max(experts, 1) * hidden * ffn > 16 * 2048 * 8192:
        experts //= 2
    topk = rng.choice([k for k in (1, 2, 2, 4, 8) if k <= max(experts, 1)])
    most = MOST_WORK // (hidden * ffn * topk) // (1 if kind == "bf16" and not odd else 64)
    tokens = _spread(rng, 1, min(32768 // topk, most))
    capacity = rng.choice([0, 0, max(1, int(1.25 * tokens * topk / experts))]) if experts else 0
    case = dict(op=op, tokens=tokens, topk=topk, experts=experts, hidden=hidden, ffn=ffn, type=kind, act=rng.choice(["silu", "gelu"]),
                masked=rng.choice([0.0, 0.0, 0.15]) if experts else 0.0, capacity=capacity, align=1 if capacity or not experts else rng.choice([1, 1, 16, 128]))
    return case if op == "ffn" else dict(case, saved=rng.choice([0, 8]))


# ---------------------------------------------------------------- what a program has in hand

def _rows_of(case):
    """Rows of the buffer that holds the sorted tokens."""
    if case["capacity"]:
        return case["experts"] * case["capacity"]
    a = case["align"]
    return -(-(case["tokens"] * case["topk"] + max(case["experts"], 1) * (a - 1)) // a) * a


def _sort(ids, case):
    """Row of each (token, choice), first row of each expert (and the end), kept tokens of each expert."""
    E, cap, a = case["experts"], case["capacity"], case["align"]
    flat = ids.reshape(-1)
    known = flat >= 0
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


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    kind = TYPES[case["type"]]
    rand = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    s = {"case": case, "seed": seed}
    if case["op"] in ("embed", "embed_grad"):
        T, V, H = case["tokens"], case["vocab"], case["hidden"]
        # words by rank: the chance of the n-th is about 1/n, and where it stands in the table says nothing
        word = torch.rand(T, generator=gen, device="cuda").mul_(math.log(V + 1)).exp_().long().sub_(1).clamp_(0, V - 1)
        ids = torch.randperm(V, generator=gen, device="cuda")[word]
        if case["masked"]:
            ids = torch.where(torch.rand(T, generator=gen, device="cuda") < case["masked"], -1, ids)
        s["ids"] = ids.to(TYPES[case["ids"]])
        s["scale"] = math.sqrt(H)
        if case["op"] == "embed":
            s["table"] = rand(V, H).mul_(0.02).to(kind)
        else:
            s["dout"] = rand(T, H).mul_(1e-4).to(kind)
        return s
    if case["op"] == "saved8":
        # activations: of different size from column to column, and a few far out
        x = rand(case["rows"], case["cols"]).mul_(rand(case["cols"]).exp_())
        x.mul_(1 + 30 * (torch.rand(case["cols"], generator=gen, device="cuda") < 0.01))
        s["x"] = x.to(kind)
        return s
    T, K, E, H, F, R = case["tokens"], case["topk"], case["experts"], case["hidden"], case["ffn"], _rows_of(case)
    x = rand(T, H).to(kind)
    if E:
        ids = (rand(T, E) + 0.3 * rand(E)).topk(K, dim=1).indices
        if case["masked"]:  # tokens of padding go to no expert
            ids = torch.where(torch.rand(T, 1, generator=gen, device="cuda") < case["masked"], -1, ids)
        s["row"], s["offsets"], s["counts"] = _sort(ids, case)
        s["x"] = torch.zeros(R, H, device="cuda", dtype=kind)
        t, k = torch.nonzero(s["row"] >= 0, as_tuple=True)
        s["x"][s["row"][t, k].long()] = x[t]
        s["ranges"] = [(e, a, a + n) for e, (a, n) in enumerate(zip(s["offsets"].tolist(), s["counts"].tolist())) if n]
        some = torch.zeros(R, 1, device="cuda")
        some[s["row"][t, k].long()] = 1
    else:
        s["x"], s["ranges"], some = x, [(0, 0, T)], 1
    many = (E,) if E else ()
    s["gate"] = torch.empty(*many, F, H, device="cuda", dtype=kind)
    s["up"] = torch.empty(*many, F, H, device="cuda", dtype=kind)
    s["down"] = torch.empty(*many, H, F, device="cuda", dtype=kind)
    for w in (s["gate"], s["up"], s["down"]):
        for one in (w if E else [w]):
            one.copy_(rand(*one.shape).mul_(one.shape[1] ** -0.5))
    if case["op"] == "ffn_train":
        s["dy"] = rand(R, H).mul_(some).mul_(1e-3).to(kind)
    return s


# ---------------------------------------------------------------- the operators

def run(s):
    return (_run_own if own else _run_plain)(s, s["case"])


def _run_own(s, case):
    from muon_newton_schulz_gb300 import checkpoint, embedding, ffn, moe

    if case["op"] == "embed":
        return {"out": embedding.embed(s["ids"], s["table"], scale=s["scale"])}
    if case["op"] == "embed_grad":
        return {"dtable": embedding.embed_backward(s["dout"], s["ids"], case["vocab"], scale=s["scale"])}
    if case["op"] == "saved8":
        return {"x": checkpoint.unpack(checkpoint.pack(s["x"]))}
    route = moe.Route(s["row"], s["offsets"], s["counts"], capacity=case["capacity"], align=case["align"]) if case["experts"] else None
    if case["op"] == "ffn":
        return {"y": ffn.gated_ffn(s["x"], s["gate"], s["up"], s["down"], route, activation=case["act"])}
    y, saved = ffn.gated_ffn_saved(s["x"], s["gate"], s["up"], s["down"], route, activation=case["act"], saved_bits=case["saved"] or None)
    dx, dgate, dup, ddown = ffn.gated_ffn_backward(s["dy"], saved, s["gate"], s["up"], s["down"])
    return {"y": y, "dx": dx, "dgate": dgate, "dup": dup, "ddown": ddown}


def _run_plain(s, case):
    kind = TYPES[case["type"]]
    if case["op"] == "embed":
        known = (s["ids"] >= 0).unsqueeze(1)
        return {"out": torch.where(known, s["table"][s["ids"].clamp(min=0)].float() * s["scale"], 0.0).to(kind)}
    if case["op"] == "embed_grad":
        V = case["vocab"]
        at = torch.where(s["ids"] >= 0, s["ids"], V)
        total = torch.zeros(V + 1, case["hidden"], device="cuda").index_add_(0, at, s["dout"].float())
        return {"dtable": (total[:V] * s["scale"]).to(kind)}
    if case["op"] == "saved8":
        return {"x": _kept8(s["x"].float()).to(kind)}
    x, many = s["x"], case["experts"] > 0
    one = lambda w, e: (w[e] if many else w).float()  # noqa: E731
    y = torch.zeros_like(x)
    if case["op"] == "ffn":
        for e, a, b in s["ranges"]:
            xe = x[a:b].float()
            h = _act(xe @ one(s["gate"], e).t(), case["act"]) * (xe @ one(s["up"], e).t())
            y[a:b] = (h @ one(s["down"], e).t()).to(kind)
        return {"y": y}
    dx = torch.zeros_like(x)
    dgate, dup, ddown = (torch.zeros_like(s[k]) for k in ("gate", "up", "down"))
    for e, a, b in s["ranges"]:
        gate, up, down = one(s["gate"], e), one(s["up"], e), one(s["down"], e)
        xe, dy = x[a:b].float(), s["dy"][a:b].float()
        g, u = xe @ gate.t(), xe @ up.t()
        y[a:b] = ((_act(g, case["act"]) * u) @ down.t()).to(kind)
        if case["saved"]:
            xe, g, u = _kept8(xe), _kept8(g), _kept8(u)
        act, slope = _act(g, case["act"]), _slope(g, case["act"])
        dh = dy @ down
        dg, du = dh * u * slope, dh * act
        dx[a:b] = (dg @ gate + du @ up).to(kind)
        for to, product in ((dgate, dg.t() @ xe), (dup, du.t() @ xe), (ddown, dy.t() @ (act * u))):
            (to[e] if many else to).copy_(product)
    return {"y": y, "dx": dx, "dgate": dgate, "dup": dup, "ddown": ddown}


def _act(g, act):
    return g * torch.sigmoid(g) if act == "silu" else g * (0.5 * (1 + torch.erf(g * math.sqrt(0.5))))


def _slope(g, act):
    if act == "silu":
        s = torch.sigmoid(g)
        return s * (1 + g * (1 - s))
    return 0.5 * (1 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)


def _kept8(x):
    """What e4m3 codes of x stand for: each 32 elements of a row are scaled by the power of two that brings the largest to
    [128, 256), and rounded to nearest."""
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    most = torch.nn.functional.pad(x, (0, blocks * BLOCK - cols)).view(rows, blocks, BLOCK).abs().amax(2)
    code = ((most.view(torch.int32) >> 23) - 7).clamp(min=1)
    each = code.repeat_interleave(BLOCK, 1)[:, :cols]
    return (x * ((254 - each) << 23).view(torch.float32)).to(torch.float8_e4m3fn).float() * (each << 23).view(torch.float32)


# ---------------------------------------------------------------- bytes and operations

def work(case):
    b = BYTES[case["type"]]
    if case["op"] == "embed":
        return {"bytes": case["tokens"] * (BYTES[case["ids"]] + 2 * case["hidden"] * b), "flops": case["tokens"] * case["hidden"]}
    if case["op"] == "embed_grad":
        return {"bytes": case["tokens"] * BYTES[case["ids"]] + (case["tokens"] + case["vocab"]) * case["hidden"] * b, "flops": case["tokens"] * case["hidden"]}
    if case["op"] == "saved8":
        n = case["rows"] * case["cols"]
        return {"bytes": n * 2 * (b + 1 + 1 / BLOCK), "flops": 2 * n}
    H, F, E = case["hidden"], case["ffn"], max(case["experts"], 1)
    kept = case["tokens"] * case["topk"] * (1 - case["masked"])
    if case["capacity"]:
        kept = min(kept, _rows_of(case))
    used = min(E, E * (1 - (1 - case["topk"] / E) ** case["tokens"])) if case["experts"] else 1  # experts with a token
    weights = 3 * used * H * F * b
    if case["op"] == "ffn":
        return {"bytes": weights + 2 * kept * H * b, "flops": 6 * kept * H * F}
    return {"bytes": 2 * weights + 4 * kept * H * b, "flops": 18 * kept * H * F}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("embed", "embed_grad"):
        ids = s["ids"].long()
        t = torch.nonzero(ids >= 0).flatten()
        if case["op"] == "embed":
            out = torch.zeros(case["tokens"], case["hidden"], device="cuda", dtype=torch.float64)
            out[t] = s["table"][ids[t]].double() * s["scale"]
            return {"out": out}
        dtable = torch.zeros(case["vocab"], case["hidden"], device="cuda", dtype=torch.float64)
        for part in t.split(16384):
            dtable.index_add_(0, ids[part], s["dout"][part].double() * s["scale"])
        return {"dtable": dtable}
    if case["op"] == "saved8":
        return {"x": torch.cat([_kept8_exact(x.double()) for x in s["x"].split(2048)])}
    many = case["experts"] > 0
    pick = lambda w, e: (w[e] if many else w).double()  # noqa: E731
    zeros = lambda t: torch.zeros(t.shape, device="cuda", dtype=torch.float64)  # noqa: E731
    out = {"y": zeros(s["x"])}
    train = case["op"] == "ffn_train"
    if train:
        out.update(dx=zeros(s["x"]), dgate=zeros(s["gate"]), dup=zeros(s["up"]), ddown=zeros(s["down"]))
    for e, a, b in s["ranges"]:
        x, wg, wu, wd = s["x"][a:b].double(), pick(s["gate"], e), pick(s["up"], e), pick(s["down"], e)
        g, u = torch.einsum("rh,fh->rf", x, wg), torch.einsum("rh,fh->rf", x, wu)
        out["y"][a:b] = torch.einsum("rf,hf->rh", _act_exact(g, case["act"])[0] * u, wd)
        if not train:
            continue
        if case["saved"]:
            x, g, u = _kept8_exact(x), _kept8_exact(g), _kept8_exact(u)
        act, slope = _act_exact(g, case["act"])
        dy = s["dy"][a:b].double()
        dh = torch.einsum("rh,hf->rf", dy, wd)
        dg, du = dh * u * slope, dh * act
        out["dx"][a:b] = torch.einsum("rf,fh->rh", dg, wg) + torch.einsum("rf,fh->rh", du, wu)
        for name, p, q in (("dgate", dg, x), ("dup", du, x), ("ddown", dy, act * u)):
            (out[name][e] if many else out[name]).copy_(torch.einsum("ri,rj->ij", p, q))
    return out


def _act_exact(g, act):
    """The activation and its derivative."""
    if act == "silu":
        down = 1 / (1 + torch.exp(g))  # 1 - sigmoid
        return g * (1 - down), (1 - down) * (1 + g * down)
    cdf = 0.5 * torch.erfc(-g / math.sqrt(2))
    return g * cdf, cdf + g * torch.exp(-g ** 2 / 2) / math.sqrt(2 * math.pi)


def _kept8_exact(x):
    rows, cols = x.shape
    at = torch.arange(cols, device="cuda") // BLOCK
    most = torch.zeros(rows, -(-cols // BLOCK), device="cuda", dtype=torch.float64).scatter_reduce_(1, at.expand(rows, cols), x.abs(), "amax")
    e = torch.where(most > 0, torch.frexp(most)[1] - 8, -126).clamp(min=-126)[:, at]
    y = x * _power_of_two(-e)
    e_y = (torch.frexp(y)[1] - 1).clamp(min=-6) - 3
    return torch.round(y * _power_of_two(-e_y)) * _power_of_two(e + e_y)


def _power_of_two(e):
    return ((e.long() + 1023) << 52).view(torch.float64)  # torch.ldexp's are an ulp off on the GPU
