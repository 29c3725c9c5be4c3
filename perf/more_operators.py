"""More operators of a QLoRA training step around its 4-bit linears, and what one pass of each costs:

- the rotation of queries and keys by their positions (half and interleaved pairs, part of the head, frequencies scaled
  for long contexts), forward and backward, and the same with a norm of every head before it;
- the Muon step over a list of adapter matrices: momentum, the update orthogonalised by Newton-Schulz products, the
  weight's step; and the orthogonalising alone.

`run` computes them in elementary torch operations in fp32 (`own` false) or through nf4_quantize_amd (`own` true).
Sizes are those of this repository's weight stack (hidden 4096, key/value 1024, MLP 14336), of its linear workload
(4096 tokens of width 8192), and generic ones."""
import math

import torch

own = False

DEV = "cuda"
NORM_EPS = 1e-6
BASE = 10000.0
LENGTH = 4096        # the context that scaled frequencies start from
LR, DECAY, MOMENTUM, MUON_EPS = 2e-3, 0.1, 0.95, 1e-7
COEFFICIENTS = (3.4445, -4.775, 2.0315)
ITERATIONS = 5


def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _bytes(name):
    return 2 if name == "bf16" else 4


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one token of one sequence at a far position, between the projections and attention: all latency
        dict(name="rotary_token", op="rotary", batch=1, tokens=1, hq=32, hk=8, dim=128, rot=128, layout="half", order="token", positions="far", scaling="none", dtype="bf16", norm=False, wt="bf16"),
        # a long prompt, queries and keys as slices of one projection's output, frequencies scaled for eight times the context
        dict(name="rotary_prompt", op="rotary", batch=1, tokens=16384, hq=32, hk=8, dim=128, rot=128, layout="half", order="fused", positions="start", scaling="yarn", dtype="bf16", norm=False, wt="bf16"),
        # the gradient for packed documents in fp32: odd numbers of tokens and heads, a quarter of the head rotated, [batch, heads, tokens, dim] in memory
        dict(name="rotary_bwd_odd", op="rotary_bwd", batch=3, tokens=1001, hq=7, hk=1, dim=80, rot=20, layout="interleaved", order="head", positions="packed", scaling="linear", dtype="f32", norm=False, wt="f32"),
        # a decoding batch: every sequence's newest token, with the norms of its heads
        dict(name="head_norm_decode", op="rotary", batch=16, tokens=1, hq=64, hk=8, dim=128, rot=128, layout="half", order="token", positions="far", scaling="wavelength", dtype="bf16", norm=True, wt="bf16"),
        # the training batch of the linear workload
        dict(name="head_norm_batch", op="rotary", batch=4, tokens=1024, hq=64, hk=8, dim=128, rot=128, layout="half", order="token", positions="start", scaling="none", dtype="bf16", norm=True, wt="f32"),
        # its backward pass, with both norms' weights, from attention's gradients in [batch, heads, tokens, dim]
        dict(name="head_norm_bwd_batch", op="rotary_bwd", batch=4, tokens=1024, hq=64, hk=8, dim=128, rot=128, layout="half", order="head", positions="start", scaling="none", dtype="bf16", norm=True, wt="f32"),
        # heads of an odd width, half of it rotated, few of them, fp32
        dict(name="head_norm_bwd_odd", op="rotary_bwd", batch=2, tokens=555, hq=5, hk=3, dim=75, rot=38, layout="interleaved", order="fused", positions="packed", scaling="ntk", dtype="f32", norm=True, wt="f32"),
        # one linear's adapter of low rank: the smallest optimizer call
        dict(name="muon_one_adapter", op="muon", hidden=4096, kv=0, mlp=0, layers=1, rank=16, w="bf16", g="bf16", m="f32", master=False, nesterov=True),
        # a layer of odd sizes with fp32 adapters and gradients
        dict(name="muon_odd_layer", op="muon", hidden=2047, kv=511, mlp=5461, layers=1, rank=13, w="f32", g="f32", m="f32", master=False, nesterov=False),
        # every adapter of the 32-layer stack at rank 64: 448 tensors, 168 million parameters, the step a QLoRA run takes
        dict(name="muon_stack", op="muon", hidden=4096, kv=1024, mlp=14336, layers=32, rank=64, w="bf16", g="bf16", m="f32", master=False, nesterov=True),
        # one linear's adapter of an odd rank, fp32, its updates alone
        dict(name="orthogonalize_small", op="orthogonalize", hidden=777, kv=0, mlp=0, layers=1, rank=9, w="f32", g="f32", m="f32", master=False, nesterov=False),
        # a layer's adapters of the largest rank that the linears take
        dict(name="orthogonalize_rank256", op="orthogonalize", hidden=4096, kv=1024, mlp=14336, layers=1, rank=256, w="bf16", g="bf16", m="f32", master=False, nesterov=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "rotary", "rotary_bwd", "rotary_bwd", "muon", "muon", "orthogonalize"])
    if op.startswith("rotary"):
        dim = rng.choice([64, 128, rng.choice([80, 96, 256]), _log_int(rng, 2, 512)])
        rot = rng.choice([dim, dim, dim // 2, dim // 4])
        rot = max(2, rot // 2 * 2)
        hk = _log_int(rng, 1, 16)
        hq = hk * rng.choice([1, 2, 4, 8]) if rng.random() < 0.8 else _log_int(rng, 1, 64)
        tokens = _log_int(rng, 1, max(1, min(65536, 60_000_000 // (dim * (hq + hk)))))
        batch = rng.choice([1, 1, 2, 3, 16])
        if batch > tokens:
            batch, tokens = tokens, 1
        else:
            tokens = max(1, tokens // batch)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        return dict(op=op, batch=batch, tokens=tokens, hq=hq, hk=hk, dim=dim, rot=rot, layout=rng.choice(["half", "interleaved"]),
                    order=rng.choice(["token", "head", "fused"]), positions=rng.choice(["start", "packed", "far"]),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn", "wavelength"]), dtype=dtype, norm=rng.random() < 0.6,
                    wt=rng.choice(["f32", dtype]))
    hidden = _log_int(rng, 48, 8192)
    kv, mlp = rng.choice([(0, 0), (max(1, hidden // 4), hidden * 7 // 2), (hidden, hidden * 8 // 3)])
    rank = rng.choice([_log_int(rng, 1, 256), rng.choice([8, 16, 32, 64, 128])])
    layers = _log_int(rng, 1, 32)
    w, g = rng.choice([("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")]) if op == "muon" else rng.choice([("bf16", "bf16"), ("f32", "f32")])
    c = dict(op=op, hidden=hidden, kv=kv, mlp=mlp, layers=layers, rank=rank, w=w, g=g, m=rng.choice(["f32", "f32", "bf16"]),
             master=op == "muon" and w == "bf16" and rng.random() < 0.5, nesterov=rng.random() < 0.7)
    most = 80e6 if w == g == "bf16" else 40e6
    while c["layers"] > 1 and sum(a * b for a, b in _shapes(c)) * max(1.0, rank / 64) > most:
        c["layers"] //= 2
    return c


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


# How a case's frequencies are scaled, as NF4Rotary takes it.
SCALINGS = {"none": None, "linear": dict(kind="linear", factor=4.0), "ntk": dict(kind="ntk", factor=4.0),
            "yarn": dict(kind="yarn", factor=8.0, length=LENGTH),
            "wavelength": dict(kind="wavelength", factor=8.0, length=LENGTH, low=1.0, high=4.0)}


def _frequencies(c):
    """Radians a position for each pair, and the factor of cosine and sine."""
    r, kind = c["rot"], c["scaling"]
    i = torch.arange(r // 2, dtype=torch.float64)
    f = BASE ** (-2.0 * i / r)
    if kind == "none":
        return f, 1.0
    s = SCALINGS[kind]["factor"]
    if kind == "linear":
        return f / s, 1.0
    if kind == "ntk":
        return (BASE * s ** (r / (r - 2.0)) if r > 2 else BASE) ** (-2.0 * i / r), 1.0
    if kind == "yarn":
        # pairs that turn more than 32 times in the first context keep their frequency, those below one turn are slowed
        def place(turns):
            return r * math.log(LENGTH / (turns * 2 * math.pi)) / (2 * math.log(BASE))

        low, high = max(math.floor(place(32.0)), 0), min(math.ceil(place(1.0)), r - 1)
        ramp = ((i - low) / max(high - low, 1e-3)).clamp(0, 1)
        return f / s * ramp + f * (1 - ramp), 0.1 * math.log(s) + 1.0
    turns = LENGTH * f / (2 * math.pi)  # in the first context: slowed below one, kept above four, blended between
    blend = ((turns - 1.0) / 3.0).clamp(0, 1)
    return f / s * (1 - blend) + f * blend, 1.0


def _heads(g, c, n, like):
    """[batch, tokens, n, dim] values in the case's order in memory."""
    b, t, d = c["batch"], c["tokens"], c["dim"]
    channel = torch.exp(0.4 * _randn(g, d))  # some channels carry more than others
    if c["order"] == "head":
        return (_randn(g, b, n, t, d) * channel).to(_dt(c["dtype"])).transpose(1, 2)
    return like.copy_(_randn(g, b, t, n, d) * channel) if like is not None else (_randn(g, b, t, n, d) * channel).to(_dt(c["dtype"]))


def _query_key(g, c):
    """Queries and keys, in the fused order as slices of one projection's rows (with as many values as keys behind them)."""
    if c["order"] != "fused":
        return _heads(g, c, c["hq"], None), _heads(g, c, c["hk"], None)
    both = torch.zeros(c["batch"], c["tokens"], c["hq"] + 2 * c["hk"], c["dim"], dtype=_dt(c["dtype"]), device=DEV)
    q, k = both[:, :, :c["hq"]], both[:, :, c["hq"]:c["hq"] + c["hk"]]
    return _heads(g, c, c["hq"], q), _heads(g, c, c["hk"], k)


def _prepare_rotary(c, seed):
    g = _gen(seed)
    b, t = c["batch"], c["tokens"]
    s = {"c": c, "q": None, "k": None, "w_q": None, "w_k": None}
    if c["op"] == "rotary" or c["norm"]:
        s["q"], s["k"] = _query_key(g, c)
    if c["op"] == "rotary_bwd":
        s["dq"], s["dk"] = _query_key(g, {**c, "order": "head" if c["order"] == "head" else "token"})
    if c["norm"]:
        s["w_q"], s["w_k"] = ((1 + 0.2 * _randn(g, c["dim"])).to(_dt(c["wt"])) for _ in range(2))
    s["positions"] = None
    if c["positions"] == "packed":  # documents of different lengths one after the other in every row
        cut = torch.rand(b, t, generator=g, device=DEV) < 8.0 / t
        at = torch.arange(t, device=DEV).expand(b, t)
        s["positions"] = (at - torch.cummax(torch.where(cut, at, 0), 1).values).int()
    elif c["positions"] == "far":  # every sequence at its own length
        s["positions"] = torch.randint(0, 1_000_000, (b, 1), generator=g, device=DEV) + torch.arange(t, device=DEV)
    if own:
        import nf4_quantize_amd as nq

        s["rope"] = nq.NF4Rotary(c["rot"], base=BASE, layout=c["layout"], scaling=SCALINGS[c["scaling"]], device=DEV)
    else:
        f, s["scale"] = _frequencies(c)
        s["frequencies"] = f.to(DEV)
    return s


def _shapes(c):
    """Adapter tensors [K, r] and [r, N] of each linear: q, k, v, o, gate, up, down (the first alone where kv is 0)."""
    h, kv, mlp, r = c["hidden"], c["kv"], c["mlp"], c["rank"]
    linears = [(h, h), (h, kv), (h, kv), (h, h), (h, mlp), (h, mlp), (mlp, h)] if kv else [(h, h)]
    return [s for _ in range(c["layers"]) for k, n in linears for s in ((k, r), (r, n))]


def _short_side_mixed(g, x, short_first):
    """Gives the rows or columns of the shorter side unlike sizes and correlates them, as gradients of one adapter are."""
    n = x.shape[0 if short_first else 1]
    mix = _randn(g, n, n) / math.sqrt(n) * torch.exp(0.5 * _randn(g, n, 1))
    return mix @ x if short_first else x @ mix


def _views(c, flat):
    """The case's tensors in one buffer, each from a multiple of 256 elements on."""
    out, at = [], 0
    for a, b in _shapes(c):
        out.append(flat[at:at + a * b].view(a, b))
        at += -(-a * b // 256) * 256
    return out


def _flat(c, name):
    return torch.zeros(sum(-(-a * b // 256) * 256 for a, b in _shapes(c)), dtype=_dt(name), device=DEV)


def _prepare_muon(c, seed):
    g = _gen(seed)
    s = {"c": c, "grads": _views(c, _flat(c, c["g"]))}
    if c["op"] == "orthogonalize":
        s["flat"] = {"out": _flat(c, c["g"])}
    else:
        s["flat"] = {"w": _flat(c, c["w"]), "m": _flat(c, c["m"]), **({"masters": _flat(c, "f32")} if c["master"] else {})}
    s.update({k: _views(c, x) for k, x in s["flat"].items()})
    for i, (a, b) in enumerate(_shapes(c)):
        u = _short_side_mixed(g, _randn(g, a, b), a < b) * 1e-3
        s["grads"][i].copy_(u)
        if c["op"] == "muon":
            s["m"][i].copy_(0.4 * u + 3e-4 * _randn(g, a, b))
            w = _randn(g, a, b) * 0.02
            s["w"][i].copy_(w)
            if c["master"]:
                s["masters"][i].copy_(w)
    if own and c["op"] == "muon":
        import nf4_quantize_amd as nq

        s["opt"] = nq.NF4Muon([dict(params=s["w"], masters=s.get("masters"))], lr=LR, weight_decay=DECAY, momentum=MOMENTUM,
                              nesterov=c["nesterov"], coefficients=COEFFICIENTS, iterations=ITERATIONS, eps=MUON_EPS,
                              state_bits=32 if c["m"] == "f32" else 16, adjust="shape")
        s["opt"].bind_state(s["m"])
    return s


def prepare(case, seed):
    return (_prepare_rotary if case["op"].startswith("rotary") else _prepare_muon)(case, seed)


# ------------------------------------------------------------------ plain forms

def _cos_sin(s):
    c = s["c"]
    at = torch.arange(c["tokens"], device=DEV).unsqueeze(0) if s["positions"] is None else s["positions"]
    angle = at.double().unsqueeze(2) * s["frequencies"]
    return [(f(angle) * s["scale"]).float().unsqueeze(2) for f in (torch.cos, torch.sin)]


def _rotated(c, x, cos, sin):
    r = c["rot"]
    out = x.clone()
    if c["layout"] == "half":
        first, second = slice(0, r // 2), slice(r // 2, r)
    else:
        first, second = slice(0, r, 2), slice(1, r, 2)
    a, b = x[..., first], x[..., second]
    out[..., first] = a * cos - b * sin
    out[..., second] = b * cos + a * sin
    return out


def _plain_rotary(s):
    c = s["c"]
    cos, sin = _cos_sin(s)
    out = []
    for x, w in ((s["q"], s["w_q"]), (s["k"], s["w_k"])):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(3, keepdim=True) + NORM_EPS) * w.float()
        out.append(_rotated(c, y, cos, sin).to(x.dtype))
    return out


def _plain_rotary_bwd(s):
    c = s["c"]
    cos, sin = _cos_sin(s)
    out = []
    for dy, x, w in ((s["dq"], s["q"], s["w_q"]), (s["dk"], s["k"], s["w_k"])):
        g = _rotated(c, dy.float(), cos, -sin)
        if w is not None:
            r = torch.rsqrt((x.float() * x.float()).mean(3, keepdim=True) + NORM_EPS)
            n = x.float() * r
            out.append((g * n).sum((0, 1, 2)).to(w.dtype))
            p = g * w.float()
            g = r * (p - n * (p * n).mean(3, keepdim=True))
        out.append(g.to(dy.dtype))
    return out


def _plain_orthogonal(u):
    a, b, c = COEFFICIENTS
    x = u / torch.sqrt((u * u).sum()).clamp_min(MUON_EPS)
    flip = x.shape[0] > x.shape[1]
    x = x.t().contiguous() if flip else x
    for _ in range(ITERATIONS):
        gram = x @ x.t().contiguous()
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.t() if flip else x


def _adjust(shape):
    return math.sqrt(max(1.0, shape[0] / shape[1]))


def _plain_muon(s):
    c = s["c"]
    for i, g in enumerate(s["grads"]):
        g = g.float()
        if c["op"] == "orthogonalize":
            s["out"][i].copy_(_plain_orthogonal(g))
            continue
        w = (s["masters"] if c["master"] else s["w"])[i].float()
        m = MOMENTUM * s["m"][i].float() + (1 - MOMENTUM) * g
        u = MOMENTUM * m + (1 - MOMENTUM) * g if c["nesterov"] else m
        w = w * (1 - LR * DECAY) - LR * _adjust(g.shape) * _plain_orthogonal(u)
        s["m"][i].copy_(m)
        s["w"][i].copy_(w)
        if c["master"]:
            s["masters"][i].copy_(w)
    return s["flat"]


# ------------------------------------------------------------------ one pass

def run(state):
    s, c = state, state["c"]
    op = c["op"]
    if not own:
        return {"rotary": _plain_rotary, "rotary_bwd": _plain_rotary_bwd}.get(op, _plain_muon)(s)
    import nf4_quantize_amd as nq

    if op == "rotary":
        return list(nq.rotary_forward(s["q"], s["k"], s["positions"], s["rope"], s["w_q"], s["w_k"], eps=NORM_EPS))
    if op == "rotary_bwd":
        dq, dk, dw_q, dw_k = nq.rotary_backward(s["dq"], s["dk"], s["positions"], s["rope"], s["q"], s["k"], s["w_q"], s["w_k"], eps=NORM_EPS)
        return [dw_q, dq, dw_k, dk] if c["norm"] else [dq, dk]
    if op == "orthogonalize":
        nq.orthogonalize(s["grads"], coefficients=COEFFICIENTS, iterations=ITERATIONS, eps=MUON_EPS, outs=s["out"])
    else:
        s["opt"].step(s["grads"])
    return s["flat"]


# ------------------------------------------------------------------ the floor

def work(case):
    c = case
    if c["op"].startswith("rotary"):
        rows = c["batch"] * c["tokens"]
        n = rows * (c["hq"] + c["hk"]) * c["dim"]
        arrays = 3 if c["op"] == "rotary_bwd" and c["norm"] else 2
        at = {"start": 0, "packed": 4, "far": 8}[c["positions"]] * rows
        return {"bytes": n * arrays * _bytes(c["dtype"]) + at, "flops": n * (3 + (0 if not c["norm"] else 4 if arrays == 2 else 10))}
    n = sum(a * b for a, b in _shapes(c))
    # the Gram matrix (half of it, being symmetric) and the product with a polynomial of it
    flops = sum(3 * a * b * min(a, b) for a, b in _shapes(c))
    if c["op"] == "orthogonalize":
        return {"bytes": n * 2 * _bytes(c["g"]), "flops": flops}
    w = _bytes(c["w"]) + 8 if c["master"] else 2 * _bytes(c["w"])
    return {"bytes": n * (w + _bytes(c["g"]) + 2 * _bytes(c["m"])), "flops": flops + 8 * n}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_rotary(c, s):
    """Pairs as complex numbers, turned by exp(i position f)."""
    at = torch.arange(c["tokens"], device=DEV).unsqueeze(0).expand(c["batch"], -1) if s["positions"] is None else s["positions"]
    turn = s["scale"] * torch.exp(1j * (at.double()[:, :, None] * s["frequencies"]).to(torch.complex128))[:, :, None]
    r = c["rot"]

    def apply(x, z):
        pairs = (torch.stack((x[..., :r // 2], x[..., r // 2:r]), -1) if c["layout"] == "half" else x[..., :r].unflatten(-1, (r // 2, 2)))
        y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
        y = torch.cat((y[..., 0], y[..., 1]), -1) if c["layout"] == "half" else y.flatten(-2)
        return torch.cat((y, x[..., r:]), -1)

    out = []
    for x, dy, w in ((s["q"], s.get("dq"), s["w_q"]), (s["k"], s.get("dk"), s["w_k"])):
        if w is not None:
            x, w = x.double(), w.double()
            size = (x.pow(2).sum(3, keepdim=True) / c["dim"] + NORM_EPS).sqrt()
        if dy is None:
            out.append(apply(x.double() if w is None else x / size * w, turn))
            continue
        g = apply(dy.double(), turn.conj())
        if w is not None:
            out.append((g * x / size).sum((0, 1, 2)))
            # d(x / size): 1 / size on the difference, and size's own gradient x / (dim size)
            g = g * w / size - x * ((g * w * x).sum(3, keepdim=True) / (c["dim"] * size ** 3))
        out.append(g)
    return out


def _exact_orthogonal(u):
    a, b, c = COEFFICIENTS
    x = u / max(float(u.norm()), MUON_EPS)
    for _ in range(ITERATIONS):  # with the longer side's Gram matrix never formed: x g, g the shorter side's
        if x.shape[0] >= x.shape[1]:
            xg = x @ (x.mT @ x)
            x = a * x + b * xg + c * (xg @ (x.mT @ x))
        else:
            gx = (x @ x.mT) @ x
            x = a * x + b * gx + c * ((x @ x.mT) @ gx)
    return x


def _exact_muon(c, s):
    flat = {k: torch.zeros(x.numel(), dtype=torch.float64, device=DEV) for k, x in s["flat"].items()}
    out = {k: _views(c, x) for k, x in flat.items()}
    for i, g in enumerate(s["grads"]):
        g = g.double()
        if c["op"] == "orthogonalize":
            out["out"][i].copy_(_exact_orthogonal(g))
            continue
        m = s["m"][i].double() + (1 - MOMENTUM) * (g - s["m"][i].double())
        u = m + (1 - MOMENTUM) * (g - m) if c["nesterov"] else m
        w = (s["masters"] if c["master"] else s["w"])[i].double()
        out["m"][i].copy_(m)
        out["w"][i].copy_(w - LR * (DECAY * w + _adjust(g.shape) * _exact_orthogonal(u)))
        if c["master"]:
            out["masters"][i].copy_(out["w"][i])
    return flat


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return (_exact_rotary if case["op"].startswith("rotary") else _exact_muon)(case, s)
