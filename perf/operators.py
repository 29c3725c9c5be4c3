"""The operators of a QLoRA training step that stand outside its 4-bit linears, and what one pass of each costs:

- the AdamW step over a list of adapter tensors, moments in 8 bits (E4M3 codes, one fp32 scale a block of 256,
  stochastic rounding from a seed) or in 32 bits, with clipping by the gradients' global norm;
- the residual step between two blocks, h' = h + alpha gate * norm(y) and x = norm(h'), forward and backward;
- the token embedding with its scale, from a dense or an NF4 table, and the table's gradient.

`run` computes them in elementary torch operations in fp32 (`own` false) or through nf4_quantize_amd (`own` true).
Sizes are those of this repository's weight stack (hidden 4096, key/value 1024, MLP 14336), of its linear workload
(4096 tokens of width 8192) and generic vocabularies."""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 256          # elements that share one scale of the 8-bit moments
E4M3_MAX = 448.0
BETA1, BETA2, EPS, LR, STEP = 0.9, 0.999, 1e-8, 2e-4, 100
MAX_NORM = 0.3
NORM_EPS = 1e-6
# The 16 levels of 4-bit NormalFloat.
NF4 = (-1.0, -0.6961928009986877, -0.5250730514526367, -0.39491748809814453, -0.28444138169288635, -0.18477343022823334,
       -0.09105003625154495, 0.0, 0.07958029955625534, 0.16093020141124725, 0.24611230194568634, 0.33791524171829224,
       0.44070982933044434, 0.5626170039176941, 0.7229568362236023, 1.0)


def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _bytes(name):
    return 2 if name == "bf16" else 4


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one linear's adapter of low rank: the smallest optimizer call, all latency
        dict(name="adamw8_one_adapter", op="adamw", bits=8, hidden=4096, kv=0, mlp=0, layers=1, rank=16, w="bf16", g="bf16", master=False, clip=True),
        # a layer of odd sizes with fp32 adapters and gradients, no clipping: partial blocks everywhere
        dict(name="adamw8_odd_layer", op="adamw", bits=8, hidden=2047, kv=511, mlp=5461, layers=1, rank=13, w="f32", g="f32", master=False, clip=False),
        # every adapter of the 32-layer stack at rank 64: 448 tensors, 168 million parameters, the step a QLoRA run takes
        dict(name="adamw8_stack", op="adamw", bits=8, hidden=4096, kv=1024, mlp=14336, layers=32, rank=64, w="bf16", g="bf16", master=False, clip=True),
        # 8 layers of it with 32-bit moments, fp32 gradients and an fp32 master copy of the bf16 weights
        dict(name="adamw32_master", op="adamw", bits=32, hidden=4096, kv=1024, mlp=14336, layers=8, rank=64, w="bf16", g="f32", master=True, clip=True),
        # one token between two blocks while decoding
        dict(name="norm_fwd_token", op="norm_fwd", rows=1, dim=8192, dtype="bf16", res="bf16", wt="bf16", post=True, gate="channel"),
        # the training batch of the linear workload
        dict(name="norm_fwd_batch", op="norm_fwd", rows=4096, dim=8192, dtype="bf16", res="bf16", wt="bf16", post=True, gate="channel"),
        # its backward pass, with the gradients of both norms' weights and of the gate
        dict(name="norm_bwd_batch", op="norm_bwd", rows=4096, dim=8192, dtype="bf16", res="bf16", wt="f32", post=True, gate="channel"),
        # a ragged batch of odd width, fp32 residual stream, a gate for every token
        dict(name="norm_bwd_odd", op="norm_bwd", rows=1111, dim=2049, dtype="bf16", res="f32", wt="f32", post=False, gate="token"),
        # a decoding batch's tokens from an NF4 table
        dict(name="embed_nf4_decode", op="embed_fwd", tokens=16, vocab=32000, dim=4096, table="nf4", out="bf16"),
        # a long prompt from a large table
        dict(name="embed_fwd_prompt", op="embed_fwd", tokens=16384, vocab=128000, dim=8192, table="bf16", out="bf16"),
        # the dense gradient of a table, text-like (a few tokens are most of the batch)
        dict(name="embed_bwd_dense", op="embed_bwd", tokens=16384, vocab=32000, dim=4096, dtype="bf16", grad="bf16", accumulate=False),
        # a micro-batch added to an fp32 gradient that is already there, odd sizes
        dict(name="embed_bwd_add_odd", op="embed_bwd", tokens=5003, vocab=50021, dim=1601, dtype="bf16", grad="f32", accumulate=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adamw", "adamw", "norm_fwd", "norm_bwd", "embed_fwd", "embed_bwd"])
    if op == "adamw":
        bits = rng.choice([8, 8, 32])
        hidden = _log_int(rng, 64, 8192)
        kv, mlp = rng.choice([(0, 0), (hidden // 4, hidden * 7 // 2), (hidden, hidden * 8 // 3)])
        rank = _log_int(rng, 4, 128)
        layers = _log_int(rng, 1, 32)
        w, g = rng.choice([("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
        while layers > 1 and sum(a * b for a, b in _shapes(dict(hidden=hidden, kv=kv, mlp=mlp, layers=layers, rank=rank))) > (160e6 if bits == 8 and w == g == "bf16" else 40e6):
            layers //= 2
        return dict(op=op, bits=bits, hidden=hidden, kv=kv, mlp=mlp, layers=layers, rank=rank, w=w, g=g,
                    master=w == "bf16" and rng.random() < 0.5, clip=rng.random() < 0.7)
    if op in ("norm_fwd", "norm_bwd"):
        dim = rng.choice([_log_int(rng, 64, 16384), 64 * _log_int(rng, 1, 256)])
        rows = _log_int(rng, 1, max(1, min(16384, 30_000_000 // dim)))
        dtype, res = rng.choice([("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
        return dict(op=op, rows=rows, dim=dim, dtype=dtype, res=res, wt=rng.choice(["f32", dtype]), post=rng.random() < 0.5,
                    gate=rng.choice(["none", "channel", "token"]))
    dim = rng.choice([_log_int(rng, 64, 8192), 64 * _log_int(rng, 1, 128)])
    vocab = _log_int(rng, 256, 131072)
    tokens = _log_int(rng, 1, max(1, min(65536, 130_000_000 // dim)))
    if op == "embed_fwd":
        table = rng.choice(["bf16", "f32", "nf4"])
        if table == "nf4":
            dim = max(64, dim // 64 * 64)
        return dict(op=op, tokens=tokens, vocab=vocab, dim=dim, table=table, out=rng.choice(["bf16", "f32"]))
    vocab = min(vocab, max(256, 260_000_000 // dim))
    return dict(op=op, tokens=tokens, vocab=vocab, dim=dim, dtype=rng.choice(["bf16", "f32"]), grad=rng.choice(["bf16", "f32"]),
                accumulate=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _shapes(c):
    """Adapter tensors [K, r] and [r, N] of each linear: q, k, v, o, gate, up, down (the first alone where kv is 0)."""
    h, kv, mlp, r = c["hidden"], c["kv"], c["mlp"], c["rank"]
    linears = [(h, h), (h, kv), (h, kv), (h, h), (h, mlp), (h, mlp), (mlp, h)] if kv else [(h, h)]
    return [s for _ in range(c["layers"]) for k, n in linears for s in ((k, r), (r, n))]


def _pad(n):
    return -(-n // BLOCK) * BLOCK


def _prepare_adamw(c, seed):
    g = _gen(seed)
    shapes = _shapes(c)
    sizes = [a * b for a, b in shapes]
    starts = [0]
    for n in sizes:
        starts.append(starts[-1] + _pad(n))
    total = starts[-1]
    # every tensor is a view of one buffer, at a multiple of 256 elements; what lies between them stays as it is
    valid = torch.zeros(total, dtype=torch.bool, device=DEV)
    for n, at in zip(sizes, starts):
        valid[at:at + n] = True
    entry = torch.repeat_interleave(torch.arange(len(sizes), device=DEV), torch.tensor([_pad(n) // BLOCK for n in sizes], device=DEV))
    first = torch.tensor(starts[:-1], device=DEV)[entry] // BLOCK
    grad = _randn(g, total)
    grad *= (torch.exp(_randn(g, total // BLOCK, 1)) * 1e-3).expand(-1, BLOCK).reshape(-1)
    grad *= valid
    w = _randn(g, total) * 0.02 * valid
    m = (_randn(g, total) * 0.3 * grad.abs().clamp_min(1e-5)) * valid
    v = (grad.square() * torch.exp(0.5 * _randn(g, total)) + 1e-10) * valid
    s = {"c": c, "n": len(sizes), "valid": valid, "entry": entry, "block_in_entry": torch.arange(total // BLOCK, device=DEV) - first,
         "seed": seed * 7919 + 13}
    # adapters A [K, r] decay, adapters B [r, N] do not and step faster
    s["lr"] = torch.tensor([LR, 2 * LR], device=DEV)[torch.arange(len(sizes), device=DEV) % 2][entry].unsqueeze(1)
    s["wd"] = torch.tensor([0.01, 0.0], device=DEV)[torch.arange(len(sizes), device=DEV) % 2][entry].unsqueeze(1)
    s["w"], s["grad"] = w.to(_dt(c["w"])), grad.to(_dt(c["g"]))
    if c["master"]:
        s["master"] = w
    if c["bits"] == 8:
        for name, x in (("m", m), ("v", v)):
            b = x.view(-1, BLOCK)
            scale = b.abs().amax(1, keepdim=True) * (1.0 / E4M3_MAX)
            s[name] = (b / scale.clamp_min(1e-30)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(-1)
            s[name + "_scale"] = scale.view(-1)
    else:
        s["m"], s["v"] = m, v
    if own:
        import nf4_quantize_amd as nq

        def views(x):
            return [x[at:at + a * b].view(a, b) for (a, b), at in zip(shapes, starts)]

        params, s["grads"] = views(s["w"]), views(s["grad"])
        masters = views(s["master"]) if c["master"] else None
        opt = nq.NF4AdamW([dict(params=params[0::2], lr=LR, weight_decay=0.01, masters=masters and masters[0::2]),
                           dict(params=params[1::2], lr=2 * LR, weight_decay=0.0, masters=masters and masters[1::2])],
                          betas=(BETA1, BETA2), eps=EPS, state_bits=c["bits"], max_grad_norm=MAX_NORM if c["clip"] else 0.0)
        s["grads"] = s["grads"][0::2] + s["grads"][1::2]
        opt.bind_state(*(views_of_state(x, sizes, starts) if x is not None else None
                         for x in (s["m"], s["v"], s.get("m_scale"), s.get("v_scale"))))
        s["opt"] = opt
    return s


def views_of_state(x, sizes, starts):
    """The optimizer's order of the tensors' parts of a state buffer: the first group's, then the second's."""
    per = BLOCK if x.dtype == torch.float32 and x.numel() * BLOCK == starts[-1] else 1
    parts = [x[at // per:at // per + -(-n // per)] for n, at in zip(sizes, starts)]
    return parts[0::2] + parts[1::2]


def _prepare_norm(c, seed):
    g = _gen(seed)
    t, d = c["rows"], c["dim"]
    dtype, res, wt = _dt(c["dtype"]), _dt(c["res"]), _dt(c["wt"])
    channel = torch.exp(0.4 * _randn(g, d))  # some channels carry more than others
    s = {"c": c, "alpha": 0.7071}
    s["y"] = (_randn(g, t, d) * channel * 3.0).to(dtype)
    s["w_pre"] = (1 + 0.2 * _randn(g, d)).to(wt)
    s["w_post"] = (1 + 0.2 * _randn(g, d)).to(wt) if c["post"] else None
    s["gate"] = (0.5 + 0.2 * _randn(g, d)).to(wt) if c["gate"] == "channel" else torch.sigmoid(_randn(g, t, d)).to(dtype) if c["gate"] == "token" else None
    s["h"] = (_randn(g, t, d) * channel * 1.5).to(res)  # the residual stream: before the step, or (backward) after it
    if c["op"] == "norm_bwd":
        s["dx"], s["dh_out"] = _randn(g, t, d).to(dtype), (0.5 * _randn(g, t, d)).to(res)
        s["rstd_pre"] = torch.rsqrt(s["h"].double().square().mean(1) + NORM_EPS).float()
        s["rstd_post"] = torch.rsqrt(s["y"].double().square().mean(1) + NORM_EPS).float() if c["post"] else None
    return s


def _zipf(vocab):
    return 1.0 / (torch.arange(vocab, dtype=torch.float64) + 2.7)


def _tokens(c, g):
    """Token numbers as text has them: a few make up most of the batch, in a shuffled vocabulary; some places are empty (-1)."""
    cdf = torch.cumsum(_zipf(c["vocab"]), 0).to(DEV)
    rank = torch.searchsorted(cdf, torch.rand(c["tokens"], generator=g, device=DEV, dtype=torch.float64) * cdf[-1]).clamp_max(c["vocab"] - 1)
    ids = torch.randperm(c["vocab"], generator=g, device=DEV)[rank]
    if c["op"] == "embed_bwd":
        ids[torch.rand(c["tokens"], generator=g, device=DEV) < 0.02] = -1
    return ids


def _prepare_embed(c, seed):
    g = _gen(seed)
    v, d = c["vocab"], c["dim"]
    s = {"c": c, "scale": math.sqrt(d), "ids": _tokens(c, g)}
    if c["op"] == "embed_bwd":
        s["dy"] = (_randn(g, c["tokens"], d) * 1e-2).to(_dt(c["dtype"]))
        if c["accumulate"]:
            s["grad"] = _randn(g, v, d).to(_dt(c["grad"]))
        return s
    if c["table"] != "nf4":
        s["table"] = torch.empty(v, d, dtype=_dt(c["table"]), device=DEV).normal_(0, 0.02, generator=g)
        return s
    n = v * d
    s["codes"] = torch.randint(0, 256, (n // 2,), generator=g, device=DEV, dtype=torch.uint8)
    s["absmax_q"] = torch.randint(0x60, 0x7F, (n // 64,), generator=g, device=DEV, dtype=torch.uint8)
    s["absmax_scale"] = torch.rand(-(-n // 16384), generator=g, device=DEV) * 1e-4 + 1e-4
    s["levels"] = torch.tensor(NF4, device=DEV)
    if own:
        import nf4_quantize_amd as nq

        s["table"] = nq.NF4Tensor(s["codes"], None, s["absmax_q"], s["absmax_scale"], (v, d))
    return s


def prepare(case, seed):
    kind = case["op"].split("_")[0]
    return {"adamw": _prepare_adamw, "norm": _prepare_norm, "embed": _prepare_embed}[kind](case, seed)


# ------------------------------------------------------------------ plain forms

def _mix(x):
    """32 bits mixed by two rounds of shift, exclusive or and product (the fractions of the roots of 2 and 3)."""
    x = (x ^ (x >> 16)) * 0x6A09E667 & 0xFFFFFFFF
    x = (x ^ (x >> 15)) * 0xBB67AE85 & 0xFFFFFFFF
    return x ^ (x >> 16)


def _random_bits(s):
    """32 random bits for every element, from the seed, the tensor's place in the list and the element's in the tensor."""
    seed = s["seed"]
    # the optimizer's list: the A adapters first, then the B adapters
    place = s["entry"] // 2 + (s["entry"] % 2) * ((s["n"] + 1) // 2)
    key = _mix((_mix(place * 0x9E3779B9 + (seed >> 32) & 0xFFFFFFFF) + seed) & 0xFFFFFFFF)
    i = s["block_in_entry"].unsqueeze(1) * BLOCK + torch.arange(BLOCK, device=DEV)
    return _mix(i * 0x9E3779B9 + key.unsqueeze(1) & 0xFFFFFFFF)


def _to_e4m3(t, r20):
    """E4M3 codes of t in [-448, 448], rounded away from zero where the 20 random bits carry."""
    a = t.abs()
    small = a < 2.0 ** -6
    bits = torch.where(small, a + 2.0 ** -6, a).view(torch.int32)
    code = ((bits + r20) >> 20) - torch.where(small, 968, 960)
    return torch.where(t < 0, code + 128, code).to(torch.uint8)


def _stored(x, r20, floor):
    """(codes, scales) of the 8-bit storage of x [blocks, 256]."""
    scale = x.abs().amax(1, keepdim=True) * (1.0 / E4M3_MAX)
    scale = torch.where(scale < 2.0 ** -126, 0.0, scale)
    t = x * torch.where(scale > 0, 1.0 / scale, 0.0)
    t = t.clamp(2.0 ** -9, E4M3_MAX) if floor else t.clamp(-E4M3_MAX, E4M3_MAX)
    return _to_e4m3(t, r20), scale


def _plain_adamw(s):
    c = s["c"]
    g = s["grad"].float().view(-1, BLOCK)
    valid = s["valid"].view(-1, BLOCK)
    out = {}
    if c["clip"]:
        norm = g.double().square().sum().sqrt().float()
        out["grad_norm"] = norm.view(1)
        g = g * torch.where(norm > MAX_NORM, MAX_NORM / norm, 1.0)
    w = (s["master"] if c["master"] else s["w"].float()).view(-1, BLOCK)
    m, v = s["m"].float().view(-1, BLOCK), s["v"].float().view(-1, BLOCK)
    if c["bits"] == 8:
        m, v = m * s["m_scale"].unsqueeze(1), v * s["v_scale"].unsqueeze(1)
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * (g * g)
    w = w * (1 - s["lr"] * s["wd"]) - s["lr"] / (1 - BETA1 ** STEP) * m / ((v * (1 / (1 - BETA2 ** STEP))).sqrt() + EPS)
    if c["bits"] == 8:
        r = _random_bits(s)
        for name, x, r20 in (("m", m, (r >> 16) << 4), ("v", v, (r & 0xFFFF) << 4)):
            code, scale = _stored(x, r20.int(), name == "v")
            old = s[name].view(torch.uint8).view(-1, BLOCK)
            s[name] = torch.where(valid, code, old).view(torch.float8_e4m3fn).view(-1)
            s[name + "_scale"] = scale.view(-1)
            out[name + "_scale"] = s[name + "_scale"]
    else:
        s["m"], s["v"] = m.view(-1), v.view(-1)
    out["m"], out["v"] = s["m"], s["v"]
    if c["master"]:
        s["master"] = out["master"] = w.view(-1)
    s["w"] = out["w"] = w.view(-1).to(_dt(c["w"]))
    return out


def _plain_norm_fwd(s):
    z = s["y"].float()
    r = {}
    if s["w_post"] is not None:
        r["rstd_post"] = torch.rsqrt((z * z).mean(1) + NORM_EPS)
        z = z * r["rstd_post"].unsqueeze(1) * s["w_post"].float()
    if s["gate"] is not None:
        z = z * s["gate"].float()
    h = s["h"].float() + s["alpha"] * z
    r["rstd_pre"] = torch.rsqrt((h * h).mean(1) + NORM_EPS)
    r["x"] = (h * r["rstd_pre"].unsqueeze(1) * s["w_pre"].float()).to(s["y"].dtype)
    r["h"] = h.to(s["h"].dtype)
    return r


def _plain_norm_bwd(s):
    c = s["c"]
    dtype, wt = _dt(c["dtype"]), _dt(c["wt"])
    dx, w1, r1 = s["dx"].float(), s["w_pre"].float(), s["rstd_pre"].unsqueeze(1)
    n1 = s["h"].float() * r1
    p = dx * w1
    dh = s["dh_out"].float() + r1 * (p - n1 * (p * n1).mean(1, keepdim=True))
    out = {"dw_pre": (dx * n1).sum(0).to(wt), "dh": dh.to(s["h"].dtype)}
    dz = s["alpha"] * dh
    z = n2 = s["y"].float()
    if c["post"]:
        r2, w2 = s["rstd_post"].unsqueeze(1), s["w_post"].float()
        n2 = z * r2
        z = n2 * w2
    if s["gate"] is not None:
        dgate = dz * z
        out["dgate"] = dgate.sum(0).to(wt) if c["gate"] == "channel" else dgate.to(dtype)
        dz = dz * s["gate"].float()
    if c["post"]:
        out["dw_post"] = (dz * n2).sum(0).to(wt)
        p = dz * w2
        dz = r2 * (p - n2 * (p * n2).mean(1, keepdim=True))
    out["dy"] = dz.to(dtype)
    return out


def _plain_embed_fwd(s):
    c = s["c"]
    if c["table"] != "nf4":
        return (s["table"][s["ids"]].float() * s["scale"]).to(_dt(c["out"]))
    d = c["dim"]
    b = s["codes"].view(-1, d // 2)[s["ids"]]
    q = s["levels"][torch.stack((b & 15, b >> 4), 2).view(-1, d).int()]
    block = s["ids"].unsqueeze(1) * (d // 64) + torch.arange(d // 64, device=DEV)
    scale = s["absmax_q"][block].view(torch.float8_e4m3fn).float() * s["absmax_scale"][block // 256]
    return ((q.view(-1, d // 64, 64) * scale.unsqueeze(2)).view(-1, d) * s["scale"]).to(_dt(c["out"]))


def _plain_embed_bwd(s):
    c = s["c"]
    live = s["ids"] >= 0
    rows = torch.where(live.unsqueeze(1), s["dy"].float() * s["scale"], 0.0)
    grad = torch.zeros(c["vocab"], c["dim"], device=DEV).index_add_(0, s["ids"].clamp_min(0), rows)
    if c["accumulate"]:
        s["grad"] = (s["grad"].float() + grad).to(_dt(c["grad"]))
        return s["grad"]
    return grad.to(_dt(c["grad"]))


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["c"]["op"]
    if not own:
        return {"adamw": _plain_adamw, "norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd,
                "embed_fwd": _plain_embed_fwd, "embed_bwd": _plain_embed_bwd}[op](state)
    import nf4_quantize_amd as nq

    s, c = state, state["c"]
    if op == "adamw":
        s["opt"].step(s["grads"], step=STEP, seed=s["seed"])
        out = {k: s[k] for k in ("w", "m", "v", "master", "m_scale", "v_scale") if k in s}
        if c["clip"]:
            out["grad_norm"] = s["opt"].grad_norm
        return out
    if op == "norm_fwd":
        h, x, rstd_pre, rstd_post = nq.residual_norm_forward(s["y"], s["h"], s["w_pre"], s["w_post"], s["gate"], alpha=s["alpha"], eps=NORM_EPS)
        out = {"h": h, "x": x, "rstd_pre": rstd_pre}
        return out if rstd_post is None else {**out, "rstd_post": rstd_post}
    if op == "norm_bwd":
        names = ("dy", "dh", "dw_pre", "dw_post", "dgate")
        got = nq.residual_norm_backward(s["dx"], s["dh_out"], s["y"], s["h"], s["rstd_pre"], s["w_pre"], s["rstd_post"], s["w_post"], s["gate"], alpha=s["alpha"])
        return {k: x for k, x in zip(names, got) if x is not None}
    if op == "embed_fwd":
        return nq.embedding_forward(s["ids"], s["table"], scale=s["scale"], out_dtype=_dt(c["out"]))
    return nq.embedding_backward(s["ids"], s["dy"], c["vocab"], scale=s["scale"], grad=s.get("grad"), grad_dtype=_dt(c["grad"]))


# ------------------------------------------------------------------ the floor

def _distinct(c):
    """The rows that a batch of tokens touches, on the average."""
    p = _zipf(c["vocab"])
    return float((1 - (1 - p / p.sum()) ** c["tokens"]).sum())


def work(case):
    c = case
    if c["op"] == "adamw":
        n = sum(a * b for a, b in _shapes(c))
        state = 4 * (1 + 4 / BLOCK) if c["bits"] == 8 else 16
        w = _bytes(c["w"]) * (1 if c["master"] else 2) + (8 if c["master"] else 0)
        return {"bytes": n * (w + _bytes(c["g"]) + state), "flops": n * 20}
    if c["op"].startswith("norm"):
        n, a, r = c["rows"] * c["dim"], _bytes(c["dtype"]), _bytes(c["res"])
        token = a if c["gate"] == "token" else 0
        if c["op"] == "norm_fwd":
            return {"bytes": n * (2 * a + 2 * r + token), "flops": n * 10}
        return {"bytes": n * (3 * a + 3 * r + 2 * token), "flops": n * 22}
    rows = _distinct(c)
    if c["op"] == "embed_fwd":
        row = c["dim"] * (33 / 64 if c["table"] == "nf4" else _bytes(c["table"]))
        return {"bytes": c["tokens"] * 8 + rows * row + c["tokens"] * c["dim"] * _bytes(c["out"]), "flops": c["tokens"] * c["dim"]}
    table = 2 * rows if c["accumulate"] else c["vocab"]
    return {"bytes": c["tokens"] * (8 + c["dim"] * _bytes(c["dtype"])) + table * c["dim"] * _bytes(c["grad"]), "flops": 2 * c["tokens"] * c["dim"]}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_e4m3(t, frac):
    """E4M3 values around t, the upper one where the fraction of the step plus `frac` in [0, 1) reaches one."""
    a = t.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -6))) - 3)
    return torch.sign(t) * torch.floor(a / step + frac) * step


def _exact_adamw(c, s):
    f8 = c["bits"] == 8
    g, valid = s["grad"].double(), s["valid"]
    out = {}
    if c["clip"]:
        norm = (g * g).sum().sqrt()
        out["grad_norm"] = norm.view(1)
        g = g * min(1.0, MAX_NORM / float(norm))
    old = {k: s[k].double() for k in ("m", "v")}
    per = {k: (s[k + "_scale"].double().repeat_interleave(BLOCK) if f8 else 1.0) for k in ("m", "v")}
    new = {"m": BETA1 * (old["m"] * per["m"]) + (1 - BETA1) * g, "v": BETA2 * (old["v"] * per["v"]) + (1 - BETA2) * g ** 2}
    hat_m, hat_v = new["m"] / (1 - BETA1 ** STEP), new["v"] / (1 - BETA2 ** STEP)
    odd = (s["entry"] % 2).repeat_interleave(BLOCK)
    lr = torch.where(odd == 1, 2 * LR, LR).double()
    w = (s["master"] if c["master"] else s["w"]).double()
    w = w - lr * torch.where(odd == 1, 0.0, 0.01) * w - lr * hat_m / (hat_v.sqrt() + EPS)
    out["w"] = w
    if c["master"]:
        out["master"] = w
    if not f8:
        return {**out, **new}
    bits = _random_bits(s).view(-1)
    for k, r in (("m", bits >> 16), ("v", bits & 0xFFFF)):
        scale = new[k].view(-1, BLOCK).abs().amax(1) / E4M3_MAX
        t = new[k] / scale.repeat_interleave(BLOCK).clamp_min(1e-300)
        t = t.clamp_min(2.0 ** -9) if k == "v" else t
        out[k] = torch.where(valid, _exact_e4m3(t, r.double() / 65536), old[k])
        out[k + "_scale"] = scale
    return out


def _exact_norm(c, s):
    def f64(k):
        return None if s.get(k) is None else s[k].double()

    y, h, w1, w2, gate, alpha = f64("y"), f64("h"), f64("w_pre"), f64("w_post"), f64("gate"), s["alpha"]
    gate = 1.0 if gate is None else gate
    if c["op"] == "norm_fwd":
        out = {}
        z = y
        if c["post"]:
            out["rstd_post"] = 1 / (y.pow(2).mean(1) + NORM_EPS).sqrt()
            z = y * out["rstd_post"][:, None] * w2
        out["h"] = h + alpha * gate * z
        out["rstd_pre"] = 1 / (out["h"].pow(2).mean(1) + NORM_EPS).sqrt()
        out["x"] = out["h"] * out["rstd_pre"][:, None] * w1
        return out
    # the norms' gradients by the product rule on n = a (a.a / D + eps)^(-1/2)
    def through(a, r, dn):
        return r[:, None] * dn - a * (r ** 3 / c["dim"] * (dn * a).sum(1))[:, None]

    dx, r1 = f64("dx"), f64("rstd_pre")
    out = {"dw_pre": (dx * h * r1[:, None]).sum(0)}
    dh = out["dh"] = f64("dh_out") + through(h, r1, dx * w1)
    r2 = f64("rstd_post")
    n2 = y * r2[:, None] if c["post"] else y
    z = n2 * w2 if c["post"] else y
    if c["gate"] != "none":
        out["dgate"] = (alpha * dh * z).sum(0) if c["gate"] == "channel" else alpha * dh * z
    dz = alpha * dh * gate
    if c["post"]:
        out["dw_post"] = (dz * n2).sum(0)
        dz = through(y, r2, dz * w2)
    out["dy"] = dz
    return out


def _exact_embed(c, s):
    ids = s["ids"]
    if c["op"] == "embed_bwd":
        grad = s["grad"].double() if c["accumulate"] else torch.zeros(c["vocab"], c["dim"], dtype=torch.float64, device=DEV)
        live = torch.nonzero(ids >= 0).view(-1)
        return grad.index_put_((ids[live],), s["dy"][live].double() * s["scale"], accumulate=True)
    if c["table"] != "nf4":
        return s["table"][ids].double() * s["scale"]
    d = c["dim"]
    at = ids[:, None] * d + torch.arange(d, device=DEV)
    code = (s["codes"][at // 2].int() >> (4 * (at % 2))) & 15
    e = s["absmax_q"][at // 64].double()
    e4m3 = torch.where(e < 8, e / 512, torch.exp2(torch.floor(e / 8) - 7) * (1 + torch.remainder(e, 8) / 8))
    return s["levels"].double()[code] * e4m3 * s["absmax_scale"][at // 16384].double() * s["scale"]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    kind = case["op"].split("_")[0]
    return {"adamw": _exact_adamw, "norm": _exact_norm, "embed": _exact_embed}[kind](case, s)
