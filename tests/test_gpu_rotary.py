"""Rotation of queries and keys with their heads' norms against the formulas in 64
bits: forward, backward and the autograd function.

Tolerances. u = 2^-24. Cosine and sine are off by 2^-24 of their own rounding, 3e-9 of the polynomial and the
phase's 32 bits, below 4 u in all; products, sums and the norm (a sum of up to 512 squares in a tree after 16 of a
lane, a root, a quotient) add a few u each: 16 u of the pair's |a| + |b| covers a forward value, and the output's
half step is relative. The backward pass has one more sum of the same kind: 32 u of the terms' magnitudes. The sums
of the weights' gradients add up to a thousand rows after a few of a lane: 64 u of the sum of the terms' magnitudes."""
import math

import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def half_step(dt):
    import torch

    return torch.finfo(dt).eps / 2


def gen(dev, seed):
    import torch

    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return g


def make(dev, seed, lead, heads, dim, dt, order):
    """[*lead x heads x dim] values in an order in memory; "fused": with values before and behind every token's."""
    import torch

    g = gen(dev, seed)
    x = torch.randn(*lead, heads, dim, generator=g, device=dev) * torch.exp(0.5 * torch.randn(dim, generator=g, device=dev))
    x = x.to(dt)
    if order == "head":
        return x.transpose(-3, -2).contiguous().transpose(-3, -2)
    if order == "fused":
        wide = torch.full((*lead, heads + 3, dim), 7.0, dtype=dt, device=dev)
        wide[..., 1:1 + heads, :] = x
        return wide[..., 1:1 + heads, :]
    return x


def turn(x, cos, sin, rope):
    """The rotation in 64 bits, and of |x| with |cos| and |sin| (the terms' magnitudes)."""
    r = rope.dim
    a, b = ((x[..., :r // 2], x[..., r // 2:r]) if rope.layout == "half" else (x[..., 0:r:2], x[..., 1:r:2]))
    y = x.clone()
    one, two = a * cos - b * sin, b * cos + a * sin
    if rope.layout == "half":
        y[..., :r // 2], y[..., r // 2:r] = one, two
    else:
        y[..., 0:r:2], y[..., 1:r:2] = one, two
    return y


def angles(positions, lead, rope, dev):
    """cos and sin in 64 bits from the angle reduced in integers, |cos| + |sin| bounds the magnitude."""
    import torch

    at = torch.arange(lead[-1], device=dev).expand(lead) if positions is None else positions.long().expand(lead)
    f = torch.tensor(rope.frequencies, dtype=torch.float64, device=dev)
    angle = at.double().unsqueeze(-1) * f
    return torch.cos(angle).unsqueeze(-2) * rope.scale, torch.sin(angle).unsqueeze(-2) * rope.scale


def normed(x, w, eps, off):
    if w is None:
        return x
    return x * (x.pow(2).mean(-1, keepdim=True) + eps).rsqrt() * (w.double() + off)


def check(got, want, size, steps, dt, what):
    tol = steps * U * size + half_step(dt) * want.abs() + 1e-30
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}, worst {((got.double() - want).abs() / tol).max():.2f}"


def spread(y, rope):
    """|a| + |b| of every pair at both its places: the magnitude of a turned value's terms."""
    import torch

    one = torch.ones((), dtype=y.dtype, device=y.device)
    return turn_abs(y.abs(), rope) * max(1.0, abs(rope.scale)) * one


def turn_abs(x, rope):
    r = rope.dim
    y = x.clone()
    if rope.layout == "half":
        s = x[..., :r // 2] + x[..., r // 2:r]
        y[..., :r // 2], y[..., r // 2:r] = s, s
    else:
        s = x[..., 0:r:2] + x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = s, s
    return y


def reference_backward(dy, x, w, cos, sin, rope, eps, off):
    """(dx, its terms' magnitude, dw, its terms' magnitude)."""
    g = turn(dy, cos, -sin, rope)
    size = spread(dy, rope)
    if w is None:
        return g, size, None, None
    d = x.shape[-1]
    r = (x.pow(2).mean(-1, keepdim=True) + eps).rsqrt()
    n, wp = x * r, w.double() + off
    lead = tuple(range(x.dim() - 1))
    dx = r * (g * wp - n * (g * wp * n).sum(-1, keepdim=True) / d)
    big = r * (size * wp.abs() + n.abs() * (size * wp.abs() * n.abs()).sum(-1, keepdim=True) / d)
    return dx, big, (g * n).sum(lead), (size * n.abs()).sum(lead)


# dim, rotated, layout, dtype, w dtype, heads of queries, of keys, lead, order, positions, norm of (q, k), scaling
CASES = [
    # whole vectors: 16 bytes, 8, 4 and one element; one and several units a lane
    (128, 128, "half", "bf16", "bf16", 32, 8, (2, 5), "token", "far", "qk", None),
    (128, 128, "interleaved", "bf16", "f32", 8, 8, (9,), "head", "packed", "qk", None),
    (64, 32, "half", "f32", "f32", 3, 1, (3, 7), "token", "start", "qk", "yarn"),
    (64, 64, "half", "f32", "f32", 5, 2, (2, 3), "fused", "shared", "", None),
    (80, 20, "interleaved", "bf16", "bf16", 7, 1, (2, 11), "head", "packed", "qk", "linear"),
    (80, 24, "half", "bf16", "f32", 7, 1, (2, 11), "head", "packed", "k", None),
    (96, 8, "half", "bf16", "bf16", 1, 1, (4, 1), "token", "far", "q", None),
    (72, 36, "half", "bf16", "bf16", 6, 3, (2, 5), "fused", "start", "qk", None),
    (72, 36, "interleaved", "f32", "f32", 6, 3, (2, 5), "fused", "start", "qk", "ntk"),
    (75, 38, "half", "f32", "f32", 5, 3, (3, 4), "fused", "packed", "qk", None),
    (75, 38, "interleaved", "bf16", "f32", 5, 3, (3, 4), "token", "packed", "qk", None),
    (512, 512, "half", "bf16", "bf16", 3, 2, (1, 3), "token", "far", "qk", None),
    (512, 256, "interleaved", "f32", "f32", 3, 0, (5,), "head", "start", "q", None),
    (511, 510, "half", "bf16", "f32", 2, 1, (2, 2), "token", "far", "qk", None),
    (511, 2, "interleaved", "f32", "f32", 2, 1, (2, 2), "fused", "start", "qk", None),
    (510, 510, "half", "f32", "f32", 1, 1, (3,), "token", "start", "qk", None),
    (508, 500, "half", "bf16", "bf16", 2, 1, (3,), "token", "start", "qk", None),
    (200, 196, "half", "f32", "f32", 2, 1, (3,), "token", "start", "qk", None),
    (260, 260, "interleaved", "f32", "bf16", 2, 1, (3,), "head", "start", "qk", None),
    (2, 2, "half", "f32", "f32", 3, 2, (2, 3), "token", "far", "qk", None),
    (3, 2, "interleaved", "bf16", "bf16", 3, 2, (2, 3), "token", "far", "qk", None),
    (16, 16, "half", "bf16", "bf16", 65, 33, (1, 1), "token", "far", "qk", None),
    # many tokens: a wave takes whole tokens, workgroups several
    (64, 64, "half", "bf16", "bf16", 3, 1, (2, 4099), "token", "packed", "qk", "wavelength"),
    (32, 32, "interleaved", "f32", "f32", 1, 1, (17000,), "token", "start", "qk", None),
    (16, 8, "half", "f32", "f32", 1, 0, (3, 30011), "head", "packed", "q", None),
]


def case(dev, c, seed=0):
    import torch

    import nf4_quantize_amd as nq

    dim, rot, layout, dt, wt, hq, hk, lead, order, kind, norm, scaling = c
    dt, wt = (torch.bfloat16 if n == "bf16" else torch.float32 for n in (dt, wt))
    full = {None: None, "linear": dict(kind="linear", factor=4), "ntk": dict(kind="ntk", factor=4),
            "yarn": dict(kind="yarn", factor=8, length=64), "wavelength": dict(kind="wavelength", factor=8, length=64)}
    rope = nq.NF4Rotary(rot, layout=layout, scaling=full[scaling], device=dev)
    g = gen(dev, seed + 1)
    positions = None
    if kind == "far":
        positions = torch.randint(0, 1 << 20, (*lead[:-1], 1), generator=g, device=dev) + torch.arange(lead[-1], device=dev)
    elif kind == "packed":
        positions = torch.randint(0, 5000, lead, generator=g, device=dev, dtype=torch.int32)
    elif kind == "shared":
        positions = torch.arange(lead[-1], device=dev, dtype=torch.int32) * 3 - 4
    q = make(dev, seed + 2, lead, hq, dim, dt, order)
    k = make(dev, seed + 3, lead, hk, dim, dt, order) if hk else None
    w = {n: (1 + 0.3 * torch.randn(dim, generator=g, device=dev)).to(wt) if n in norm else None for n in "qk"}
    if k is None:
        w["k"] = None
    return rope, positions, q, k, w["q"], w["k"], lead


@pytest.mark.parametrize("c", CASES, ids=lambda c: "-".join(map(str, c[:9])).replace(" ", ""))
def test_forward(dev, c):
    import nf4_quantize_amd as nq

    rope, positions, q, k, w_q, w_k, lead = case(dev, c)
    off = 0.25 if c[0] % 4 == 0 else 0.0
    got = nq.rotary_forward(q, k, positions, rope, w_q, w_k, eps=1e-5, w_offset=off)
    cos, sin = angles(positions, lead, rope, dev)
    for x, w, y, name in ((q, w_q, got[0], "q"), (k, w_k, got[1], "k")):
        if x is None:
            assert y is None
            continue
        n = normed(x.double(), w, 1e-5, off)
        assert y.dtype == x.dtype and y.shape == x.shape
        check(y, turn(n, cos, sin, rope), spread(n, rope), 16, x.dtype, name)


@pytest.mark.parametrize("c", CASES, ids=lambda c: "-".join(map(str, c[:9])).replace(" ", ""))
def test_backward(dev, c):
    import nf4_quantize_amd as nq

    rope, positions, q, k, w_q, w_k, lead = case(dev, c)
    order = "head" if c[8] == "token" else "token"
    dq_out = make(dev, 11, lead, q.shape[-2], c[0], q.dtype, order)
    dk_out = None if k is None else make(dev, 12, lead, k.shape[-2], c[0], q.dtype, order)
    dq, dk, dw_q, dw_k = nq.rotary_backward(dq_out, dk_out, positions, rope, q, k, w_q, w_k, eps=1e-5, w_offset=0.1)
    again = nq.rotary_backward(dq_out, dk_out, positions, rope, q, k, w_q, w_k, eps=1e-5, w_offset=0.1)
    cos, sin = angles(positions, lead, rope, dev)
    for dy, x, w, dx, dw, other, name in ((dq_out, q, w_q, dq, dw_q, again[2], "q"), (dk_out, k, w_k, dk, dw_k, again[3], "k")):
        if dy is None:
            assert dx is None and dw is None
            continue
        want, big, dw_want, dw_big = reference_backward(dy.double(), x.double(), w, cos, sin, rope, 1e-5, 0.1)
        check(dx, want, big, 32, dx.dtype, "d" + name)
        if w is None:
            assert dw is None
        else:
            assert dw.dtype == w.dtype and bool((dw == other).all())  # the same bits each time
            check(dw, dw_want, dw_big, 64, dw.dtype, "dw_" + name)


def test_far_and_negative_positions(dev):
    """The angle is reduced in integers: at any int64 position it is exact to 2^-65 turns a position."""
    import torch
    from fractions import Fraction

    import nf4_quantize_amd as nq
    from nf4_quantize_amd.heads import TWO_PI

    rope = nq.NF4Rotary(16, layout="half", device=dev)
    at = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 40 + 12345, -3 * 2 ** 45]
    q = torch.zeros(len(at), 1, 16, device=dev)
    q[..., :8] = 1.0
    y, _ = nq.rotary_forward(q, None, torch.tensor(at, device=dev), rope)
    y = y[:, 0].double().cpu()
    for i, p in enumerate(at):
        for j, f in enumerate(rope.frequencies):
            rest = float((Fraction(p) * Fraction(f) / TWO_PI) % 1) * 2 * math.pi
            tol = 4 * U + abs(p) * 2.0 ** -65 * 2 * math.pi
            assert abs(y[i, j].item() - math.cos(rest)) <= tol and abs(y[i, 8 + j].item() - math.sin(rest)) <= tol


@pytest.mark.parametrize("norm", [False, True])
def test_in_place_and_given_outputs(dev, norm):
    """Slices of one projection's rows, in place: what lies beside them stays."""
    import torch

    import nf4_quantize_amd as nq

    g = gen(dev, 3)
    rows = torch.randn(2, 9, 8, 64, generator=g, device=dev).bfloat16()
    w = torch.rand(64, generator=g, device=dev) + 0.5 if norm else None
    rope = nq.NF4Rotary(64, device=dev)
    q, k = rows[:, :, :4], rows[:, :, 4:6]
    want = nq.rotary_forward(q, k, None, rope, w, w)
    keep = rows.clone()
    got = nq.rotary_forward(q, k, None, rope, w, w, q_out=q, k_out=k)
    assert got[0].data_ptr() == rows.data_ptr()
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(rows[:, :, 6:], keep[:, :, 6:])
    wide = torch.full((2, 4 + 3, 9, 70), -5.0, device=dev).bfloat16()
    rows.copy_(keep)
    nq.rotary_forward(q, k, None, rope, w, w, q_out=wide[:, 1:5, :, 4:68].transpose(1, 2))
    assert torch.equal(wide[:, 1:5, :, 4:68].transpose(1, 2), want[0])
    wide[:, 1:5, :, 4:68] = -5.0
    assert bool((wide == -5.0).all())


def test_refusals(dev):
    import torch

    import nf4_quantize_amd as nq

    rope = nq.NF4Rotary(64, device=dev)
    x = torch.randn(3, 6, 64, device=dev)
    q, k, w = x[:, :4], x[:, 4:], torch.ones(64, device=dev)
    bad = [
        dict(q=q.transpose(1, 2)), dict(q=q.bfloat16()), dict(k=k[:2]), dict(k=k[..., :32]), dict(q=q[0]),
        dict(rope=nq.NF4Rotary(128, device=dev)), dict(w_q=w[:32]), dict(w_q=w.bfloat16(), w_k=w), dict(w_k=w, k=None),
        dict(w_q=torch.ones(128, device=dev)[::2]), dict(positions=torch.zeros(2, dtype=torch.int32, device=dev)),
        dict(positions=torch.zeros(6, dtype=torch.int32, device=dev)[::2]), dict(positions=torch.zeros(3, dtype=torch.int32)),
        dict(q_out=x[:, 1:5]), dict(q_out=x[:, 2:6]), dict(k_out=q[:, :2]), dict(q_out=torch.empty(64, device=dev).expand(3, 4, 64)),
        dict(q_out=torch.empty(3, 3, 64, device=dev)), dict(q_out=torch.empty(3, 4, 64, device=dev).bfloat16()),
        dict(w_q=x.view(-1)[64:128], q_out=q), dict(rope=nq.NF4Rotary(64, device="cpu")),
    ]
    for b in bad:
        a = dict(q=q, k=k, positions=None, rope=rope, w_q=None, w_k=None)
        a.update(b)
        with pytest.raises((ValueError, TypeError)):
            nq.rotary_forward(**a)
    with pytest.raises(TypeError):
        nq.rotary_forward(q, k, torch.zeros(3, device=dev), rope)
    both = torch.empty(3, 6, 64, device=dev)
    with pytest.raises(ValueError, match="share"):
        nq.rotary_forward(q, k, None, rope, q_out=both[:, :4], k_out=both[:, 3:5])
    with pytest.raises(ValueError):
        nq.rotary_backward(q, k, None, rope, None, None, w, w)
    with pytest.raises(ValueError):
        nq.rotary_backward(None, k, None, rope, q, k, w, w)


@pytest.mark.parametrize("lead", [(0,), (2, 0), (0, 3)])
def test_no_tokens(dev, lead):
    import torch

    import nf4_quantize_amd as nq

    rope, w = nq.NF4Rotary(8, device=dev), torch.ones(8, device=dev)
    q, k = torch.empty(*lead, 2, 8, device=dev), torch.empty(*lead, 1, 8, device=dev)
    assert nq.rotary_forward(q, k, None, rope, w, w)[0].shape == q.shape
    dq, dk, dw_q, dw_k = nq.rotary_backward(q, k, None, rope, q, k, w, w)
    assert dq.shape == q.shape and not dw_q.any() and not dw_k.any()


def test_non_finite_rows_stay_apart(dev):
    """A head with NaN or infinity leaves the others, and rows of zeros are zeros with eps > 0."""
    import torch

    import nf4_quantize_amd as nq

    rope, w = nq.NF4Rotary(32, device=dev), torch.ones(32, device=dev)
    q = torch.randn(5, 4, 32, device=dev)
    want, _ = nq.rotary_forward(q, None, None, rope, w)
    bad = q.clone()
    bad[1, 2, 3], bad[3, 0, 31] = float("nan"), float("inf")
    bad[4, 1] = 0.0
    got, _ = nq.rotary_forward(bad, None, None, rope, w)
    live = torch.ones(5, 4, dtype=torch.bool, device=dev)
    live[1, 2] = live[3, 0] = live[4, 1] = False
    assert torch.equal(got[live], want[live]) and not got[4, 1].any() and bool(torch.isnan(got[1, 2]).all())


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("norm", ["", "q", "qk"])
def test_autograd(dev, layout, norm):
    """Gradients of the function against torch's of the formulas in 64 bits, and against differences."""
    import torch

    import nf4_quantize_amd as nq

    g = gen(dev, 7)
    rope = nq.NF4Rotary(24, layout=layout, device=dev)
    at = torch.randint(0, 100, (2, 5), generator=g, device=dev)
    q, k = (torch.randn(2, 5, n, 40, generator=g, device=dev, requires_grad=True) for n in (4, 2))
    w = [(torch.rand(40, generator=g, device=dev) + 0.5).requires_grad_() if n in norm else None for n in "qk"]
    leaves = [t for t in (q, k, *w) if t is not None]
    a, b = (torch.randn(2, 5, n, 40, generator=g, device=dev) for n in (4, 2))

    def loss(q, k, w_q, w_k):
        y, z = nq.rotary(q, k, at, rope, w_q, w_k, eps=1e-5)
        return (y.double() * a).sum() + (z.double() * b).sum()

    got = torch.autograd.grad(loss(q, k, *w), leaves)
    cos, sin = angles(at, (2, 5), rope, dev)
    leaves64 = [t.detach().double().requires_grad_() for t in leaves]
    q64, k64 = leaves64[:2]
    rest = iter(leaves64[2:])
    w64 = [None if t is None else next(rest) for t in w]
    plain = (turn(normed(q64, w64[0], 1e-5, 0.0), cos, sin, rope) * a).sum() + (turn(normed(k64, w64[1], 1e-5, 0.0), cos, sin, rope) * b).sum()
    for x, y in zip(got, torch.autograd.grad(plain, leaves64)):
        # as in test_backward, with the largest value in the place of each one's terms
        assert (x.double() - y).abs().max() <= 64 * U * max(1.0, y.abs().max().item()) * 8
    # a difference along a random direction: h = 2^-7 leaves h^2 / 6 of a third derivative and the loss's rounding
    h = 2.0 ** -7
    dirs = [torch.randn(t.shape, generator=g, device=dev) for t in leaves]

    def moved(sign):
        ts = [t.detach() + sign * h * d for t, d in zip(leaves, dirs)]
        rest = iter(ts[2:])
        return loss(ts[0], ts[1], *(None if t is None else next(rest) for t in w)).item()

    slope = (moved(1) - moved(-1)) / (2 * h)
    want = sum((x.double() * d).sum().item() for x, d in zip(got, dirs))
    scale = sum((x.double() * d).abs().sum().item() for x, d in zip(got, dirs))
    assert abs(slope - want) <= scale * (h * h + 2.0 ** -12)


def test_autograd_of_one_output(dev):
    """An output that the loss does not use, expanded gradients, and inputs that need none."""
    import torch

    import nf4_quantize_amd as nq

    rope, w = nq.NF4Rotary(16, device=dev), torch.ones(16, device=dev, requires_grad=True)
    q = torch.randn(4, 2, 16, device=dev, requires_grad=True)
    k = torch.randn(4, 1, 16, device=dev, requires_grad=True)
    y, z = nq.rotary(q, k, None, rope, w, w)
    z.sum().backward()
    assert q.grad is None or not q.grad.any()
    want = nq.rotary_backward(None, torch.ones_like(z), None, rope, None, k.detach(), None, w.detach())
    assert torch.equal(k.grad, want[1]) and torch.equal(w.grad, want[3])
    y, none = nq.rotary(q, None, None, rope, w.detach())
    assert none is None
    w.grad = q.grad = None
    y.square().sum().backward()
    assert w.grad is None and q.grad is not None
    with pytest.raises(RuntimeError, match="once_differentiable|twice"):
        (gq,) = torch.autograd.grad(nq.rotary(q, None, None, rope)[0].square().sum(), q, create_graph=True)
        gq.sum().backward()


def test_other_stream_and_graph(dev):
    """On a stream of the caller's, and captured: every replay gives the eager result."""
    import torch

    import nf4_quantize_amd as nq

    g = gen(dev, 5)
    rope, w = nq.NF4Rotary(64, device=dev), torch.rand(64, generator=g, device=dev)
    q, k = (torch.randn(2, 300, n, 64, generator=g, device=dev).bfloat16() for n in (4, 2))
    at = torch.randint(0, 1000, (2, 300), generator=g, device=dev, dtype=torch.int32)

    def both(q, k):
        y, z = nq.rotary_forward(q, k, at, rope, w, w)
        return (y, z, *nq.rotary_backward(y, z, at, rope, q, k, w, w))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    want = both(q, k)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        got = both(q, k)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both(q, k)
    for seed in range(3):
        q.copy_(torch.randn(q.shape, generator=gen(dev, 20 + seed), device=dev))
        want = both(q, k)
        for t in held:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(held, want)), seed


def test_offsets_past_32_bits(dev):
    """Tokens whose elements lie more than 2^31 elements apart."""
    import torch

    import nf4_quantize_amd as nq

    rope = nq.NF4Rotary(32, device=dev)
    flat = torch.zeros(2 ** 32 + 4096, dtype=torch.bfloat16, device=dev)
    q = flat.as_strided((3, 2, 32), (2 ** 31 + 64, 32, 1))
    q.copy_(torch.randn(3, 2, 32, device=dev))
    w = torch.rand(32, device=dev)
    dense = q.contiguous()
    want, _ = nq.rotary_forward(dense, None, None, rope, w)
    dwant = nq.rotary_backward(want, None, None, rope, dense, None, w)
    got = nq.rotary_backward(want, None, None, rope, q, None, w)
    assert torch.equal(got[0], dwant[0]) and torch.equal(got[2], dwant[2])
    nq.rotary_forward(q, None, None, rope, w, q_out=q)
    assert torch.equal(q, want) and int((flat != 0).sum()) == int((want != 0).sum())
