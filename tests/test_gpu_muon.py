"""The Muon step and the orthogonalising alone against their formulas in 64 bits.

Tolerances. u = 2^-24. The update u and X0 are off by 4 u of their terms. S = X0^T X0 is summed in fp32 over 32
rows and in fp64 beyond: off by 64 u of the sum of the terms' magnitudes, at most |X0|^2 = 1 in the
Frobenius norm. O = X0 P(S) moves with S by the divided differences of P's polynomial, |dO| <= max_ij sigma_i
|p[lambda_i, lambda_j]| |dS|, taken here from the spectrum itself. Steps in fp64 add nothing to speak of. Steps in
fp32 (all but the first where the weights are bf16 alone, all but two where there are fp32 weights) have products
off by w = 2 u (s / 32 + 2) of |x| |y| in the Frobenius norm; what that does to A_k moves O as above, with the steps that
are left, and what it does to P_k is multiplied by those steps' polynomials. The product in fp32 adds (s + 4) u of |X0| |P|, element by element, P being rounded to fp32 as well.
Then the output's half step. All in the Frobenius norm, which one wrong element of O exceeds."""
import math

import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
COEF = (3.4445, -4.775, 2.0315)


def half_step(dt):
    import torch

    return torch.finfo(dt).eps / 2


def gen(dev, seed):
    import torch

    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return g


def definition(u, coef=COEF, iterations=5, eps=1e-7):
    a, b, c = coef
    x = u / max(float(u.norm()), eps)
    flip = x.shape[0] < x.shape[1]
    x = x.mT.contiguous() if flip else x
    for _ in range(iterations):
        s = x.mT.contiguous() @ x
        x = a * x + b * (x @ s) + c * (x @ (s @ s))
    return x.mT if flip else x


def allowed(u, coef=COEF, iterations=5, eps=1e-7, terms=None, exact=16):
    """The Frobenius norm of O's error by the arithmetic above; `terms`: of u's magnitudes, where u is a sum;
    `exact`: the steps in fp64."""
    import torch

    a, b, c = coef
    norm = max(float(u.norm()), eps)
    x = u.double().cpu() / norm
    x = x if x.shape[0] >= x.shape[1] else x.mT
    lam, v = torch.linalg.eigh(x.mT.contiguous() @ x)
    lam = lam.clamp_min(0)

    def p(t, steps):
        y, out = t.clone(), torch.ones_like(t)
        for _ in range(steps):
            q = a + b * y + c * y * y
            out, y = out * q, y * q * q
        return out

    def moves(lam, steps):
        f, gap, h = p(lam, steps), lam[:, None] - lam[None, :], 1e-7
        near = gap.abs() < 1e-9
        slope = (p(lam + h, steps) - p((lam - h).clamp_min(0), steps)) / (lam + h - (lam - h).clamp_min(0))
        div = torch.where(near, (slope[:, None].abs() + slope[None, :].abs()),
                          (f[:, None] - f[None, :]) / torch.where(near, 1.0, gap))
        return float((lam.sqrt()[:, None] * div.abs()).max())

    f = p(lam, iterations)
    k = moves(lam, iterations)
    extra, at, so_far = 0.0, lam.clone(), torch.ones_like(lam)
    for step in range(iterations):
        q = a + b * at + c * at * at
        if step >= exact:
            w = 2 * U * (x.shape[1] / 32 + 2)
            # A_k as it came (its rounding, and two products in the step that made it), then P Q
            extra += moves(at, iterations - step) * (U + 2 * w * float(q.norm()) * float(q.abs().max())) * float(at.norm())
            extra += w * float(so_far.norm()) * float(q.norm()) * float(p(at, iterations - step).div(q).abs().max())
        so_far, at = so_far * q, at * q * q
    big = v.abs() @ (f.abs()[:, None] * v.mT.abs())  # not below |P|, element by element
    big = torch.minimum(big, f.abs().max())
    ratio = 1.0 if terms is None else max(1.0, float(terms.norm()) / norm)
    product = (x.shape[1] + 4) * U * float((x.abs() @ (v * f @ v.mT).abs()).norm())
    return extra + (64 + 8 * ratio) * U * k + 4 * U * ratio * float(f.abs().max()) + product


def check(got, want, tol, dt, what):
    err = float((got.double() - want).norm())
    bound = tol + half_step(dt) * float(want.norm()) + 1e-30
    assert err <= bound, f"{what}: error {err:.3e}, bound {bound:.3e}"


SHAPES = [(1, 1), (1, 300), (300, 1), (2, 2), (13, 2047), (2047, 13), (16, 16), (20, 17), (1000, 16), (32, 1000), (33, 5000),
          (5000, 33), (48, 50), (64, 64), (4096, 64), (64, 4099), (65, 65), (65, 70), (129, 100), (128, 900), (1001, 200),
          (200, 1001), (256, 256), (3000, 256), (255, 3001), (20000, 8), (7, 20001)]


@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}")
def test_orthogonalize(dev, shape, dt):
    import torch

    import nf4_quantize_amd as nq

    dt = getattr(torch, dt)
    u = (torch.randn(*shape, generator=gen(dev, 1), device=dev) * 1e-3).to(dt)
    (got,) = nq.orthogonalize([u])
    assert got.dtype == dt and got.shape == u.shape
    check(got, definition(u.double()), allowed(u, exact=16 if dt == torch.float32 else 1), dt, shape)
    if min(shape) > 1 and shape != (2, 2):  # between the coefficients' bounds, as far as nothing was near zero
        s = torch.linalg.svdvals(definition(u.double()))
        assert s.max() < 1.3


@pytest.mark.parametrize("shape", [(512, 64), (48, 700), (600, 130)], ids=str)
@pytest.mark.parametrize("kind", ["low_rank", "spread", "equal"])
def test_spectra(dev, shape, kind):
    """Updates of few directions, of singular values over six decades, and orthogonal ones."""
    import torch

    import nf4_quantize_amd as nq

    g = gen(dev, 2)
    s = min(shape)
    q1 = torch.linalg.qr(torch.randn(shape[0], s, generator=g, device=dev, dtype=torch.float64))[0]
    q2 = torch.linalg.qr(torch.randn(shape[1], s, generator=g, device=dev, dtype=torch.float64))[0]
    at = torch.arange(s, device=dev, dtype=torch.float64)
    sigma = {"low_rank": (at < 3).double(), "spread": 10.0 ** (-6 * at / s), "equal": torch.ones_like(at)}[kind]
    u = (q1 * sigma @ q2.mT).float().contiguous()
    (got,) = nq.orthogonalize([u])
    check(got, definition(u.double()), allowed(u), torch.float32, kind)


@pytest.mark.parametrize("iterations, coef", [(1, COEF), (2, (1.5, -0.5, 0.0)), (3, COEF), (6, (2.0, -1.5, 0.5))])
@pytest.mark.parametrize("shape", [(300, 40), (90, 300)], ids=str)
def test_iterations(dev, shape, iterations, coef):
    import torch

    import nf4_quantize_amd as nq

    u = torch.randn(*shape, generator=gen(dev, 3), device=dev)
    (got,) = nq.orthogonalize([u], coefficients=coef, iterations=iterations)
    check(got, definition(u.double(), coef, iterations), allowed(u, coef, iterations), torch.float32, shape)


def test_sizes_of_the_norm(dev):
    """Zeros, norms below eps, elements of 1e-15 and of 1e15."""
    import torch

    import nf4_quantize_amd as nq

    x = torch.randn(200, 24, generator=gen(dev, 4), device=dev)
    for scale in (0.0, 1e-12, 1e-15, 1e15):
        for u in (x * scale, (x * scale).t().contiguous()):
            (got,) = nq.orthogonalize([u])
            if scale == 0.0:
                assert not got.any()
            else:
                check(got, definition(u.double()), allowed(u), torch.float32, scale)
    (got,) = nq.orthogonalize([x * 1e-15], eps=1e-12)
    check(got, definition((x * 1e-15).double(), eps=1e-12), allowed(x * 1e-15, eps=1e-12), torch.float32, "small eps")


def test_lists_of_all_sizes(dev):
    """More matrices than a launch of the table takes, small and large ones mixed, empty ones among them: each as alone."""
    import torch

    import nf4_quantize_amd as nq

    g = gen(dev, 5)
    shapes = [(3 + 7 * i % 90, 500 - 3 * i) for i in range(40)] + [(0, 5), (700, 80), (5, 0), (80, 700), (256, 300), (4, 4)] * 5
    us = [torch.randn(*s, generator=g, device=dev) for s in shapes]
    got = nq.orthogonalize(us)
    again = nq.orthogonalize(us)
    for u, x, y in zip(us, got, again):
        assert torch.equal(x, y)  # the same bits each time
        if u.numel():
            check(x, definition(u.double()), allowed(u), torch.float32, u.shape)


def test_in_place_and_neighbours(dev):
    """Outputs that are the updates, and outputs between guards."""
    import torch

    import nf4_quantize_amd as nq

    g = gen(dev, 6)
    for shape in ((130, 12), (12, 131), (300, 77), (77, 300), (64, 64)):
        u = torch.randn(*shape, generator=g, device=dev).bfloat16()
        (want,) = nq.orthogonalize([u])
        n = u.numel()
        wide = torch.full((n + 64,), -3.0, device=dev).bfloat16()
        (got,) = nq.orthogonalize([u], outs=[wide[32:32 + n].view(shape)])
        assert torch.equal(got, want) and bool((wide[:32] == -3).all()) and bool((wide[32 + n:] == -3).all())
        nq.orthogonalize([u], outs=[u])
        assert torch.equal(u, want)
    u = torch.randn(16, 4, device=dev)
    with pytest.raises(ValueError, match="share memory"):
        nq.orthogonalize([u, u], outs=[u, torch.empty_like(u)])
    with pytest.raises(ValueError, match="share memory"):
        nq.orthogonalize([u, u], outs=[torch.empty_like(u)] * 2)
    a, b = nq.orthogonalize([u, u], outs=[torch.empty_like(u), torch.empty_like(u)])
    assert torch.equal(a, b)
    for bad in ([torch.empty(300, 300, device=dev)], [torch.empty(4, device=dev)], [u.t()], [u, u.bfloat16()], [u.half()]):
        with pytest.raises((ValueError, TypeError)):
            nq.orthogonalize(bad)
    with pytest.raises(ValueError):
        nq.orthogonalize([u], outs=[u.bfloat16()])
    with pytest.raises(nq.NF4Error):
        nq.orthogonalize([u], workspace=torch.empty(64, dtype=torch.uint8, device=dev))


LISTS = [(40, 16), (16, 41), (500, 64), (64, 333), (300, 100), (100, 303), (1, 7), (7, 1)]


@pytest.mark.parametrize("w, gt, bits, master, nesterov", [
    ("bfloat16", "bfloat16", 32, False, True), ("bfloat16", "bfloat16", 16, True, False), ("bfloat16", "float32", 32, True, True),
    ("bfloat16", "float32", 16, False, True), ("float32", "float32", 32, False, False), ("float32", "float32", 16, False, True),
    ("float32", "bfloat16", 32, False, True), ("float32", "bfloat16", 16, False, False)])
def test_steps(dev, w, gt, bits, master, nesterov):
    """Three steps, each against the definition from the state before it."""
    import torch

    import nf4_quantize_amd as nq

    g = gen(dev, 7)
    wt, gt = getattr(torch, w), getattr(torch, gt)
    params = [(torch.randn(*s, generator=g, device=dev) * 0.02).to(wt) for s in LISTS]
    half = len(params) // 2
    lr, wd, mu = (2e-2, 5e-3), (0.1, 0.0), 0.9
    opt = nq.NF4Muon([dict(params=params[:half], lr=lr[0], weight_decay=wd[0], masters=master or None),
                      dict(params=params[half:], lr=lr[1], weight_decay=wd[1], masters=master or None)],
                     momentum=mu, nesterov=nesterov, state_bits=bits, adjust="rms" if master else "shape")
    mu, one = (float(torch.tensor(x, dtype=torch.float32)) for x in (mu, 1 - mu))
    for _ in range(3):
        grads = [(torch.randn(*s, generator=g, device=dev) * 1e-2).to(gt) for s in LISTS]
        old_w = [x.double().clone() for x in (opt.masters if master else opt.params)]
        old_m = [x.double().clone() for x in opt.m]
        opt.step(grads)
        for i, (p, gr, w0, m0, m1) in enumerate(zip(params, grads, old_w, old_m, opt.m)):
            gr = gr.double()
            m = mu * m0 + one * gr
            terms = mu * m0.abs() + one * gr.abs()
            assert ((m1.double() - m).abs() <= 4 * U * terms + half_step(m1.dtype) * m.abs()).all()
            u = mu * m + one * gr if nesterov else m
            if nesterov:
                terms = mu * terms + one * gr.abs()
            k = i >= half
            scale = 0.2 * math.sqrt(max(p.shape)) if master else math.sqrt(max(1.0, p.shape[0] / p.shape[1]))
            want = w0 * (1 - lr[k] * wd[k]) - lr[k] * scale * definition(u)
            tol = lr[k] * scale * (allowed(u, terms=terms, exact=2 if master or wt == torch.float32 else 1) + 4 * U * float(definition(u).norm())) + 4 * U * float(w0.norm())
            check(opt.masters[i] if master else p, want, tol, torch.float32 if master else wt, p.shape)
            if master:
                assert torch.equal(p, opt.masters[i].to(wt))
    assert opt.steps == 3


def test_norms_that_are_not_finite(dev):
    """A matrix with a NaN, an infinity or too large elements keeps weight and momentum; the others step as without it."""
    import torch

    import nf4_quantize_amd as nq

    g = gen(dev, 8)
    for shape in ((50, 20), (20, 50), (200, 90)):
        params = [torch.randn(*shape, generator=g, device=dev) for _ in range(4)]
        alone = params[3].clone()
        grads = [torch.randn(*shape, generator=g, device=dev) for _ in range(4)]
        grads[0][3, 4], grads[1][7, 1] = float("nan"), float("-inf")
        grads[2] *= 1e25
        keep = [p.clone() for p in params]
        opt, one = nq.NF4Muon(params), nq.NF4Muon([alone])
        opt.step(grads), one.step(grads[3:])
        for i in range(3):
            assert torch.equal(params[i], keep[i]) and not opt.m[i].any()
        assert torch.equal(params[3], alone) and torch.equal(opt.m[3], one.m[0])
        out = nq.orthogonalize(grads)
        assert all(bool(torch.isnan(x).all()) for x in out[:3]) and bool(torch.isfinite(out[3]).all())


def test_contracts(dev):
    """What the other optimizer over a list refuses, this one refuses; states travel."""
    import copy

    import torch

    import nf4_quantize_amd as nq

    g = gen(dev, 9)

    def fresh():
        return [torch.randn(30, 8, generator=gen(dev, 1), device=dev), torch.randn(8, 40, generator=gen(dev, 2), device=dev)]

    def grads():
        return [torch.randn(30, 8, generator=g, device=dev), torch.randn(8, 40, generator=g, device=dev)]

    with pytest.raises(ValueError, match="at most 256"):
        nq.NF4Muon([torch.zeros(300, 300, device=dev)])
    for shape in ((5,), (2, 3, 4), ()):
        with pytest.raises(ValueError, match="matrices"):
            nq.NF4Muon([torch.zeros(shape, device=dev)])
    p = torch.zeros(20, 20, device=dev)
    with pytest.raises(ValueError, match="share memory"):
        nq.NF4Muon([p, p])
    with pytest.raises(ValueError, match="adjust"):
        nq.NF4Muon([p], adjust="size")
    params = fresh()
    opt = nq.NF4Muon(params, lr=1e-2)
    with pytest.raises(TypeError):
        copy.deepcopy(opt)
    with pytest.raises(ValueError, match="no gradient"):
        opt.step()
    for bad in (grads()[:1], [grads()[0]] * 2, [x.t().contiguous() for x in grads()], [grads()[0], grads()[1].bfloat16()],
                [grads()[0].t().contiguous().t(), grads()[1]], [x.cpu() for x in grads()]):
        with pytest.raises(ValueError):
            opt.step(bad)
    opt.step(grads())
    opt.m[0] = torch.zeros_like(opt.m[0])
    with pytest.raises(ValueError, match="bind_state"):
        opt.step(grads())
    opt.bind_state([x.clone() for x in opt.state_dict()["m"]])
    opt.step(grads())
    for bad in ([opt.m[0]], [opt.m[0].t().contiguous(), opt.m[1]], [x.bfloat16() for x in opt.m], [params[0], opt.m[1]]):
        with pytest.raises(ValueError):
            opt.bind_state(bad)
    # a state in another optimizer: both go on alike
    other = [p.clone() for p in params]
    twin = nq.NF4Muon(other, lr=5.0)
    twin.load_state_dict(opt.state_dict())
    more = grads()
    opt.step(more), twin.step(more)
    assert all(torch.equal(x, y) for x, y in zip(params + opt.m, other + twin.m)) and twin.steps == opt.steps == 3
    with pytest.raises(ValueError):
        nq.NF4Muon(fresh(), state_bits=16).load_state_dict(opt.state_dict())
    with pytest.raises(ValueError):
        nq.NF4Muon(fresh()[:1]).load_state_dict(opt.state_dict())
    # other memory is found again, another shape refused
    params[0].data = params[0].data.clone()
    opt.step(grads())
    params[0].data = params[0].data.view(8, 30)
    with pytest.raises(ValueError, match="shape"):
        opt.step(grads())


def test_autograd_sees_the_step(dev):
    import torch

    import nf4_quantize_amd as nq

    w = torch.randn(20, 6, device=dev, requires_grad=True)
    x = torch.randn(5, 20, device=dev, requires_grad=True)
    opt = nq.NF4Muon([w])
    y = (x @ w).square().sum()
    y.backward(retain_graph=True)
    opt.step()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    opt.zero_grad()
    assert w.grad is None


def test_stream_and_graph(dev):
    """On another stream, and captured: each replay steps on from the state that it finds."""
    import torch

    import nf4_quantize_amd as nq

    g = gen(dev, 10)
    shapes = [(200, 16), (16, 300), (150, 80), (64, 64)]
    params = [torch.randn(*s, generator=g, device=dev) for s in shapes]
    eager = [p.clone() for p in params]
    opt, ref = nq.NF4Muon(params, lr=1e-2), nq.NF4Muon(eager, lr=1e-2)
    grads = [torch.randn(*s, generator=g, device=dev) for s in shapes]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        opt.step(grads)
    torch.cuda.current_stream().wait_stream(s)
    ref.step(grads)
    assert all(torch.equal(x, y) for x, y in zip(params, eager))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        opt.step(grads)
    for _ in range(3):
        for x in grads:
            x.copy_(torch.randn(x.shape, generator=g, device=dev))
        graph.replay()
        torch.cuda.synchronize()
        ref.step(grads)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(params + opt.m, eager + ref.m))


def test_largest_matrices(dev):
    """Matrices of nearly 2^30 elements, whose bytes lie up to 2^32 apart: rows near their end; larger ones are refused."""
    import torch

    import nf4_quantize_amd as nq

    n, r = (1 << 27) - 1, 8
    u = torch.zeros(n, r, device=dev)
    u[-500:] = torch.randn(500, r, generator=gen(dev, 11), device=dev)
    (got,) = nq.orthogonalize([u])
    want = definition(u[-500:].double())
    check(got[-500:], want, allowed(u[-500:]), torch.float32, "end")
    assert int((got != 0).any(1).sum()) <= 500
    del got
    wide = u.view(r, n)
    wide.zero_()
    wide[:, -500:] = torch.randn(r, 500, generator=gen(dev, 12), device=dev)
    (got,) = nq.orthogonalize([wide])
    check(got[:, -500:], definition(wide[:, -500:].double()), allowed(wide[:, -500:]), torch.float32, "end")
    del got
    with pytest.raises(nq.NF4Error):
        nq.orthogonalize([torch.empty(1 << 27, 8, dtype=torch.bfloat16, device=dev)])
