"""The residual norms (nf4_residual_norm_forward / _backward) against their
formulas in 64 bits, through torch's own differentiation of them, and against
differences of the kernel's own forward.

Tolerances: a row's statistics are fp32 sums of squares (a lane adds at most 32
terms, then a tree of 10: 48 u of a sum of positive terms, u = 2^-24, halved by
the root); products with weights and gates add a few u. So fp32 outputs are
within 64 u = 4e-6 of the largest term that they are made of, and bfloat16
outputs within 2^-8 of themselves besides. A sum over rows adds `rows` terms at
most in sequence: (rows + 64) u of the sum of their magnitudes."""
import numpy as np
import pytest

import nf4_quantize_amd as nq
from gpu_util import log

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ALPHA, EPS = 0.6, 1e-5


def make(dev, rows, dim, dtype, res, wt, gate, seed=0):
    import torch

    g = torch.Generator(device=dev)
    g.manual_seed(seed * 100003 + rows * 131 + dim)

    def randn(*s):
        return torch.randn(*s, generator=g, device=dev)

    y, h = (3 * randn(rows, dim)).to(dtype), randn(rows, dim).to(res)
    if rows > 2:
        y[1] = 0                      # a masked place: nothing to add, nothing to normalise
        h[1] = 0
        y[2] *= 1e-3
    w_pre, w_post = (1 + 0.3 * randn(dim)).to(wt), (0.3 * randn(dim)).to(wt)
    gt = {"none": None, "channel": (0.5 + 0.3 * randn(dim)).to(wt), "token": torch.sigmoid(randn(rows, dim)).to(dtype)}[gate]
    return y, h, w_pre, w_post, gt, randn(rows, dim).to(dtype), (0.5 * randn(rows, dim)).to(res)


def reference(y, h, w_pre, w_post, gate, off=0.0):
    z = y
    if w_post is not None:
        z = y / (y.square().mean(-1, keepdim=True) + EPS).sqrt() * (w_post + off)
    t = ALPHA * (z if gate is None else gate * z)
    out = h + t
    x = out / (out.square().mean(-1, keepdim=True) + EPS).sqrt() * (w_pre + off)
    return out, x, t


def close(got, want, size, bf16, what):
    import torch

    err = (got.double() - want).abs()
    tol = 64 * U * size + (2.0 ** -8 * want.abs() if bf16 else 0.0)
    bad = err > tol
    assert not bool(bad.any()), (what, torch.nonzero(bad)[:3].tolist(), float((err / tol.clamp_min(1e-300)).max()))


DIMS = [1, 7, 8, 9, 63, 64, 65, 100, 500, 513, 1024, 2047, 2049, 4100, 8192, 8200, 12345, 16384, 20000, 32768]
TYPES = [("bfloat16", "bfloat16", "bfloat16"), ("bfloat16", "float32", "float32"), ("float32", "float32", "float32"),
         ("float32", "float32", "bfloat16")]


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("types", TYPES)
def test_forward(dev, dim, types):
    import torch

    dtype, res, wt = (getattr(torch, t) for t in types)
    for rows, gate, post, off in ((1, "channel", True, 0.0), (5, "token", False, 1.0), (67, "none", True, 1.0),
                                  (300 if dim < 5000 else 9, "channel", False, 0.0)):
        log(f"norm fwd {rows}x{dim} {types} gate={gate} post={post}")
        y, h, w_pre, w_post, g, _, _ = make(dev, rows, dim, dtype, res, wt, gate)
        w_post = w_post if post else None
        got_h, got_x, rstd_pre, rstd_post = nq.residual_norm_forward(y, h, w_pre, w_post, g, ALPHA, EPS, off)
        d = [None if t is None else t.double() for t in (y, h, w_pre, w_post, g)]
        want_h, want_x, t = reference(*d, off=off)
        size = d[1].abs() + t.abs()
        close(got_h, want_h, size, res == torch.bfloat16, "h")
        r1 = 1 / (want_h.square().mean(-1, keepdim=True) + EPS).sqrt()
        # x: its own terms, and the row's statistic under them
        row = (size.square().mean(-1, keepdim=True) + EPS).sqrt() * r1
        close(got_x, want_x, (size + want_h.abs() * row) * r1 * (d[2] + off).abs(), dtype == torch.bfloat16, "x")
        close(rstd_pre, r1[:, 0], r1[:, 0] * row[:, 0] ** 2, False, "rstd_pre")
        if post:
            r2 = 1 / (d[0].square().mean(-1) + EPS).sqrt()
            close(rstd_post, r2, r2, False, "rstd_post")
        else:
            assert rstd_post is None


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("types", TYPES)
def test_backward(dev, dim, types):
    import torch

    dtype, res, wt = (getattr(torch, t) for t in types)
    for rows, gate, post, off in ((1, "channel", True, 0.0), (5, "token", False, 1.0), (67, "none", True, 1.0),
                                  (1030 if dim < 1100 else 9, "channel", True, 0.0), (21, "token", True, 0.0)):
        log(f"norm bwd {rows}x{dim} {types} gate={gate} post={post}")
        y, h, w_pre, w_post, g, dx, dh_out = make(dev, rows, dim, dtype, res, wt, gate, seed=1)
        w_post = w_post if post else None
        # the saved stream is what the backward pass differentiates at
        d = [None if t is None else t.double().requires_grad_() for t in (y, h, w_pre, w_post, g)]
        n2 = d[0]
        r2 = None
        if post:
            r2 = 1 / (d[0].square().mean(-1, keepdim=True) + EPS).sqrt()
            n2 = d[0] * r2
        z = n2 * (d[3] + off) if post else n2
        t = ALPHA * (z if g is None else d[4] * z)
        stream = d[1] + (t - t.detach())  # h' is the given h: only its gradient goes on to y
        r1 = 1 / (stream.square().mean(-1, keepdim=True) + EPS).sqrt()
        x = stream * r1 * (d[2] + off)
        ((x * dx.double()).sum() + (stream * dh_out.double()).sum()).backward()
        rstd_pre = r1.detach()[:, 0].float()
        rstd_post = r2.detach()[:, 0].float() if post else None
        dy, dh, dw_pre, dw_post, dgate = nq.residual_norm_backward(dx, dh_out, y, h, rstd_pre, w_pre, rstd_post, w_post, g,
                                                                   ALPHA, off)
        with torch.no_grad():
            w1 = (d[2] + off).abs()
            q = dx.double().abs() * w1
            n1 = (h.double() * r1).abs()
            # sizes of the terms of dh, and of what they are multiplied into
            s_dh = dh_out.double().abs() + r1 * (q + n1 * (q * n1).mean(-1, keepdim=True))
            close(dh, d[1].grad, s_dh, res == torch.bfloat16, "dh")
            ga = ALPHA * (1.0 if g is None else d[4].abs())
            s_dz = ga * s_dh
            if post:
                w2 = (d[3] + off).abs()
                s_dy = r2 * (s_dz * w2 + n2.abs() * (s_dz * w2 * n2.abs()).mean(-1, keepdim=True))
            else:
                s_dy = s_dz
            close(dy, d[0].grad, s_dy, dtype == torch.bfloat16, "dy")
            rows_u = (rows + 64) / 64.0
            bf = wt == torch.bfloat16
            close(dw_pre, d[2].grad, rows_u * (dx.double().abs() * n1).sum(0), bf, "dw_pre")
            if post:
                close(dw_post, d[3].grad, rows_u * (s_dz * n2.abs()).sum(0), bf, "dw_post")
            else:
                assert dw_post is None
            if gate == "channel":
                close(dgate, d[4].grad, rows_u * (ALPHA * s_dh * z.abs()).sum(0), bf, "dgate")
            elif gate == "token":
                close(dgate, d[4].grad, ALPHA * s_dh * z.abs(), dtype == torch.bfloat16, "dgate")
            else:
                assert dgate is None


@pytest.mark.parametrize("dim,gate", [(96, "channel"), (1030, "token"), (4097, "channel")])
def test_gradient_against_differences(dev, dim, gate):
    """Along a random direction of every input: two central differences of the
    kernel's forward, at e and e / 2, joined so that the error of order e^2 goes.
    The forward's rounding (64 u of the terms) over the smaller step 2^-6 is
    2.5e-4 of the sum of the terms' magnitudes over their square root's worth of
    independent errors; what is left is of order e^4 = 1e-6."""
    import torch

    rows = 12
    y, h, w_pre, w_post, g, dx, dh_out = make(dev, rows, dim, torch.float32, torch.float32, torch.float32, gate, seed=2)
    y[1], h[1] = 1.0, 0.5
    y[2] *= 1e3
    inputs = [t.clone().requires_grad_() for t in (y, h, w_pre, w_post, g)]

    def loss(ts):
        out, x = nq.residual_norm(ts[0], ts[1], ts[2], ts[3], ts[4], ALPHA, EPS)
        return (x.double() * dx.double()).sum() + (out.double() * dh_out.double()).sum(), x, out

    value, x, out = loss(inputs)
    value.backward()
    size = float((x.double() * dx.double()).square().sum().sqrt() + (out.double() * dh_out.double()).square().sum().sqrt())
    for k, t in enumerate(inputs):
        direction = torch.randn(t.shape, device=dev) * t.detach().abs().mean()

        def at(e):
            ts = [u.detach() for u in inputs]
            ts[k] = ts[k] + e * direction
            return loss(ts)[0].item()

        e = 2.0 ** -5
        d1, d2 = ((at(s) - at(-s)) / (2 * s) for s in (e, e / 2))
        diff = (4 * d2 - d1) / 3
        grad = float((t.grad.double() * direction.double()).sum())
        # rounding errors of the elements are independent: their sum is of the size of the terms' norm
        tol = 8 * 64 * U * size * 2 / e + 1e-4 * float((t.grad.double() * direction.double()).square().sum().sqrt())
        assert abs(diff - grad) <= tol, (k, diff, grad, tol)


def test_norm_alone_and_absent_gradients(dev):
    """y absent (x = norm(h)); dx or dh_out absent; gradients that are not wanted."""
    import torch

    y, h, w_pre, w_post, g, dx, dh_out = make(dev, 33, 777, torch.bfloat16, torch.bfloat16, torch.float32, "channel")
    h2, x, rstd, none = nq.residual_norm_forward(None, h, w_pre, eps=EPS)
    assert h2 is h and none is None
    d = h.double()
    r = 1 / (d.square().mean(-1, keepdim=True) + EPS).sqrt()
    close(x, d * r * w_pre.double(), (d * r * w_pre.double()).abs(), True, "x")
    dy, dh, dw, dwp, dg = nq.residual_norm_backward(dx, None, None, h, rstd, w_pre)
    zero = torch.zeros_like(dh_out)
    full = nq.residual_norm_backward(dx, zero, None, h, rstd, w_pre)
    assert dy is None and dwp is None and dg is None
    assert torch.equal(dh, full[1]) and torch.equal(dw, full[2])
    rp = torch.ones(33, device=dev)
    a = nq.residual_norm_backward(None, dh_out, y, h, rstd, w_pre, rp, w_post, g, ALPHA)
    b = nq.residual_norm_backward(torch.zeros_like(dx), dh_out, y, h, rstd, w_pre, rp, w_post, g, ALPHA)
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    assert torch.equal(a[1], dh_out) and not bool(a[2].any())
    c = nq.residual_norm_backward(dx, dh_out, y, h, rstd, w_pre, rp, w_post, g, ALPHA)
    for k in range(5):
        want = [j == k for j in range(5)]
        part = nq.residual_norm_backward(dx, dh_out, y, h, rstd, w_pre, rp, w_post, g, ALPHA, want=want)
        assert [t is not None for t in part] == want and torch.equal(part[k], c[k])


def test_no_rows(dev):
    import torch

    y, h, w_pre, w_post, g, dx, dh_out = make(dev, 0, 64, torch.bfloat16, torch.bfloat16, torch.float32, "channel")
    out = nq.residual_norm_forward(y, h, w_pre, w_post, g)
    assert out[0].shape == (0, 64) and out[2].shape == (0,)
    grads = nq.residual_norm_backward(dx, dh_out, y, h, out[2], w_pre, out[3], w_post, g)
    assert all(not bool(t.any()) for t in grads[2:]) and grads[0].shape == (0, 64)


def test_in_place_guards_and_repeat(dev):
    """The residual stream updated in place gives the same bits; what surrounds
    outputs of odd width keeps its bytes; a second call gives the same bits."""
    import torch

    for rows, dim in ((3, 5), (17, 511), (40, 2049)):
        y, h, w_pre, w_post, g, dx, dh_out = make(dev, rows, dim, torch.bfloat16, torch.bfloat16, torch.float32, "channel")
        h1, x1, r1, r2 = nq.residual_norm_forward(y, h, w_pre, w_post, g, ALPHA, EPS)
        n = rows * dim
        big = torch.full((2, n + 128), 7.0, dtype=torch.bfloat16, device=dev)
        big = [big[0].clone(), big[1].clone()]
        hv, xv = (b[64:64 + n].view(rows, dim) for b in big)
        hv.copy_(h)
        nq.residual_norm_forward(y, hv, w_pre, w_post, g, ALPHA, EPS, h_out=hv, x_out=xv)
        assert torch.equal(hv, h1) and torch.equal(xv, x1)
        for b in big:
            assert bool((b[:64] == 7).all()) and bool((b[64 + n:] == 7).all())
        first = nq.residual_norm_backward(dx, dh_out, y, h1, r1, w_pre, r2, w_post, g, ALPHA)
        again = nq.residual_norm_backward(dx, dh_out, y, h1, r1, w_pre, r2, w_post, g, ALPHA)
        assert all(torch.equal(s, t) for s, t in zip(first, again))


def test_many_rows_go_round(dev):
    """Rows of one element, more than a launch has workgroups' places for."""
    import torch

    rows = (1 << 20) * 32 + 5
    h = torch.full((rows, 1), 2.0, dtype=torch.bfloat16, device=dev)
    h[-1] = -3.0
    _, x, rstd, _ = nq.residual_norm_forward(None, h, torch.ones(1, device=dev), eps=0.0)
    assert bool((x[:-1] == 1).all()) and float(x[-1]) == -1 and float(rstd[0]) == 0.5


def test_refusals_on_device(dev):
    import torch

    y = torch.zeros(4, 64, device=dev)
    w = torch.ones(64, device=dev)
    with pytest.raises(ValueError):
        nq.residual_norm_forward(y.t(), y.t(), torch.ones(4, device=dev))
    with pytest.raises(ValueError):
        nq.residual_norm_forward(y, y, w, h_out=torch.zeros(4, 32, device=dev))
    with pytest.raises(nq.NF4Error):
        nq.residual_norm_forward(y, y.bfloat16(), w)
    with pytest.raises(nq.NF4Error):
        nq.residual_norm_forward(None, torch.zeros(1, 40000, device=dev), torch.ones(40000, device=dev))
    with pytest.raises(ValueError):
        nq.residual_norm_backward(y, y, y, y, torch.ones(3, device=dev), w)
