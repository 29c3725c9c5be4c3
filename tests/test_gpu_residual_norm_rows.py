"""The residual norms with more rows than a launch has places for: a workgroup
takes several sets of rows, the next one's loads in flight while it works on one,
and its last set may be ragged. No row of zeros; formulas and tolerances are those
of test_gpu_residual_norm.py."""
import pytest

import nf4_quantize_amd as nq
import test_gpu_residual_norm as base
from gpu_util import log
from test_gpu_residual_norm import ALPHA, EPS, close

pytestmark = pytest.mark.gpu

TYPES = [("bfloat16", "bfloat16", "bfloat16"), ("bfloat16", "float32", "float32"), ("float32", "float32", "float32")]


def make(dev, rows, dim, types, gate, seed):
    import torch

    dtype, res, wt = (getattr(torch, t) for t in types)
    y, h, w_pre, w_post, g, dx, dh_out = base.make(dev, rows, dim, dtype, res, wt, gate, seed=seed)
    y[1:3], h[1] = y[3:5] + y[5:7], h[3] - h[4]  # rows like the others
    return y, h, w_pre, w_post, g, dx, dh_out


def f64(*ts):
    return [None if t is None else t.double() for t in ts]


# Workgroups of a launch: 512 of one row at 8192 columns, 2048 / 128 x 256 at 1024, 2048 of four rows
# up to 512 columns and of 32 at 64
@pytest.mark.parametrize("rows,dim", [(1601, 8192), (1030, 8184), (4107, 1024), (4099, 1000), (9003, 500), (65603, 64),
                                      (1100, 4100), (1030, 12288)])
@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("gate,post", [("channel", True), ("token", False), ("token", True), ("none", False)])
def test_forward(dev, rows, dim, types, gate, post):
    import torch

    log(f"norm fwd rows {rows}x{dim} {types} gate={gate} post={post}")
    y, h, w_pre, w_post, g, _, _ = make(dev, rows, dim, types, gate, seed=3)
    w_post = w_post if post else None
    d = f64(y, h, w_pre, w_post, g)
    want_h, want_x, t = base.reference(*d)
    size = d[1].abs() + t.abs()
    r1 = 1 / (want_h.square().mean(-1, keepdim=True) + EPS).sqrt()
    row = (size.square().mean(-1, keepdim=True) + EPS).sqrt() * r1
    for in_place in (False, True):
        stream = h.clone()
        got_h, got_x, rstd_pre, rstd_post = nq.residual_norm_forward(y, stream, w_pre, w_post, g, ALPHA, EPS,
                                                                     h_out=stream if in_place else None)
        assert in_place or torch.equal(stream, h)
        close(got_h, want_h, size, h.dtype == torch.bfloat16, "h")
        close(got_x, want_x, (size + want_h.abs() * row) * r1 * d[2].abs(), y.dtype == torch.bfloat16, "x")
        close(rstd_pre, r1[:, 0], r1[:, 0] * row[:, 0] ** 2, False, "rstd_pre")
        if post:
            r2 = 1 / (d[0].square().mean(-1) + EPS).sqrt()
            close(rstd_post, r2, r2, False, "rstd_post")


@pytest.mark.parametrize("rows,dim", [(803, 8192), (811, 4104), (805, 2049), (1501, 4096), (2311, 1024), (9003, 500),
                                      (65603, 64), (603, 9000), (410, 16384)])
@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("gate,post", [("channel", True), ("token", False), ("token", True), ("none", False)])
def test_backward(dev, rows, dim, types, gate, post):
    import torch

    log(f"norm bwd rows {rows}x{dim} {types} gate={gate} post={post}")
    y, h, w_pre, w_post, g, dx, dh_out = make(dev, rows, dim, types, gate, seed=4)
    w_post = w_post if post else None
    y_, h_, w1, w2, g_, dx_, dho = f64(y, h, w_pre, w_post, g, dx, dh_out)
    r1 = 1 / (h_.square().mean(-1, keepdim=True) + EPS).sqrt()
    r2 = 1 / (y_.square().mean(-1, keepdim=True) + EPS).sqrt() if post else None
    got = nq.residual_norm_backward(dx, dh_out, y, h, r1[:, 0].float(), w_pre, r2[:, 0].float() if post else None, w_post, g,
                                    ALPHA)
    got = dict(zip(("dy", "dh", "dw_pre", "dw_post", "dgate"), got))

    def through(a, r, dn, mag):
        """The gradient of a norm's input, and the size of its terms."""
        dot = (dn * a).mean(-1, keepdim=True)
        return r * dn - a * r ** 3 * dot, r * (mag + (a * r).abs() * (mag * (a * r).abs()).mean(-1, keepdim=True))

    act, res, bf = y.dtype == torch.bfloat16, h.dtype == torch.bfloat16, w_pre.dtype == torch.bfloat16
    rows_u = (rows + 64) / 64.0
    q = dx_ * w1
    dh, s_dh = through(h_, r1, q, q.abs())
    dh, s_dh = dh + dho, s_dh + dho.abs()
    close(got["dh"], dh, s_dh, res, "dh")
    n1 = h_ * r1
    close(got["dw_pre"], (dx_ * n1).sum(0), rows_u * (dx_ * n1).abs().sum(0), bf, "dw_pre")
    n2 = y_ * r2 if post else y_
    z = n2 * w2 if post else y_
    ga = ALPHA * (torch.ones_like(w1) if g is None else g_)
    dz, s_dz = ga * dh, ga.abs() * s_dh
    if gate == "channel":
        close(got["dgate"], (ALPHA * dh * z).sum(0), rows_u * (ALPHA * s_dh * z.abs()).sum(0), bf, "dgate")
    elif gate == "token":
        close(got["dgate"], ALPHA * dh * z, ALPHA * s_dh * z.abs(), act, "dgate")
    else:
        assert got["dgate"] is None
    if post:
        close(got["dw_post"], (dz * n2).sum(0), rows_u * (s_dz * n2.abs()).sum(0), bf, "dw_post")
        dz, s_dz = through(y_, r2, dz * w2, s_dz * w2.abs())
    else:
        assert got["dw_post"] is None
    close(got["dy"], dz, s_dz, act, "dy")
