"""What the training step's calls promise besides their formulas: small second
moments, what autograd is told, which tensors an optimizer takes and keeps, and
what it refuses. Sizes are small; the formulas' own tests are in
test_gpu_adamw.py, test_gpu_residual_norm.py and test_gpu_embedding.py."""
import copy
import io
import pickle

import numpy as np
import pytest

import nf4_quantize_amd as nq
from gpu_util import log

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


# ------------------------------------------------------------------ small moments

@pytest.mark.parametrize("eps", [0.0, 1e-24, 2.0 ** -60, 0.99 * 2.0 ** -39, 2.0 ** -39, 1e-8])
def test_root_of_small_second_moments(dev, eps):
    """Second moments among fp32's subnormals (below 2^-126) and around them: the
    step is lr m / (sqrt(v) + eps), not lr m / eps. The moments before the step are
    given, the gradient is zero, so v' = beta2 v up to one rounding: U of itself and
    2^-149, that is 2^-150 / v of the root; the bias corrections at step 100000
    are 1 in fp32 for the first and 1 - 3.5e-44 for the second. Then 24 U as in the
    other tests of the step, and 2 U of the weight."""
    import torch

    n = 300
    exps = np.linspace(-143, -110, n)
    v0 = np.exp2(exps).astype(np.float32)
    v1 = v0.astype(np.float64) * 0.999
    m0 = (np.sqrt(v0.astype(np.float64)) * np.where(np.arange(n) % 2, 1.0, -0.5)).astype(np.float32)
    p = torch.full((n,), 0.25, device=dev)
    opt = nq.NF4AdamW([p], lr=1e-2, weight_decay=0.0, eps=eps, state_bits=32)
    opt.bind_state([torch.from_numpy(m0).to(dev)], [torch.from_numpy(v0).to(dev)])
    opt.step([torch.zeros(n, device=dev)], step=100000)
    step = 1e-2 * 0.9 * m0.astype(np.float64) / (np.sqrt(v1) + float(np.float32(eps)))
    tol = 2 * U * 0.26 + np.abs(step) * (24 * U + 2.0 ** -149 / v1)
    got = p.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - (0.25 - step)) <= tol), float(np.max(np.abs(got - (0.25 - step)) / tol))


@pytest.mark.parametrize("size", [1e-17, 1e-19, 3e-20])
def test_second_moment_is_stored_under_a_stored_first_one(dev, size):
    """Blocks whose second moment over 448 is below 2^-126 keep a scale as long as the
    first moment has one: no decoded v is zero (the smallest code on the smallest scale is
    2^-135), and without eps the steps after the last gradient are those of the stored
    moments: 24 U and, as v may be among the subnormals, 2^-149 / v."""
    import torch

    n, lr = 600, 1e-3

    def moment(opt, name):
        return opt_values(getattr(opt, name)[0], getattr(opt, name + "_scale")[0], n)

    p = torch.zeros(n, device=dev)
    opt = nq.NF4AdamW([p], lr=lr, weight_decay=0.0, eps=0.0, state_bits=8)
    g = torch.full((n,), size, device=dev)
    g[256:512] = 0
    g[256:512:7] = size  # elements without a gradient beside some with one
    opt.step([g.clone().masked_fill_(g == 0, size)])
    for t in range(2, 40):
        m, v = moment(opt, "m"), moment(opt, "v")
        assert bool((opt.m_scale[0] > 0).all()) and float(v.min()) >= 2.0 ** -135, t
        was = p.double()
        grad = g if t < 4 else torch.zeros_like(g)
        opt.step([grad])
        d = grad.double()
        m, v = 0.9 * m + 0.1 * d, 0.999 * v + 0.001 * d * d
        step = lr / (1 - 0.9 ** t) * m / (v / (1 - 0.999 ** t)).sqrt()
        tol = 2 * U * (was.abs() + step.abs()) + step.abs() * (24 * U + 2.0 ** -148 / v)
        err = (p.double() - (was - step)).abs()
        assert bool((err <= tol).all()), (t, float((err / tol).max()))
        assert float(step.abs().max()) <= 2 * lr, t
    opt = nq.NF4AdamW([torch.zeros(300, device=dev)], state_bits=8)
    opt.step([torch.zeros(300, device=dev)])
    assert not bool(opt.v_scale[0].any()) and not bool(opt.m_scale[0].any())  # nothing to store


def opt_values(codes, scale, n):
    """Decoded 8-bit moments."""
    return codes.double() * scale.double().repeat_interleave(256)[:n]


# ------------------------------------------------------------------ autograd

@pytest.mark.parametrize("master", [False, True])
def test_backward_after_a_step_raises(dev, master):
    """A graph that saved a weight is stale once the step has changed it: autograd
    notices, as after any update in place."""
    import torch

    w = torch.nn.Parameter(torch.randn(64, 16, device=dev).to(torch.bfloat16))
    x = torch.randn(8, 64, device=dev).to(torch.bfloat16).requires_grad_()
    opt = nq.NF4AdamW([w], masters=[w.detach().float()] if master else None, max_grad_norm=1.0)
    versions = [t._version for t in [w, opt.grad_norm] + ([opt.masters[0]] if master else [])]
    y = x @ w
    opt.step([torch.ones_like(w)])
    assert all(t._version > v for t, v in zip([w, opt.grad_norm] + ([opt.masters[0]] if master else []), versions))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    (x @ w).sum().backward()  # and a new one is fine
    opt.step()


def test_backward_after_outputs_in_place_raises(dev):
    """The same for outputs that the caller gives: the residual stream updated in
    place, rows and gradients written into existing tensors."""
    import torch

    w = torch.ones(96, device=dev)
    ids = torch.tensor([1, 3, 1], device=dev)
    table = torch.randn(5, 96, device=dev)

    def in_place(call, out):
        p = torch.ones_like(out, requires_grad=True)
        y = p * out  # saves out
        call(out)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()

    y, h = torch.randn(3, 96, device=dev), torch.randn(3, 96, device=dev)
    in_place(lambda t: nq.residual_norm_forward(y, t, w, h_out=t), h.clone())
    in_place(lambda t: nq.residual_norm_forward(y, h, w, x_out=t), h.clone())
    in_place(lambda t: nq.embedding_forward(ids, table, out=t), h.clone())
    in_place(lambda t: nq.embedding_backward(ids, y, 5, grad=t), table.clone())
    with torch.inference_mode():  # tensors without a version
        t = h.clone()
        nq.residual_norm_forward(y, t, w, h_out=t, x_out=torch.empty_like(t))
        nq.embedding_forward(ids, table, out=t)
        nq.embedding_backward(ids, y, 5, grad=table.clone())


def test_second_derivatives_are_refused(dev):
    """The backward passes are kernels without a derivative of their own: asking for
    second derivatives raises instead of leaving terms out."""
    import torch

    def refused(out, t):
        g, = torch.autograd.grad(out.square().sum(), t, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            (g.square().sum() + t.square().sum()).backward()

    y, h = (torch.randn(3, 40, device=dev, requires_grad=True) for _ in range(2))
    w = torch.rand(40, device=dev) + 0.5
    refused(nq.residual_norm(y, h, w)[1], y)
    refused(nq.residual_norm(None, h, w)[1], h)
    table = torch.randn(7, 40, device=dev, requires_grad=True)
    refused(nq.nf4_embedding(torch.tensor([2, 2, 6], device=dev), table), table)


# ------------------------------------------------------------------ the optimizer's tensors

@pytest.mark.parametrize("bits", [8, 32])
def test_moments_are_replaced_by_bind_state_alone(dev, bits):
    """The step writes at the addresses that bind_state took: it refuses lists that hold
    other tensors, before it launches anything, and their memory stays the optimizer's
    for as long as it uses it. The lists themselves are saved like any others."""
    import torch

    names = ("m", "v") + (("m_scale", "v_scale") if bits == 8 else ())
    grads = [torch.ones(300, device=dev), torch.ones(20, device=dev)]

    def fresh():
        return nq.NF4AdamW([torch.zeros(300, device=dev), torch.zeros(20, device=dev)], state_bits=bits)

    def item(ts):
        ts[0] = ts[1] if ts[0] is None else ts[0].clone()

    def part(ts):
        ts[:] = [None if t is None else t.clone() for t in ts]
        ts[1] = grads[1]

    changes = (item, part, lambda ts: ts.append(grads[0]), lambda ts: ts.pop(), lambda ts: ts.clear(),
               lambda ts: ts.__setitem__(1, grads[1]))
    for name in names + ("params", "masters"):
        for k, change in enumerate(changes):
            if name == "masters" and k == 0:
                continue  # there are none
            opt = fresh()
            kept = list(opt.params) + list(opt.m)
            change(getattr(opt, name))
            with pytest.raises(ValueError, match=name):
                opt.step(grads)
            assert opt.steps == 0 and not any(bool(t.view(torch.uint8).any()) for t in kept)
            if name in names:
                opt.bind_state(*([t for t in fresh()._taken[n]] for n in names))
                opt.step(grads)
                assert bool(getattr(opt, name)[1].view(torch.uint8).any())
        with pytest.raises(AttributeError):
            setattr(opt, name, [])
    assert bits == 8 or not hasattr(opt, "m_scale")
    opt = fresh()
    held = {t.untyped_storage().data_ptr() for t in opt._held_state}
    assert {t.untyped_storage().data_ptr() for t in opt.m + opt.v} <= held
    file = io.BytesIO()
    opt.step(grads)
    torch.save([getattr(opt, n) for n in names], file)
    file.seek(0)
    saved = torch.load(file, weights_only=True)
    again = fresh()
    again.bind_state(*saved)
    assert all(torch.equal(s.view(torch.uint8), t.view(torch.uint8)) for s, t in zip(again.m + again.v, opt.m + opt.v))
    old = [t.view(torch.uint8).clone() for t in opt.m]
    kept = opt.m
    new = [[torch.zeros_like(t) for t in getattr(opt, n)] for n in names]
    opt.bind_state(*new)
    opt.step(grads)
    assert all(bool(t.view(torch.uint8).any()) for t in new[0]) and opt.m[0] is new[0][0]
    assert all(torch.equal(a, b.view(torch.uint8)) for a, b in zip(old, kept))


def test_weights_with_new_strides_are_refused(dev):
    """A weight that its own memory's transposed view replaces lies at the same
    address in another order; the step notices before it launches anything."""
    import torch

    p = torch.nn.Parameter(torch.randn(16, 16, device=dev).to(torch.bfloat16))
    master = torch.randn(16, 16, device=dev)
    for what in (p, master):
        opt = nq.NF4AdamW([p], masters=[master])
        g = torch.ones(16, 16, device=dev)
        opt.step([g])
        was, kept = p.data, [t.detach().clone() for t in (p, master)]
        what.data = what.data.t()
        with pytest.raises(ValueError, match="contiguous"):
            opt.step([g])
        what.data = what.data.t()
        assert opt.steps == 1 and all(torch.equal(a, b) for a, b in zip(kept, (p, master)))
        opt.step([g])
        assert not torch.equal(was, kept[0])


def test_tensors_that_share_memory_are_refused(dev):
    """Two workgroups may not update the same element: a tensor given twice, a tied
    weight in two groups, slices that overlap, shared moments. Neighbours in one
    buffer are fine."""
    import torch

    flat = torch.zeros(1024, device=dev)
    p, q = flat[:512], flat[512:]
    opt = nq.NF4AdamW([p, q, flat[512:512]])
    for bad in ([p, p], [p, p.view(32, 16)], [dict(params=[p]), dict(params=[q, p])], [p, flat[256:768]], [flat, q]):
        with pytest.raises(ValueError, match="share"):
            nq.NF4AdamW(bad)
    half = [torch.zeros(64, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    master = torch.zeros(64, device=dev)
    with pytest.raises(ValueError, match="share"):
        nq.NF4AdamW(half, masters=[master, master])
    with pytest.raises(ValueError, match="share"):
        nq.NF4AdamW(half[:1], masters=[master], state_bits=32).bind_state([master], [torch.zeros(64, device=dev)])
    opt = nq.NF4AdamW([p, q], state_bits=32)
    m, v = torch.zeros(1024, device=dev), torch.zeros(1024, device=dev)
    opt.bind_state([m[:512], m[512:]], [v[:512], v[512:]])
    for ms, vs in (([m[:512], m[:512]], [v[:512], v[512:]]), ([m[:512], m[512:]], [v[:512], m[512:]]),
                   ([p, m[512:]], [v[:512], v[512:]])):
        with pytest.raises(ValueError, match="share"):
            opt.bind_state(ms, vs)
        assert opt.m[0].data_ptr() == m.data_ptr() and opt.v[1].data_ptr() == v[512:].data_ptr()  # as it was
    a, b = torch.nn.Parameter(p.clone()), torch.nn.Parameter(q.clone())
    opt = nq.NF4AdamW([a, b])
    b.data = a.data
    with pytest.raises(ValueError, match="share"):
        opt.step([flat[:512].clone(), flat[:512].clone()])


def test_copies_are_refused(dev):
    """A copy would hold the addresses of the first one's tensors; state_dict is what
    carries a state."""
    import torch

    opt = nq.NF4AdamW([torch.zeros(64, device=dev)])
    for copied in (copy.copy, copy.deepcopy, pickle.dumps):
        with pytest.raises(TypeError, match="state_dict"):
            copied(opt)


# ------------------------------------------------------------------ the optimizer's state

def test_state_of_a_weight_without_dimensions(dev):
    """A bfloat16 weight of shape () with a master weight goes through state_dict."""
    import torch

    def fresh(x):
        half = dict(device=dev, dtype=torch.bfloat16)
        return nq.NF4AdamW([torch.tensor(x, **half), torch.full((3,), x, **half)], masters=True, lr=0.1)

    g = [torch.tensor(1.0, device=dev), torch.ones(3, device=dev)]
    a, b = fresh(1.0), fresh(2.0)
    a.step(g)
    b.load_state_dict(a.state_dict())
    a.step(g)
    b.step(g)
    for s, t in zip(a.masters + a.params, b.masters + b.params):
        assert torch.equal(s, t)


def test_states_with_parts_missing_are_refused(dev):
    """A state that lacks tensors of one of its lists is not loaded in part."""
    import torch

    opt, other = (nq.NF4AdamW([torch.ones(n, device=dev, dtype=torch.bfloat16) for n in (300, 40)], masters=True)
                  for _ in range(2))
    g = [torch.ones(300, device=dev), torch.ones(40, device=dev)]
    other.step(g)
    for name in ("m", "v", "m_scale", "v_scale", "masters"):
        for wrong in (lambda ts: ts[:1], lambda ts: ts + ts[:1]):
            d = other.state_dict()
            d[name] = wrong(d[name])
            with pytest.raises(ValueError, match="another optimizer"):
                opt.load_state_dict(d)
    assert opt.steps == 0 and not any(bool(t.view(torch.uint8).any()) for t in opt.m + opt.v)
    opt.load_state_dict(other.state_dict())
    assert opt.steps == 1 and bool(opt.m[1].view(torch.uint8).any())


def test_step_number_after_a_skipped_step(dev):
    """A step whose norm is not finite changes no tensor and still counts: the next
    one is step 2 to the bias corrections, unless the caller gives its own number."""
    import torch

    def run(bad_first, number):
        p = torch.zeros(300, device=dev)
        opt = nq.NF4AdamW([p], lr=0.5, weight_decay=0.0, state_bits=32, max_grad_norm=1e6)
        if bad_first:
            opt.step([torch.full((300,), float("inf"), device=dev)])
            assert opt.steps == 1 and not bool(p.any()) and not bool(opt.m[0].any())
        opt.step([torch.ones(300, device=dev)], step=number)
        return p, opt.steps

    skipped, steps = run(True, None)
    second, _ = run(False, 2)
    assert steps == 2 and torch.equal(skipped, second)
    given, steps = run(True, 1)
    first, _ = run(False, 1)
    assert steps == 1 and torch.equal(given, first)
    # (1 - b1) g / (1 - b1^2) over the root of (1 - b2) g^2 / (1 - b2^2), 24 U
    want = 0.5 * (0.1 / 0.19) / np.sqrt(0.001 / (1 - 0.999 ** 2))
    assert float((skipped + want).abs().max()) <= 32 * U * want


# ------------------------------------------------------------------ tables and outputs

def test_table_in_another_storage_format(dev):
    """Refused as a table: the message names the embedding and the format it takes."""
    import torch

    w = torch.randn(32, 128, device=dev).to(torch.bfloat16)
    ids = torch.tensor([1, 2], device=dev)
    for fmt in (nq.NF4Format(blocksize=128), nq.NF4Format(codebook="fp4"), nq.NF4Format(dq_format="e5m2")):
        t = nq.quantize(w, fmt=fmt)
        for call in (nq.embedding_forward, nq.nf4_embedding):
            with pytest.raises(ValueError, match="embedding") as e:
                call(ids, t)
            assert "linear" not in str(e.value)


def test_h_out_without_y_is_refused(dev):
    """Without y the stream stays as it is and nothing would be written to h_out."""
    import torch

    h = torch.randn(3, 40, device=dev)
    w = torch.ones(40, device=dev)
    with pytest.raises(ValueError, match="h_out"):
        nq.residual_norm_forward(None, h, w, h_out=torch.zeros_like(h))
    out, x, _, _ = nq.residual_norm_forward(None, h, w, h_out=h)  # the stream itself
    assert out is h
    assert nq.residual_norm_forward(None, h, w, h_out=h.view(3, 40))[0] is h
    assert nq.residual_norm_forward(None, h, w)[0] is h


def test_eps_among_the_subnormals(dev):
    """An eps below 2^-126 divides like any other: nothing moves where both moments are
    zero, and m / eps is m / eps where the second moment has left fp32 under the first."""
    import torch

    n = 400
    m0 = torch.zeros(n, device=dev)
    m0[::2] = torch.logspace(-36, -30, n // 2, device=dev)
    for eps in (2.0 ** -149, 1e-40, 1e-38, 2.0 ** -126):
        for bits in (8, 32):
            p = torch.full((n,), 0.5, device=dev)
            opt = nq.NF4AdamW([p], lr=1e-6, weight_decay=0.0, eps=eps, state_bits=bits)
            opt.step([torch.zeros(n, device=dev)])
            assert bool((p == 0.5).all()), (eps, bits)
        opt.bind_state([m0.clone()], [torch.zeros(n, device=dev)])
        opt.step([torch.zeros(n, device=dev)], step=100000)
        step = 1e-6 * 0.9 * m0.double() / float(np.float32(eps))
        want = 0.5 - step
        # 24 U of the step, the weight's rounding, and 2^-150 of m' over the eps
        tol = 26 * U * step + 2 * U * (0.5 + want.abs())
        big = step >= 2.0 ** 127
        assert bool((((p.double() - want).abs() <= tol) | big).all()), eps
        assert bool((p[1::2] == 0.5).all())
