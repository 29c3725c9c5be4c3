"""AdamW over a list of tensors (nf4_adamw_step, nf4_grad_norm) against the
formulas of nf4.h in 64 bits.

Tolerances, with u = 2^-24 and the terms' own size as the scale of each sum:
a moment is two products and a sum of fp32 values, its constants are rounded
once and the clipped gradient carries three roundings (8 u of |beta m| + |(1 -
beta) g|); the weight adds its decay (3 u of |w|) and a quotient whose root and
reciprocal are within 1 ulp each (24 u of lr / bias1 times the first moment's
terms over the denominator). A bfloat16 weight is then rounded once (2^-8).
8-bit codes are exact wherever the moment's own error cannot move it over the
place where the random bits round it."""
import numpy as np
import pytest

import nf4_quantize_amd as nq
from gpu_util import log

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TINY = 3 * 2.0 ** -149  # three roundings among fp32's smallest numbers, which are 2^-149 apart
M32 = np.uint64(0xFFFFFFFF)


def mix(x):
    x = x ^ (x >> np.uint64(16))
    x = x * np.uint64(0x6A09E667) & M32
    x = x ^ (x >> np.uint64(15))
    x = x * np.uint64(0xBB67AE85) & M32
    return x ^ (x >> np.uint64(16))


def random_bits(seed, entry, n):
    c = np.uint64(0x9E3779B9)
    with np.errstate(over="ignore"):
        key = mix(mix(np.uint64(entry) * c + np.uint64(seed >> 32) & M32) + np.uint64(seed & 0xFFFFFFFF) & M32)
        return mix(np.arange(n, dtype=np.uint64) * c + key & M32)


def blocks(x):
    """[blocks, 256] of a flat array, padded with zeros."""
    n = -(-x.size // 256) * 256
    return np.pad(x, (0, n - x.size)).reshape(-1, 256)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64).reshape(-1)


def e4m3_step(a):
    return np.exp2(np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)


def make(dev, shapes, wt, gt, bits, master, seed, **kw):
    import torch

    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    params = [torch.randn(s, generator=g, device=dev).mul_(0.02).to(wt) for s in shapes]
    masters = [p.float() + 1e-5 * torch.randn(p.shape, generator=g, device=dev) for p in params] if master else None
    grads = [torch.randn(s, generator=g, device=dev).mul_(0.01).to(gt) for s in shapes]
    opt = nq.NF4AdamW([dict(params=params[:1], lr=3e-3, weight_decay=0.1, masters=masters and masters[:1]),
                       dict(params=params[1:], lr=1e-3, weight_decay=0.0, masters=masters and masters[1:])],
                      state_bits=bits, seed=seed << 33, **kw)
    return opt, params, masters, grads


def reference_step(opt, i, w, m, v, grad, clip, number):
    """(w', m', v') in 64 bits, and the sizes of the moments' terms."""
    b1, b2 = opt.betas
    group = opt.groups[0] if i < opt.groups[0]["count"] else opt.groups[1]
    lr, wd = float(np.float32(group["lr"])), float(np.float32(group["weight_decay"]))
    g = grad * clip
    m1, v1 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    tm, tv = np.abs(b1 * m) + np.abs((1 - b1) * g), v1
    step, den = lr / (1 - b1 ** number), np.sqrt(v1 / (1 - b2 ** number)) + opt.eps
    return w * (1 - lr * wd) - step * m1 / den, m1, v1, tm, tv, step / den


def check_step(opt, before, grads, number, seed, clip):
    for i, (p, grad) in enumerate(zip(opt.params, grads)):
        master = opt.masters[i]
        w0, m0, v0 = before[i]
        w1, m1, v1, tm, tv, per = reference_step(opt, i, w0, m0, v0, f64(grad), clip, number)
        err_w = 3 * U * np.abs(w0) + 24 * U * per * tm + U * np.abs(w1)
        if master is not None:
            assert np.all(np.abs(f64(master) - w1) <= err_w), i
            assert bool((p == master.to(p.dtype)).all())
        half = 2.0 ** -8 if p.element_size() == 2 else 0.0
        assert np.all(np.abs(f64(p) - w1) <= err_w + half * (np.abs(w1) + err_w)), i
        if opt.state_bits == 32:
            assert np.all(np.abs(f64(opt.m[i]) - m1) <= 8 * U * tm), i
            assert np.all(np.abs(f64(opt.v[i]) - v1) <= 12 * U * tv + TINY), i
            continue
        r = random_bits(seed, i, m1.size)
        for name, x, t, bits in (("m", m1, tm, r >> np.uint64(16)), ("v", v1, tv, r & np.uint64(0xFFFF))):
            amax = np.abs(blocks(x)).max(1)
            scale = f64(getattr(opt, name + "_scale")[i])
            worst = 12 * U * blocks(t).max(1) / 448 + 2 * U * amax / 448
            assert np.all(np.abs(scale - amax / 448) <= worst), (i, name)
            s = np.repeat(scale, 256)[:x.size]
            live = s > 0
            q = np.where(live, x / np.where(live, s, 1.0), 0.0)
            dq = np.where(live, 12 * U * t / np.where(live, s, 1.0), 0.0) + 8 * U * np.abs(q)
            if name == "v":
                q = np.maximum(q, 2.0 ** -9)
            q = np.clip(q, -448, 448)
            got = f64(getattr(opt, name)[i])
            a = np.abs(q)
            step = e4m3_step(a)
            frac = bits.astype(np.float64) / 65536
            want = np.sign(q) * np.floor(a / step + frac) * step
            # the conversion cuts at 20 bits; near the place where it turns, either neighbour will do
            place = a / step + frac
            near = np.abs(place - np.round(place)) <= dq / step + 2.0 ** -19
            # a step's own edge, from the smallest normal code on
            near |= (np.abs(np.log2(np.maximum(a, 2.0 ** -7)) % 1.0 - 0.5) >= 0.5 - 1e-5) & (a > 0.99 * 2.0 ** -6)
            ok = (got == want) | (near & (np.abs(got - q) <= step * 2 + dq))
            assert ok.all(), (i, name, np.flatnonzero(~ok)[:5], got[~ok][:5], want[~ok][:5])
            assert near.mean() < 0.02 + 8 / x.size


SHAPES = [(1,), (7,), (8,), (255,), (256,), (257,), (2047,), (2048,), (2049,), (64, 33), (3, 5, 7), (4096, 16), (100003,)]


def snapshot(opt):
    import torch

    out = []
    for i, p in enumerate(opt.params):
        w = f64(p if opt.masters[i] is None else opt.masters[i])
        m, v = f64(opt.m[i]), f64(opt.v[i])
        if opt.state_bits == 8:
            m = m * np.repeat(f64(opt.m_scale[i]), 256)[:m.size]
            v = v * np.repeat(f64(opt.v_scale[i]), 256)[:v.size]
        out.append((w, m, v))
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("wt,gt,master", [("bfloat16", "bfloat16", False), ("bfloat16", "bfloat16", True),
                                          ("bfloat16", "float32", False), ("bfloat16", "float32", True),
                                          ("float32", "float32", False), ("float32", "bfloat16", False)])
def test_steps(dev, bits, wt, gt, master):
    import torch

    log(f"adamw bits={bits} w={wt} g={gt} master={master}")
    opt, params, masters, grads = make(dev, SHAPES, getattr(torch, wt), getattr(torch, gt), bits, master, 3,
                                       max_grad_norm=0.5)
    # one tensor without gradient, one block of zeros, tiny and large blocks, and a row at the clip's edge
    grads[5].zero_()
    grads[-1][512:768] = 0
    grads[-1][1024:1280] *= 1e-12
    grads[-1][1280:1536] *= 1e3
    for number in (1, 2, 3):
        before = snapshot(opt)
        opt.step(grads)
        torch.cuda.synchronize()
        norm = float(opt.grad_norm)
        want = np.sqrt(sum((f64(g) ** 2).sum() for g in grads))
        assert abs(norm - want) <= 2 * U * want
        check_step(opt, before, grads, number, opt.seed + number, min(1.0, 0.5 / norm))
        for g in grads:
            g.neg_().mul_(0.5)


@pytest.mark.parametrize("count", [1, 47, 48, 49, 130])
def test_many_tensors(dev, count):
    """More entries than one launch takes; empty tensors among them."""
    import torch

    log(f"adamw {count} tensors")
    sizes = [((i * 37) % 700,) for i in range(count)]
    sizes[0] = (300,)
    opt, params, masters, grads = make(dev, sizes, torch.float32, torch.float32, 8, False, 11)
    before = snapshot(opt)
    opt.step(grads)
    torch.cuda.synchronize()
    keep = [i for i, s in enumerate(sizes) if s[0]]
    assert len(keep) >= 1
    for i in range(count):
        if i not in keep:
            assert params[i].numel() == 0
    filled = [(w, m, v) for w, m, v in before]
    check_subset(opt, filled, grads, keep)


def check_subset(opt, before, grads, keep):
    class View:
        pass

    for i in keep:
        v = View()
        v.betas, v.eps, v.state_bits, v.groups = opt.betas, opt.eps, opt.state_bits, opt.groups
        w1, *_ = reference_step(opt, i, *before[i], f64(grads[i]), 1.0, 1)
        got = f64(opt.params[i])
        tm = np.abs(f64(grads[i])) * 0.1
        assert np.all(np.abs(got - w1) <= 1e-6 * (np.abs(before[i][0]) + np.abs(w1)) + 1e-8 + tm * 0), i
        r = random_bits(opt.seed + 1, i, got.size)
        m1 = (1 - 0.9) * f64(grads[i])
        s = np.repeat(f64(opt.m_scale[i]), 256)[:got.size]
        q = m1 / s
        step = e4m3_step(np.abs(q))
        place = np.abs(q) / step + (r >> np.uint64(16)).astype(np.float64) / 65536
        near = np.abs(place - np.round(place)) < 1e-4
        assert np.all((f64(opt.m[i]) == np.sign(q) * np.floor(place) * step) | near), i


def test_stochastic_rounding_has_no_bias(dev):
    """A constant moment, stored from 4096 seeds: the mean of the codes is the value
    (the variance of one rounding is at most a quarter of the step's square), the
    two moments' random bits are not correlated, and a seed gives the same codes
    again."""
    import torch

    n, runs = 256, 4096
    p = torch.zeros(n, device=dev)
    opt = nq.NF4AdamW([p], lr=0.0, weight_decay=0.0, betas=(0.0, 0.0), state_bits=8)
    g = torch.linspace(0.03, 1.0, n, device=dev)
    sm = torch.zeros(n, dtype=torch.float64, device=dev)
    sv, smv = torch.zeros_like(sm), torch.zeros_like(sm)
    for k in range(runs):
        opt.step([g], step=1, seed=k * 977 + (k << 40))
        m = opt.m[0].double() * opt.m_scale[0].double()
        v = opt.v[0].double() * opt.v_scale[0].double()
        sm += m
        sv += v
        smv += (m - g.double()) * (v - g.double() ** 2)
        if k == 5:
            first = opt.m[0].view(torch.uint8).clone(), opt.v[0].view(torch.uint8).clone()
    opt.step([g], step=1, seed=5 * 977 + (5 << 40))
    assert torch.equal(first[0], opt.m[0].view(torch.uint8)) and torch.equal(first[1], opt.v[0].view(torch.uint8))
    steps = {}
    for name, total, x in (("m", sm, g.double()), ("v", sv, (g * g).double())):
        scale = float(getattr(opt, name + "_scale")[0])
        q = (x / scale).cpu().numpy()
        step = torch.from_numpy(e4m3_step(q) * scale).to(dev)
        steps[name] = step
        err = (total / runs - x).abs()
        assert bool((err <= 6 * 0.5 * step / np.sqrt(runs) + 2.0 ** -16 * step).all()), name
    cov = (smv / runs).abs()
    assert bool((cov <= 6 * 0.25 * steps["m"] * steps["v"] / np.sqrt(runs)).all())


def test_second_moment_stays_above_zero(dev):
    """Where a first moment is stored, the second one's code is not zero: the step
    after a block's largest gradient stops stays within the learning rate's size."""
    import torch

    n = 512
    p = torch.zeros(n, device=dev)
    opt = nq.NF4AdamW([p], lr=1e-3, weight_decay=0.0)
    g = torch.full((n,), 1e-9, device=dev)
    g[::256] = 1.0
    for _ in range(20):
        opt.step([g])
    assert bool((opt.v[0].view(torch.uint8) > 0).all())
    assert float(p.abs().max()) <= 20 * 1e-3 * 1.5


def test_norm_not_finite_changes_nothing(dev):
    import torch

    for bad in (float("inf"), float("nan")):
        for bits in (8, 32):
            opt, params, masters, grads = make(dev, [(1000,), (300,)], torch.bfloat16, torch.bfloat16, bits, True, 5,
                                               max_grad_norm=1.0)
            opt.step(grads)
            saved = [t.clone() for t in params + masters + [t.view(torch.uint8) for t in opt.m + opt.v]]
            grads[1][7] = bad
            opt.step(grads)
            now = params + masters + [t.view(torch.uint8) for t in opt.m + opt.v]
            assert not np.isfinite(float(opt.grad_norm))
            assert all(torch.equal(a, b) for a, b in zip(saved, now))


@pytest.mark.parametrize("gt", ["bfloat16", "float32"])
def test_norm_sizes(dev, gt):
    """One element to many chunks; squares that underflow or overflow in fp32; the
    same bits again."""
    import torch

    for sizes, scale in (([1], 1.0), ([16383, 16384, 16385], 1e-25), ([5] * 300, 1e18), ([3_000_001, 8], 1.0)):
        log(f"grad norm {len(sizes)} tensors {gt} scale {scale}")
        opt, params, masters, grads = make(dev, [(n,) for n in sizes] + [(1,)], torch.float32, getattr(torch, gt), 32,
                                           False, 9, max_grad_norm=1.0)
        for g in grads:
            g.mul_(100 * scale)
        opt.step(grads)
        want = np.sqrt(sum((f64(g) ** 2).sum() for g in grads))
        got = float(opt.grad_norm)
        assert abs(got - want) <= 2 * U * want
        opt.step(grads)
        assert float(opt.grad_norm) == got


def test_neighbours_are_not_touched(dev):
    """Ragged tensors inside larger buffers: what surrounds them keeps its bytes."""
    import torch

    for n in (1, 9, 250, 257, 2050):
        for bits in (8, 32):
            log(f"adamw guards n={n} bits={bits}")
            big = {k: torch.full((64 + -(-n // 256) * 256 + 512,), 0x5A, dtype=torch.uint8, device=dev).repeat_interleave(4)
                   for k in ("w", "m", "v", "ms", "vs")}

            def view(k, dt, count):
                return big[k].view(dt)[64:64 + count]

            dt = torch.float8_e4m3fn if bits == 8 else torch.float32
            p = view("w", torch.bfloat16, n)
            m, v = view("m", dt, n), view("v", dt, n)
            scales = [view(k, torch.float32, -(-n // 256)) for k in ("ms", "vs")]
            for t in [p, m, v] + scales:
                t.view(torch.uint8).zero_()
            opt = nq.NF4AdamW([p], state_bits=bits)
            opt.bind_state([m], [v], *([[s] for s in scales] if bits == 8 else []))
            opt.step([torch.ones(n, device=dev, dtype=torch.bfloat16)])
            torch.cuda.synchronize()
            for k, t in (("w", p), ("m", m), ("v", v), ("ms", scales[0]), ("vs", scales[1])):
                raw = big[k].cpu().numpy()
                size = t.element_size()
                a, b = 64 * size, 64 * size + t.numel() * size
                assert (raw[:a] == 0x5A).all() and (raw[b:] == 0x5A).all(), k


def test_state_round_trip(dev):
    """A restored optimizer takes the same steps bit for bit."""
    import torch

    for bits in (8, 32):
        opt, params, masters, grads = make(dev, [(1000,), (64, 20)], torch.bfloat16, torch.bfloat16, bits, True, 21)
        opt.step(grads)
        saved, weights = opt.state_dict(), [p.clone() for p in params]
        opt.step(grads)
        again, p2, m2, _ = make(dev, [(1000,), (64, 20)], torch.bfloat16, torch.bfloat16, bits, True, 1)
        for p, w in zip(p2, weights):
            p.copy_(w)
        again.load_state_dict(saved)
        again.step(grads)
        for a, b in zip(params + opt.m + opt.v + masters, p2 + again.m + again.v + m2):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        with pytest.raises(ValueError):
            nq.NF4AdamW([params[0]], state_bits=bits).load_state_dict(saved)


def test_refuses_gradients_that_do_not_fit(dev):
    import torch

    p = torch.zeros(16, 16, device=dev)
    opt = nq.NF4AdamW([p, p.clone()])
    good = torch.zeros(16, 16, device=dev)
    for bad in ([good], [good, None], [good, good.bfloat16()], [good, good[:8]], [good, good.t()[:, :8].t()[:8]],
                [good, good.cpu()], [good, torch.zeros(16, 32, device=dev)[:, ::2]]):
        with pytest.raises(ValueError):
            opt.step(bad)
    with pytest.raises(nq.NF4Error):
        opt.step([good, torch.zeros(257, device=dev)[1:].view(16, 16)])  # not 16-byte aligned
    with pytest.raises(ValueError):
        opt.step()  # no .grad


def test_parameters_with_new_memory(dev):
    """A parameter whose data has been replaced is updated where it now lies; one
    of another type or size is refused."""
    import torch

    p = torch.nn.Parameter(torch.ones(700, device=dev))
    opt = nq.NF4AdamW([p], lr=0.5, weight_decay=0.0, state_bits=32)
    old = p.data
    p.data = torch.full((700,), 2.0, device=dev)
    opt.step([torch.ones(700, device=dev)])
    assert torch.equal(old, torch.ones_like(old))
    # first step with g = 1: m / (1 - beta1) = 1 and sqrt(v / (1 - beta2)) = 1, each
    # within a few roundings, so the weight moves by lr
    assert float((p.data - 1.5).abs().max()) < 1e-5
    kept = p.data.clone()
    p.data = kept.bfloat16()
    with pytest.raises(TypeError):
        opt.step([torch.ones(700, device=dev)])
    p.data = kept[:600].clone()
    with pytest.raises(ValueError):
        opt.step([torch.ones(600, device=dev)])
    with pytest.raises(ValueError):
        opt.step([torch.ones(700, device=dev)])


@pytest.mark.parametrize("bits,wt,gt", [(8, "bfloat16", "bfloat16"), (8, "float32", "float32"),
                                        (32, "bfloat16", "float32"), (32, "float32", "bfloat16")])
@pytest.mark.parametrize("case", ["one", "ragged", "sixteen", "seventeen", "large", "masters", "some masters", "empty", "chunks", "chunks of 48",
                                  "chunks of 49", "chunks masters", "chunks some masters"])
def test_clip_step_is_norm_then_step(dev, bits, wt, gt, case):
    """One call against the two that it stands for, bit for bit. The gradients are
    small multiples of 2^-6, so their squares add up without rounding in any order
    and the norms are equal."""
    import ctypes

    import torch
    from nf4_quantize_amd import training

    sizes = {"one": [1], "ragged": [7, 513, 2049, 1, 8191], "sixteen": [1030] * 16, "seventeen": [1030] * 17,
             "large": [131072, 9], "masters": [700, 3000], "some masters": [700, 3000, 5], "empty": [0, 600, 0],
             "chunks": [200_001, 7, 16384, 16385], "chunks of 48": [5000] * 48, "chunks of 49": [5000] * 49,
             "chunks masters": [140_000, 3], "chunks some masters": [140_000, 3000, 5]}[case]
    master = case.endswith("masters")
    if master and wt != "bfloat16":
        pytest.skip("masters are of bfloat16 weights")
    log(f"clip step {case} {bits} bits {wt} {gt}")
    rng = np.random.default_rng(len(sizes) + bits)
    start = [torch.from_numpy(rng.standard_normal(n).astype(np.float32)).to(dev) for n in sizes]
    grads = [torch.from_numpy(rng.integers(-16, 17, n).astype(np.float32) / 64).to(dev).to(getattr(torch, gt)) for n in sizes]
    got = []
    for one_call in (True, False):
        ps = [s.clone().to(getattr(torch, wt)) for s in start]
        ms = [s.clone() if master and not ("some" in case and i == 1) else None for i, s in enumerate(start)]
        opt = nq.NF4AdamW(ps, lr=1e-2, state_bits=bits, masters=ms if master else None, max_grad_norm=0.25, seed=3)
        for number in (1, 2):
            if one_call:
                opt.step(grads)
                continue
            L, e = nq.lib(), opt._entries
            e["grad"], e["lr"], e["weight_decay"] = [g.data_ptr() for g in grads], 1e-2, 0.01
            cfg = training.nf4_adamw_config(0.9, 0.999, 1e-8, 0.25, number, 3 + number)
            ws, stream = opt._workspace, torch.cuda.current_stream().cuda_stream
            code = {"float32": 0, "bfloat16": 1}
            assert L.nf4_grad_norm(e.ctypes.data, len(e), code[gt], opt.grad_norm.data_ptr(), ws.data_ptr(), ws.numel(),
                                   stream) == 0
            assert L.nf4_adamw_step(e.ctypes.data, len(e), code[wt], code[gt], bits, ctypes.byref(cfg),
                                    opt.grad_norm.data_ptr(), ws.data_ptr(), ws.numel(), stream) == 0
        parts = ps + [t for t in ms if t is not None] + opt.m + opt.v + ([] if bits == 32 else opt.m_scale + opt.v_scale)
        got.append([opt.grad_norm.clone()] + [t.clone() for t in parts])
    want = np.float32(np.sqrt(sum((f64(g) ** 2).sum() for g in grads)))
    assert float(got[0][0]) == want
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(*got) if a.numel())


def test_rates_change_between_steps(dev):
    """lr and weight_decay of a group are those of the step's time."""
    import torch

    p = torch.zeros(300, device=dev)
    opt = nq.NF4AdamW([dict(params=[p], lr=0.25, weight_decay=0.0)], state_bits=32)
    g = torch.ones(300, device=dev)
    want = 0.0
    for lr in (0.25, 0.25, 0.5, 0.125):
        opt.groups[0]["lr"] = lr
        opt.step([g])
        want -= lr  # constant gradients: m / (1 - beta1^t) = g and v / (1 - beta2^t) = g^2 up to rounding
        assert float((p - want).abs().max()) < 1e-5
    opt.groups[0].update(lr=0.5, weight_decay=0.5)
    opt.step([g])
    assert float((p - (want * 0.75 - 0.5)).abs().max()) < 1e-5
