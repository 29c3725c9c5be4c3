"""AdamW over lists that go through the workspace's table (more than 48 tensors of
a kind), with bfloat16 weights, master weights for all or some and clipping, and
with the kernels that a small eps takes. The
weights are compared with the formulas in 64 bits (test_gpu_adamw.py has the
tolerances); the moments, their scales and their codes are defined to the bit by
fp32 operations (nf4.h) and have to be equal."""
import numpy as np
import pytest

import nf4_quantize_amd as nq
from gpu_util import log
from test_gpu_adamw import U, blocks, f64, make, random_bits, reference_step, snapshot

pytestmark = pytest.mark.gpu

F = np.float32


def f32(t):
    return t.detach().float().cpu().numpy().reshape(-1)


def moments32(m, v, grad, clip):
    """The moments' update, product by product in fp32."""
    g = grad * clip
    m = F(0.9) * m + F(1.0 - 0.9) * g
    return m, F(0.999) * v + F(1.0 - 0.999) * (g * g)


def stored(x, least, bits16, second):
    """(scales, codes' values) of the 8-bit storage of fp32 x; `least`: a block's
    scale where its own would be below 2^-126."""
    scale = np.abs(blocks(x)).max(1) * F(1.0 / 448.0)
    scale = np.where(scale < F(2.0 ** -126), least, scale).astype(F)
    with np.errstate(divide="ignore"):
        inv = np.where(scale > 0, F(1.0) / scale, F(0.0)).astype(F)
    t = np.clip(x * np.repeat(inv, 256)[:x.size], F(2.0 ** -9) if second else F(-448.0), F(448.0))
    a = np.abs(t).astype(np.float64)
    step = np.exp2(np.maximum(np.frexp(a)[1] - 1, -6) - 3.0)
    # the conversion adds 20 random bits below the kept ones, here the upper 16 of them, and cuts
    return scale, np.sign(t) * np.floor(a / step + bits16 / 65536.0) * step


@pytest.mark.parametrize("count,eps", [(48, 1e-8), (49, 1e-8), (97, 1e-8), (448, 1e-8), (3, 0.0), (48, 0.0), (97, 0.0)])
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("wt,gt,master", [("bfloat16", "bfloat16", "none"), ("bfloat16", "bfloat16", "all"),
                                          ("bfloat16", "float32", "some"), ("float32", "bfloat16", "none")])
def test_steps(dev, count, eps, bits, wt, gt, master):
    import torch

    log(f"adamw list of {count}, eps {eps}, {bits} bits, {wt} {gt}, masters {master}")
    shapes = [(1 + (i * 157) % 900,) for i in range(count)]
    shapes[count // 2] = (5003,)  # more than a workgroup's share
    opt, params, masters, grads = make(dev, shapes, getattr(torch, wt), getattr(torch, gt), bits, master != "none", 17,
                                       max_grad_norm=0.5, eps=eps)
    if master == "some":
        keep = [None if i % 3 == 1 else t for i, t in enumerate(masters)]
        opt = nq.NF4AdamW([dict(params=params[:1], lr=3e-3, weight_decay=0.1, masters=keep[:1]),
                           dict(params=params[1:], lr=1e-3, weight_decay=0.0, masters=keep[1:])],
                          state_bits=bits, seed=17 << 33, max_grad_norm=0.5, eps=eps)
    for number in (1, 2):
        before = snapshot(opt)
        opt.step(grads)
        norm = float(opt.grad_norm)
        want = np.sqrt(sum((f64(g) ** 2).sum() for g in grads))
        assert abs(norm - want) <= 2 * U * want
        assert norm > 0.5  # clips
        clip = F(0.5) * (F(1.0) / F(norm))
        unclear = total = 0
        for i, (p, grad) in enumerate(zip(opt.params, grads)):
            w0, m0, v0 = before[i]
            w1, _, _, tm, _, per = reference_step(opt, i, w0, m0, v0, f64(grad), 0.5 / norm, number)
            err = 3 * U * np.abs(w0) + 24 * U * per * tm + U * np.abs(w1)
            if opt.masters[i] is not None:
                assert np.all(np.abs(f64(opt.masters[i]) - w1) <= err), i
                assert bool((p == opt.masters[i].to(p.dtype)).all()), i
            half = 2.0 ** -8 if p.element_size() == 2 else 0.0
            assert np.all(np.abs(f64(p) - w1) <= err + half * (np.abs(w1) + err)), i
            m, v = moments32(m0.astype(F), v0.astype(F), f32(grad), clip)
            if bits == 32:
                assert np.array_equal(f32(opt.m[i]), m) and np.array_equal(f32(opt.v[i]), v), i
                continue
            r = random_bits(opt.seed + number, i, m.size)
            ms, mq = stored(m, F(0.0), (r >> np.uint64(16)).astype(np.float64), False)
            vs, vq = stored(v, np.where(ms > 0, F(2.0 ** -126), F(0.0)), (r & np.uint64(0xFFFF)).astype(np.float64), True)
            for name, scale, codes in (("m", ms, mq), ("v", vs, vq)):
                assert np.array_equal(f32(getattr(opt, name + "_scale")[i]), scale), (i, name)
                differ = f64(getattr(opt, name)[i]) != codes
                # below 2^-6 the conversion may drop bits of t under its 20: one code, seldom
                assert not np.any(differ & (np.abs(codes) > 2.0 ** -6)), (i, name, np.flatnonzero(differ)[:5])
                assert np.all(np.abs(f64(getattr(opt, name)[i]) - codes)[differ] <= 2.0 ** -9), (i, name)
                unclear += int(differ.sum())
                total += differ.size
        assert unclear <= 2 + total * 2.0 ** -19
        for g in grads:
            g.neg_()
