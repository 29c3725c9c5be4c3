"""Muon's calls beside each other: two optimizers on two streams at once, one
update that a list has twice, masters of some matrices. All give the bits of the
calls by themselves."""
import pytest

pytestmark = pytest.mark.gpu

SHAPES = [(64, 1500), (777, 33), (9, 50), (700, 130), (256, 300)]


def optimizer(nq, dev, seed, dt):
    import torch

    g = torch.Generator().manual_seed(seed)
    ps = [torch.randn(s, generator=g).to(dev, dt) for s in SHAPES]
    grads = [[torch.randn(s, generator=g).to(dev, dt) for s in SHAPES] for _ in range(3)]
    return nq.NF4Muon(ps, lr=0.01, masters=dt == torch.bfloat16 or None), grads


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
def test_two_optimizers_at_once(dev, dt):
    import torch

    import nf4_quantize_amd as nq

    dt = getattr(torch, dt)
    want = []
    for seed in (1, 2):
        o, grads = optimizer(nq, dev, seed, dt)
        for g in grads:
            o.step(g)
        torch.cuda.synchronize()
        want.append([t.clone() for t in o.params + o.m])
    both = [optimizer(nq, dev, seed, dt) for seed in (1, 2)]
    streams = [torch.cuda.Stream() for _ in both]
    torch.cuda.synchronize()
    for k in range(3):
        for (o, grads), s in zip(both, streams):
            with torch.cuda.stream(s):
                o.step(grads[k])
    torch.cuda.synchronize()
    for (o, _), w in zip(both, want):
        assert all(torch.equal(x, y) for x, y in zip(o.params + o.m, w))


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
def test_one_update_twice(dev, dt):
    import torch

    import nf4_quantize_amd as nq

    g = torch.Generator().manual_seed(3)
    us = [torch.randn(s, generator=g).to(dev, getattr(torch, dt)) for s in SHAPES]
    kept = [u.clone() for u in us]
    first = nq.orthogonalize(us + us)
    n = len(us)
    assert all(torch.equal(x, y) for x, y in zip(first[:n], first[n:]))
    outs = [torch.empty_like(u) for u in us + us]
    given = nq.orthogonalize(us + us, outs=outs)
    assert all(x is y for x, y in zip(given, outs)) and all(torch.equal(x, y) for x, y in zip(given, first))
    assert all(torch.equal(u, k) for u, k in zip(us, kept))
    # as its own output and read for another: refused, nothing is written
    with pytest.raises(ValueError, match="share memory"):
        nq.orthogonalize([us[0], us[0]], outs=[us[0], torch.empty_like(us[0])])
    assert torch.equal(us[0], kept[0])


def test_masters_of_some(dev):
    """A first step rounds the same fp32 weight whether or not it is kept as a master."""
    import torch

    import nf4_quantize_amd as nq

    g = torch.Generator().manual_seed(4)
    start = [torch.randn(s, generator=g).to(dev, torch.bfloat16) for s in SHAPES]
    grads = [torch.randn(s, generator=g).to(dev, torch.bfloat16) for s in SHAPES]

    def step(groups):
        ps = [x.clone() for x in start]
        o = nq.NF4Muon([dict(params=ps[a:b], lr=0.01, weight_decay=0.1, masters=m) for a, b, m in groups])
        o.step(grads)
        return o

    n = len(start)
    every = step([(0, n, True)])
    for cut in (1, 3):
        for first in (True, None):
            some = step([(0, cut, first), (cut, n, None if first else True)])
            assert all(torch.equal(x, y) for x, y in zip(some.params, every.params))
            assert all(torch.equal(x, y) for x, y in zip(some.m, every.m))
            kept = [m is not None for m in some.masters]
            assert kept == [(i < cut) == bool(first) for i in range(n)]
            assert all(torch.equal(x, y) for x, y in zip(some.masters, every.masters) if x is not None)
