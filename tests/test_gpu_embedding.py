"""The token embedding (nf4_embedding_forward, its NF4 form, nf4_embedding_backward).

The forward is one product in fp32 and one rounding: equal bit for bit to the
same in torch. A row's gradient is an fp32 sum of its tokens' terms, each with
one more rounding by the scale: (count + 2) u of the sum of their magnitudes,
u = 2^-24, and 2^-8 of itself in bfloat16."""
import numpy as np
import pytest

import nf4_quantize_amd as nq
from gpu_util import log

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def draw(dev, kind, tokens, vocab, seed=0):
    import torch

    g = torch.Generator(device=dev)
    g.manual_seed(seed + tokens * 7 + vocab)
    if kind == "one":
        return torch.full((tokens,), vocab // 2, device=dev)
    if kind == "none":
        return torch.full((tokens,), -1, device=dev)
    if kind == "descending":
        return (torch.arange(tokens, device=dev).flip(0) * 3) % vocab
    ids = torch.randint(0, vocab, (tokens,), generator=g, device=dev)
    if kind == "few":                 # most of the batch is three ids, some places are empty or out of range
        r = torch.rand(tokens, generator=g, device=dev)
        ids = torch.where(r < 0.6, torch.randint(0, min(3, vocab), (tokens,), generator=g, device=dev), ids)
        ids = torch.where(r > 0.97, torch.full_like(ids, -1), ids)
        ids = torch.where(r > 0.985, torch.full_like(ids, vocab), ids)
        ids = torch.where(r > 0.995, torch.full_like(ids, (1 << 31) - 1), ids)
    return ids


@pytest.mark.parametrize("dim", [1, 3, 8, 63, 64, 250, 2048, 2049, 5000])
@pytest.mark.parametrize("types", [("bfloat16", "bfloat16"), ("bfloat16", "float32"), ("float32", "bfloat16"),
                                   ("float32", "float32")])
def test_lookup(dev, dim, types):
    import torch

    dt, od = (getattr(torch, t) for t in types)
    vocab = 301
    table = torch.randn(vocab, dim, device=dev).to(dt)
    for tokens, it in ((0, torch.int64), (1, torch.int32), (5, torch.int64), (1037, torch.int32)):
        log(f"lookup {tokens} of {vocab}x{dim} {types}")
        ids = draw(dev, "few", tokens, vocab).to(it)
        got = nq.embedding_forward(ids, table, scale=1.7, out_dtype=od)
        inside = (ids >= 0) & (ids < vocab)
        want = (table.float()[ids.long().clamp(0, vocab - 1)] * 1.7) * inside.unsqueeze(1)
        assert torch.equal(got, want.to(od))


@pytest.mark.parametrize("dim", [64, 128, 192, 2048, 4160])
@pytest.mark.parametrize("dq", [True, False])
def test_lookup_packed(dev, dim, dq):
    import torch

    vocab = 259
    w = torch.randn(vocab, dim, device=dev).mul_(0.02).to(torch.bfloat16)
    w[3] = 0
    t = nq.quantize(w, double_quant=dq)
    full = nq.dequantize(t, torch.float32)
    for tokens, od in ((1, torch.bfloat16), (7, torch.float32), (600, torch.bfloat16)):
        log(f"packed lookup {tokens} of {vocab}x{dim} dq={dq}")
        ids = draw(dev, "few", tokens, vocab)
        inside = (ids >= 0) & (ids < vocab)
        want = (full[ids.clamp(0, vocab - 1)] * 8.0) * inside.unsqueeze(1)
        assert torch.equal(nq.embedding_forward(ids, t, scale=8.0, out_dtype=od), want.to(od))
        assert torch.equal(nq.nf4_embedding(ids.view(1, -1), t, 8.0, out_dtype=od)[0], want.to(od))


def check_gradient(ids, dy, vocab, scale, grad0, got, padding=None):
    import torch

    inside = (ids >= 0) & (ids < vocab)
    if padding is not None:
        inside &= ids != padding
    # on the host, where many equal ids cost nothing
    at, rows = ids[inside].cpu(), dy[inside].double().cpu() * scale
    want = torch.zeros(vocab, dy.shape[1], dtype=torch.float64).index_add_(0, at, rows)
    size = torch.zeros_like(want).index_add_(0, at, rows.abs()).to(dy.device)
    count = torch.bincount(at, minlength=vocab).double().unsqueeze(1).to(dy.device)
    want = want.to(dy.device)
    if grad0 is not None:
        want += grad0.double()
        size += grad0.double().abs()
    tol = (count + 3) * U * size + (2.0 ** -8 if got.dtype == torch.bfloat16 else U) * want.abs()
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), (float(err.max()), torch.nonzero(err > tol)[:3].tolist())
    untouched = (count == 0).squeeze(1)
    if grad0 is None:
        assert not bool(got[untouched].any())
    else:
        assert torch.equal(got[untouched], grad0[untouched])


SIZES = [(0, 5, 8), (1, 1, 1), (1, 100, 64), (15, 7, 9), (16, 7, 512), (17, 3, 513), (33, 1000, 65), (255, 40, 130),
         (1000, 129, 1030), (4096, 50, 72), (8192, 3000, 24), (8193, 3000, 24), (20000, 70000, 16), (100001, 33, 12),
         (70000, 1025, 8), (30000, 2000000, 8)]


@pytest.mark.parametrize("tokens,vocab,dim", SIZES)
@pytest.mark.parametrize("kind", ["few", "one", "descending", "none"])
def test_gradient(dev, tokens, vocab, dim, kind):
    import torch

    ids = draw(dev, kind, tokens, vocab)
    base = torch.randn(tokens, dim, device=dev)
    for dt, gd, acc, it in ((torch.bfloat16, torch.bfloat16, False, torch.int64), (torch.float32, torch.float32, True, torch.int64),
                            (torch.bfloat16, torch.float32, False, torch.int32)):
        log(f"embedding gradient {tokens} tokens {vocab}x{dim} {kind} {dt} {gd} acc={acc}")
        dy = base.to(dt)
        grad0 = torch.randn(vocab, dim, device=dev).to(gd) if acc else None
        i = ids.to(it)
        got = nq.embedding_backward(i, dy, vocab, 1.5, grad=None if grad0 is None else grad0.clone(), grad_dtype=gd)
        again = nq.embedding_backward(i, dy, vocab, 1.5, grad=None if grad0 is None else grad0.clone(), grad_dtype=gd)
        check_gradient(ids, dy, vocab, 1.5, grad0, got)
        assert torch.equal(got, again)


def test_padding_and_autograd(dev):
    """The autograd function: the gradient of the table through a loss, none for the
    padding id, ids of any shape; and a difference of the loss along a direction
    (it is linear in the table, so the difference is exact up to fp32 sums)."""
    import torch

    vocab, dim = 97, 40
    table = torch.randn(vocab, dim, device=dev).requires_grad_()
    ids = draw(dev, "few", 120, vocab).view(4, 30)
    out = nq.nf4_embedding(ids, table, 2.0, padding_id=1)
    assert out.shape == (4, 30, dim)
    up = torch.randn_like(out)
    (out * up).sum().backward()
    check_gradient(ids.reshape(-1), up.view(-1, dim), vocab, 2.0, None, table.grad, padding=1)
    assert not bool(table.grad[1].any())
    direction = torch.randn_like(table)
    direction[1] = 0
    with torch.no_grad():
        a, b = ((nq.nf4_embedding(ids, table + s * direction, 2.0).double() * up.double()).sum() for s in (1.0, -1.0))
    want = float((table.grad.double() * direction.double()).sum())
    assert abs(float(a - b) / 2 - want) <= 1e-5 * float((table.grad.double() * direction.double()).abs().sum())


def test_gradient_guards(dev):
    """Rows of odd width inside a larger buffer: what surrounds the gradient keeps its
    bytes."""
    import torch

    for tokens, vocab, dim in ((50, 13, 7), (900, 100, 515)):
        for gd in (torch.bfloat16, torch.float32):
            ids = draw(dev, "few", tokens, vocab)
            dy = torch.randn(tokens, dim, device=dev)
            n = vocab * dim
            big = torch.full((n + 128,), 7.0, dtype=gd, device=dev)
            view = big[64:64 + n].view(vocab, dim)
            L = nq.lib()
            ws = torch.empty(L.nf4_embedding_backward_workspace_size(tokens, vocab, dim), dtype=torch.uint8, device=dev)
            st = L.nf4_embedding_backward(ids.data_ptr(), 1, tokens, dy.data_ptr(), 0, vocab, dim, 1.0, -1, view.data_ptr(),
                                          0 if gd == torch.float32 else 1, 0, ws.data_ptr(), ws.numel(),
                                          torch.cuda.current_stream().cuda_stream)
            assert st == 0
            check_gradient(ids, dy, vocab, 1.0, None, view)
            assert bool((big[:64] == 7).all()) and bool((big[64 + n:] == 7).all())


def test_large_offsets(dev):
    """A table and a gradient of more than 2^32 bytes and 2^31 elements."""
    import torch

    vocab, dim = 300_000, 8192
    table = torch.zeros(vocab, dim, dtype=torch.bfloat16, device=dev)
    ids = torch.tensor([vocab - 1, 0, 262_144, vocab - 1, 262_143], device=dev)
    table[ids] = torch.randn(5, dim, device=dev).to(torch.bfloat16)
    assert torch.equal(nq.embedding_forward(ids, table, 2.0), (table[ids].float() * 2).to(torch.bfloat16))
    dy = torch.randn(5, dim, device=dev).to(torch.bfloat16)
    table.fill_(3.0)
    grad = nq.embedding_backward(ids, dy, vocab, grad=None)
    rows = dy.double()
    want = {vocab - 1: rows[0] + rows[3], 0: rows[1], 262_144: rows[2], 262_143: rows[4]}
    for row, w in want.items():
        assert bool(((grad[row].double() - w).abs() <= 2.0 ** -7 * (w.abs() + 1e-6)).all())
    keep = torch.ones(vocab, dtype=torch.bool, device=dev)
    keep[ids] = False
    assert int(torch.count_nonzero(grad.view(torch.int16).view(vocab, dim)[keep].sum(1))) == 0


def test_refusals_on_device(dev):
    import torch

    ids = torch.zeros(3, dtype=torch.int64, device=dev)
    table = torch.zeros(5, 8, device=dev)
    with pytest.raises(ValueError):
        nq.embedding_forward(ids, table.t())
    with pytest.raises(TypeError):
        nq.embedding_forward(ids.to(torch.int16), table)
    with pytest.raises(ValueError):
        nq.embedding_forward(ids, table, out=torch.zeros(3, 9, device=dev))
    with pytest.raises(ValueError):
        nq.embedding_backward(ids, torch.zeros(3, 8, device=dev), 5, grad=torch.zeros(4, 8, device=dev))
    with pytest.raises(nq.NF4Error):
        nq.embedding_backward(ids, torch.zeros(3, 8, device=dev), 5, workspace=torch.zeros(8, dtype=torch.uint8, device=dev))


@pytest.mark.parametrize("tokens", [1, 2, 63, 64, 65, 127, 128, 129, 130])
@pytest.mark.parametrize("vocab,dim", [(1, 1), (3, 7), (40, 8), (300, 511), (2100, 513), (37, 4100)])
@pytest.mark.parametrize("kind", ["few", "one", "descending", "none"])
def test_gradient_of_few_tokens(dev, tokens, vocab, dim, kind):
    """Around the sizes that one launch takes, into memory that holds NaN where the
    call writes every row, with padding, and with bytes around the gradient."""
    import torch
    from nf4_quantize_amd import training

    log(f"embedding gradient of few tokens {tokens} {vocab}x{dim} {kind}")
    ids = draw(dev, kind, tokens, vocab, seed=tokens)
    L, pad = nq.lib(), 64
    for dt, gd, acc in ((torch.bfloat16, torch.float32, 0), (torch.float32, torch.bfloat16, 1), (torch.bfloat16, torch.bfloat16, 0)):
        dy = torch.randn(tokens, dim, device=dev).to(dt)
        buf = torch.full((pad + vocab * dim + pad,), 7.0, device=dev, dtype=gd)
        grad = buf[pad:pad + vocab * dim].view(vocab, dim)
        grad0 = torch.randn(vocab, dim, device=dev).to(gd) if acc else None
        grad.copy_(grad0) if acc else grad.fill_(float("nan"))
        padding = int(ids[0]) if 0 <= int(ids[0]) < vocab and tokens > 1 else -1
        ws = torch.empty(L.nf4_embedding_backward_workspace_size(tokens, vocab, dim), dtype=torch.uint8, device=dev)
        assert L.nf4_embedding_backward(ids.data_ptr(), 1, tokens, dy.data_ptr(), training._code(dt), vocab, dim, 0.75,
                                        padding, grad.data_ptr(), training._code(gd), acc, ws.data_ptr(), ws.numel(),
                                        torch.cuda.current_stream().cuda_stream) == 0
        check_gradient(ids, dy, vocab, 0.75, grad0, grad, padding if padding >= 0 else None)
        assert bool((buf[:pad] == 7.0).all()) and bool((buf[pad + vocab * dim:] == 7.0).all())
