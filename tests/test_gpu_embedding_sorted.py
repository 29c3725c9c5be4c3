"""The table's gradient above 128 tokens, where the tokens are sorted: each way of
sorting (one launch up to 6144 tokens, tiles and a merge up to 32768, digits
above), rows of whole cache lines and others, every pair of types, written over
memory that holds NaN and added; offsets past 2^31 elements.

The tolerance is that of test_gpu_embedding.py: (count + 3) u of the sum of a
row's magnitudes, u = 2^-24, and 2^-8 of itself in bfloat16."""
import pytest

import nf4_quantize_amd as nq
from gpu_util import log
from test_gpu_embedding import U, draw

pytestmark = pytest.mark.gpu

# tokens, vocabulary, width; a line of 128 bytes is 64 bf16 or 32 fp32
SIZES = [(129, 97, 64), (300, 97, 96), (700, 50, 4096), (1000, 129, 512), (5000, 700, 2048), (6144, 9000, 32),
         (6145, 300, 544), (9000, 500, 1024), (20000, 300, 96), (32768, 3000, 64), (32769, 40, 64), (40000, 300, 128),
         (33000, 70000, 192)]


def backward(ids, dy, grad, acc, scale, padding=-1):
    """The C entry, into a gradient and a workspace that hold NaN where they may."""
    import torch
    from nf4_quantize_amd import training

    L, (vocab, dim) = nq.lib(), grad.shape
    size = L.nf4_embedding_backward_workspace_size(ids.numel(), vocab, dim)
    ws = torch.full((size // 4,), float("nan"), device=dy.device)
    st = L.nf4_embedding_backward(ids.data_ptr(), 1, ids.numel(), dy.data_ptr(), training._code(dy.dtype), vocab, dim, scale,
                                  padding, grad.data_ptr(), training._code(grad.dtype), acc, ws.data_ptr(), size,
                                  torch.cuda.current_stream().cuda_stream)
    assert st == 0


@pytest.mark.parametrize("tokens,vocab,dim", SIZES)
@pytest.mark.parametrize("kind", ["few", "any"])
@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
def test_gradient(dev, tokens, vocab, dim, kind, dt):
    import torch

    ids = draw(dev, kind, tokens, vocab, seed=7)
    inside = (ids >= 0) & (ids < vocab)
    padding = int(ids[inside][-1])
    dy = torch.randn(tokens, dim, device=dev).to(getattr(torch, dt))
    live = inside & (ids != padding)
    at, rows = ids[live].cpu(), dy[live].double().cpu() * 0.75
    want = torch.zeros(vocab, dim, dtype=torch.float64).index_add_(0, at, rows).to(dev)
    size = torch.zeros(vocab, dim, dtype=torch.float64).index_add_(0, at, rows.abs()).to(dev)
    count = torch.bincount(at, minlength=vocab).double().unsqueeze(1).to(dev)
    for gd in (torch.bfloat16, torch.float32):
        for acc in (0, 1):
            log(f"sorted gradient {tokens} tokens {vocab}x{dim} {kind} {dt} {gd} acc={acc}")
            grad0 = torch.randn(vocab, dim, device=dev).to(gd) if acc else None
            grad = grad0.clone() if acc else torch.full((vocab, dim), float("nan"), dtype=gd, device=dev)
            backward(ids, dy, grad, acc, 0.75, padding)
            total = want + (grad0.double() if acc else 0.0)
            terms = size + (grad0.double().abs() if acc else 0.0)
            tol = (count + 3) * U * terms + (2.0 ** -8 if gd == torch.bfloat16 else U) * total.abs()
            err = (grad.double() - total).abs()
            assert bool((err <= tol).all()), (float(err.max()), torch.nonzero(~(err <= tol))[:3].tolist())
            silent = (count == 0).squeeze(1)
            assert torch.equal(grad[silent], grad0[silent] if acc else torch.zeros_like(grad[silent]))


@pytest.mark.parametrize("acc", [0, 1])
def test_table_past_32_bit_offsets(dev, acc):
    """A gradient of more than 2^31 elements and 2^32 bytes, from 200 tokens, some of
    whose runs cross chunks."""
    import torch

    vocab, dim, tokens = 300_000, 8192, 200
    log(f"sorted gradient {tokens} tokens {vocab}x{dim} acc={acc}")
    rows = torch.tensor([0, 5, 262_143, 262_144, 299_998, 299_999], device=dev)
    ids = rows[torch.randint(0, 6, (tokens,), device=dev)]
    dy = torch.randn(tokens, dim, device=dev).to(torch.bfloat16)
    grad = torch.full((vocab, dim), 1.0 if acc else 3.0, dtype=torch.bfloat16, device=dev)
    backward(ids, dy, grad, acc, 1.0)
    for row in rows.tolist():
        mine = dy[ids == row].double()
        want, size = mine.sum(0) + acc, mine.abs().sum(0) + acc
        tol = (mine.shape[0] + 3) * U * size + 2.0 ** -8 * want.abs()
        assert bool(((grad[row].double() - want).abs() <= tol).all()), row
    keep = torch.ones(vocab, dtype=torch.bool, device=dev)
    keep[rows] = False
    bad = 0
    for part in range(0, vocab, 50_000):
        k = keep[part:part + 50_000]
        bad += int((grad[part:part + 50_000][k] != float(acc)).sum())
    assert bad == 0


def test_tokens_past_32_bit_offsets(dev):
    """Incoming gradients of more than 2^31 elements and 2^32 bytes: the last tokens'
    rows are found."""
    import torch

    tokens, vocab, dim = 270_000, 50, 8192
    log(f"sorted gradient {tokens} tokens {vocab}x{dim}")
    ids = torch.randint(0, vocab - 2, (tokens,), device=dev)
    ids[-3:] = vocab - 1  # a row of the last tokens alone
    dy = torch.randn(tokens, dim, device=dev, dtype=torch.bfloat16)
    grad = torch.full((vocab, dim), float("nan"), device=dev)
    backward(ids, dy, grad, 0, 1.0)
    last = dy[-3:].double()
    assert bool(((grad[-1].double() - last.sum(0)).abs() <= 6 * U * last.abs().sum(0)).all())
    assert not bool(grad[-2].any())
    count = torch.bincount(ids, minlength=vocab).double().unsqueeze(1)
    for col in (0, 511, 512, 4095, 8191):
        c = dy[:, col:col + 1].double()
        want = torch.zeros(vocab, 1, dtype=torch.float64, device=dev).index_add_(0, ids, c)
        size = torch.zeros(vocab, 1, dtype=torch.float64, device=dev).index_add_(0, ids, c.abs())
        err = (grad[:, col:col + 1].double() - want).abs()
        assert bool((err <= (count + 3) * U * size).all()), col
