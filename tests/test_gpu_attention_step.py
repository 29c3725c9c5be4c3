"""The rotation with its norms and the Muon step as a training step and a decoding loop
use them: in the example's model, token by token, and captured together."""
import math
import os
import sys

import pytest

from conftest import ROOT
from gpu_util import log

sys.path.insert(0, os.path.join(ROOT, "examples"))

import nf4_quantize_amd as nq  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("optimizer", ["adamw", "muon"])
def test_example_runs_with_attention(dev, optimizer):
    import qlora_training

    losses = qlora_training.train(steps=4, vocab=200, dim=256, hidden=512, rank=8, batch=4, length=33, heads=4,
                                  optimizer=optimizer)
    assert len(losses) == 4 and all(math.isfinite(x) for x in losses)


def test_gradients_of_the_model_with_attention(dev):
    """Every trainable tensor's gradient against the same model in fp32 torch (the bases dequantized): within the
    roundings of bf16 activations along the way. A rounding is off by up to 2^-9 of a value; the path through one
    block has eight tensors of bf16 forward and as many backward, four of them in a softmax's scores: 32 such
    roundings added as independent ones, over two blocks, are 2^-9 sqrt(64) = 1.6e-2 of the gradient's norm, doubled
    for the scores' amplification."""
    import torch
    import torch.nn.functional as F
    import qlora_training

    model = qlora_training.Model(vocab=300, dim=256, hidden=512, blocks=2, rank=8, seed=3, heads=4)
    linears = ("up", "down", "attention.q", "attention.k", "attention.v", "attention.o")
    with torch.no_grad():
        for b in model.blocks:  # adapters and norms that matter
            for name in linears:
                b.get_submodule(name).lora_b.normal_(0, 0.05)
            for w in (b.attention.norm_q, b.attention.norm_k):
                w.mul_(1 + 0.2 * torch.randn_like(w))
    ids = torch.randint(0, 300, (4, 50), device=dev)
    target = torch.randint(0, 300, (4, 50), device=dev)
    F.cross_entropy(model(ids).float().view(-1, 300), target.view(-1)).backward()

    p = {n: t.detach().float().requires_grad_() for n, t in model.named_parameters()}

    def norm(x, w):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w

    def linear(x, lin, name):
        w = nq.dequantize(lin.weight, torch.float32)
        return F.linear(x, w) + lin.scale * (x @ p[name + ".lora_a"]) @ p[name + ".lora_b"]

    def turned(x, rope):
        half = rope.dim // 2
        angle = torch.arange(x.shape[1], device=dev).double()[:, None] * torch.tensor(rope.frequencies, device=dev).double()
        c, s = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
        return torch.cat((x[..., :half] * c - x[..., half:] * s, x[..., half:] * c + x[..., :half] * s), -1)

    def attention(x, a, name):
        q, k, v = (linear(x, getattr(a, n), f"{name}.{n}").unflatten(-1, (-1, a.head)) for n in "qkv")
        q, k = turned(norm(q, p[name + ".norm_q"]), a.rope), turned(norm(k, p[name + ".norm_k"]), a.rope)
        q, k, v = (y.transpose(1, 2) for y in (q, k, v))
        k, v = k.repeat_interleave(2, 1), v.repeat_interleave(2, 1)
        scores = q @ k.transpose(2, 3).contiguous() / math.sqrt(a.head)
        scores = scores.masked_fill(torch.ones_like(scores, dtype=torch.bool).triu(1), float("-inf"))
        return linear((scores.softmax(-1) @ v).transpose(1, 2).flatten(2), a.o, name + ".o")

    h = p["table"][ids] * model.scale
    x = norm(h, p["norm_in"])
    for i, b in enumerate(model.blocks):
        x = x + attention(x, b.attention, f"blocks.{i}.attention")
        z = linear(F.silu(linear(x, b.up, f"blocks.{i}.up")), b.down, f"blocks.{i}.down")
        h = h + model.alpha * p[f"blocks.{i}.gate"] * norm(z, p[f"blocks.{i}.norm_after"])
        x = norm(h, p[f"blocks.{i}.norm_before_next"])
    F.cross_entropy((x @ p["table"].t()).view(-1, 300), target.view(-1)).backward()
    for n, t in model.named_parameters():
        got, want = t.grad.double(), p[n].grad.double()
        err = float((got - want).norm() / want.norm())
        log(f"{n}: {err:.2e}")
        assert err < 3.2e-2, n


def test_prompt_and_single_tokens(dev):
    """A prompt rotated at once, and its tokens one after the other as a batch decodes them: the same bits."""
    import torch

    g = torch.Generator(device=dev)
    g.manual_seed(1)
    rope = nq.NF4Rotary(96, layout="interleaved", scaling=dict(kind="yarn", factor=4, length=32), device=dev)
    w = torch.rand(128, generator=g, device=dev) + 0.5
    q, k = (torch.randn(3, 40, n, 128, generator=g, device=dev).bfloat16() for n in (6, 2))
    first = torch.tensor([0, 7, 100000], device=dev)
    at = first[:, None] + torch.arange(40, device=dev)
    want = nq.rotary_forward(q, k, at, rope, w, w)
    for t in (0, 1, 17, 39):
        got = nq.rotary_forward(q[:, t:t + 1], k[:, t:t + 1], at[:, t:t + 1], rope, w, w)
        assert all(torch.equal(x, y[:, t:t + 1]) for x, y in zip(got, want))
        # packed: the batch as tokens of one sequence
        got = nq.rotary_forward(q[:, t], k[:, t], at[:, t].contiguous(), rope, w, w)
        assert all(torch.equal(x, y[:, t]) for x, y in zip(got, want))


def test_captured_together(dev):
    """Norms and rotation forward and backward and a Muon step of the norms' neighbours, captured in one graph:
    every replay gives the eager bits."""
    import torch

    def make():
        g = torch.Generator(device=dev)
        g.manual_seed(2)
        a, b = torch.randn(256, 16, generator=g, device=dev).bfloat16(), torch.randn(16, 256, generator=g, device=dev).bfloat16()
        return [a, b], nq.NF4Muon([a, b], lr=1e-2, state_bits=16)

    g = torch.Generator(device=dev)
    g.manual_seed(3)
    rope, w = nq.NF4Rotary(64, device=dev), torch.rand(64, generator=g, device=dev) + 0.5
    x = torch.randn(256, 256, generator=g, device=dev).bfloat16()

    def step(params, opt):
        a, b = params
        q = ((x @ a) @ b).view(64, 16, 64)
        y, _ = nq.rotary_forward(q, None, None, rope, w)
        dq, _, dw, _ = nq.rotary_backward(y, None, None, rope, q, None, w)
        d = dq.reshape(256, 256)
        opt.step([(x.t().contiguous() @ (d @ b.t().contiguous())), (x @ a).t().contiguous() @ d])
        return y, dq, dw

    eager, opt = make()
    graphed, opt_g = make()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(graphed, opt_g)
    torch.cuda.current_stream().wait_stream(side)
    step(eager, opt)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(graphed, opt_g)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        want = step(eager, opt)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip([*held, *graphed, *opt_g.m], [*want, *eager, *opt.m]))
