"""The training-step operators together: the example's model trains, with 8-bit
moments as with 32; its gradients are those of the same model in plain fp32
torch; the calls replay from a HIP graph and run on a stream of the caller's;
offsets past 2^31 elements."""
import math
import os
import sys

import numpy as np
import pytest

import nf4_quantize_amd as nq
from conftest import ROOT
from gpu_util import log

sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def test_example_trains(dev):
    """From the untrained model's loss (its tied table foretells the token it has just
    read) towards the data's entropy (noise 0.1: 0.33 + 0.1 ln 1024 = 1.02); 8-bit
    moments end near 32-bit ones."""
    import qlora_training

    ends = {}
    for moments in (8, 32):
        losses = qlora_training.train(steps=80, moments=moments)
        log(f"moments {moments}: {losses[0]:.3f} -> {losses[-1]:.3f}")
        assert all(math.isfinite(x) for x in losses)
        assert losses[-1] < 0.6 * losses[0]
        ends[moments] = sum(losses[-5:]) / 5
    assert abs(ends[8] - ends[32]) < 0.25 * ends[32]


def test_gradients_of_the_model(dev):
    """Every trainable tensor's gradient against the same model in fp32 torch (the
    bases dequantized): within the roundings of bf16 activations along the way,
    3e-2 of the gradient's norm."""
    import torch
    import torch.nn.functional as F
    import qlora_training

    model = qlora_training.Model(vocab=300, dim=256, hidden=512, blocks=2, rank=8, seed=3)
    with torch.no_grad():
        for b in model.blocks:  # adapters that matter
            for lin in (b.up, b.down):
                lin.lora_b.normal_(0, 0.05)
    ids = torch.randint(0, 300, (4, 50), device=dev)
    target = torch.randint(0, 300, (4, 50), device=dev)
    F.cross_entropy(model(ids).float().view(-1, 300), target.view(-1)).backward()

    p = {n: t.detach().float().requires_grad_() for n, t in model.named_parameters()}

    def norm(x, w):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w

    def linear(x, lin, name):
        w = nq.dequantize(lin.weight, torch.float32)
        return F.linear(x, w) + lin.scale * (x @ p[name + ".lora_a"]) @ p[name + ".lora_b"]

    h = p["table"][ids] * model.scale
    x = norm(h, p["norm_in"])
    for i, b in enumerate(model.blocks):
        z = linear(F.silu(linear(x, b.up, f"blocks.{i}.up")), b.down, f"blocks.{i}.down")
        h = h + model.alpha * p[f"blocks.{i}.gate"] * norm(z, p[f"blocks.{i}.norm_after"])
        x = norm(h, p[f"blocks.{i}.norm_before_next"])
    F.cross_entropy((x @ p["table"].t()).view(-1, 300), target.view(-1)).backward()
    for n, t in model.named_parameters():
        got, want = t.grad.double(), p[n].grad.double()
        err = float((got - want).norm() / want.norm())
        log(f"{n}: {err:.2e}")
        assert err < 3e-2, n


def work(dev, seed=0):
    """Inputs of one pass through every operator, and the pass."""
    import torch

    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rows, dim, vocab = 200, 1030, 500

    def randn(*s):
        return torch.randn(*s, generator=g, device=dev)

    ids = torch.randint(-1, vocab, (rows,), generator=g, device=dev)
    table = randn(vocab, dim).to(torch.bfloat16)
    packed = nq.quantize(randn(64, 128).to(torch.bfloat16))
    w_pre, w_post, gate = 1 + 0.1 * randn(dim), 1 + 0.1 * randn(dim), randn(dim)
    dx, dh = randn(rows, dim).to(torch.bfloat16), randn(rows, dim).to(torch.bfloat16)
    params = [randn(n).to(torch.bfloat16) for n in (1, 300, 70000)] + [randn(97).to(torch.bfloat16) for _ in range(60)]
    grads = [randn(p.numel()).to(torch.bfloat16) for p in params]
    opt = nq.NF4AdamW(params, state_bits=8, max_grad_norm=1.0)

    def run():
        y = nq.embedding_forward(ids, table, 3.0)
        e = nq.embedding_forward(ids.clamp(-1, 63), packed, 2.0)
        h, x, r1, r2 = nq.residual_norm_forward(y, dh, w_pre, w_post, gate)
        back = nq.residual_norm_backward(dx, dh, y, h, r1, w_pre, r2, w_post, gate)
        dtable = nq.embedding_backward(ids, back[0], vocab, 3.0)
        opt.step(grads, step=3, seed=11)
        return [y, e, h, x, r1, r2, dtable, opt.grad_norm, *back]

    state = params + [t.view(torch.uint8) for t in opt.m + opt.v] + opt.m_scale + opt.v_scale
    return run, state


def bits(ts):
    import torch

    return [t.detach().clone().contiguous().view(torch.uint8) for t in ts]


def test_graph_replays_match_eager(dev):
    import torch

    run, state = work(dev)
    start = [t.clone() for t in state]

    def restore():
        for t, s in zip(state, start):
            t.copy_(s)

    want = []
    for _ in range(3):  # the optimizer's state goes on from call to call
        out = run()
        want.append(bits(out + state))
    restore()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    restore()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    torch.cuda.synchronize()
    for rep in range(3):
        for t in out:
            t.view(torch.uint8).fill_(0xA5)  # eager work between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        log(f"graph replay {rep}")
        for i, (a, b) in enumerate(zip(bits(out + state), want[rep])):
            assert torch.equal(a, b), (rep, i)


def test_on_a_stream_of_the_callers(dev):
    """Inputs made on one stream and used on another after an event: the operators'
    launches and their own buffers are the current stream's."""
    import torch

    run, state = work(dev, seed=5)
    start = [t.clone() for t in state]
    want = bits(run() + state)
    for t, s in zip(state, start):
        t.copy_(s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device=dev)
    for _ in range(8):
        big = big @ big * 1e-3  # keeps the default stream busy
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = run()
        got = bits(out + state)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_adamw_past_32_bit_offsets(dev):
    """The last elements of a tensor of more than 2^32 bytes and 2^31 elements."""
    import torch

    n, tail = (1 << 31) + 1000, 5000
    w = torch.full((n,), 0.5, dtype=torch.bfloat16, device=dev)
    g = torch.zeros(n, dtype=torch.bfloat16, device=dev)
    g[-tail:] = torch.randn(tail, device=dev).to(torch.bfloat16)
    small_w, small_g = w[-tail:].clone(), g[-tail:].clone()
    for bits_ in (8, 32):
        log(f"adamw {n} elements, {bits_}-bit moments")
        if bits_ == 8:
            opt = nq.NF4AdamW([w], lr=0.01, weight_decay=0.0, state_bits=8, max_grad_norm=1.0)
            opt.step([g])
            norm = float(opt.grad_norm)
            assert abs(norm - float(g[-tail:].double().norm())) <= 1e-6 * norm
            assert int(torch.count_nonzero(opt.m[0][: n - tail].view(torch.uint8))) == 0
            # the same elements alone: the weights do not depend on the random bits
            ref = nq.NF4AdamW([small_w], lr=0.01, weight_decay=0.0, state_bits=8, max_grad_norm=1.0)
            ref.step([small_g])
            assert torch.equal(w[-tail:], small_w)
            assert bool((w[: n - tail] == 0.5).all())
            del opt, ref
        else:
            w.fill_(0.5)
            small_w.fill_(0.5)
            opt = nq.NF4AdamW([w], lr=0.01, weight_decay=0.0, state_bits=32)
            ref = nq.NF4AdamW([small_w], lr=0.01, weight_decay=0.0, state_bits=32)
            opt.step([g])
            ref.step([small_g])
            assert torch.equal(w[-tail:], small_w) and torch.equal(opt.v[0][-tail:], ref.v[0])
            del opt, ref


def test_norm_past_32_bit_offsets(dev):
    """The last rows of more than 2^31 elements."""
    import torch

    rows, dim = 264_000, 8200
    assert rows * dim > 1 << 31
    y = torch.zeros(rows, dim, dtype=torch.bfloat16, device=dev)
    h = torch.zeros(rows, dim, dtype=torch.bfloat16, device=dev)
    y[-3:] = torch.randn(3, dim, device=dev).to(torch.bfloat16)
    h[-3:] = torch.randn(3, dim, device=dev).to(torch.bfloat16)
    w = torch.rand(dim, device=dev) + 0.5
    small = nq.residual_norm_forward(y[-3:].contiguous(), h[-3:].contiguous(), w, w)
    big = nq.residual_norm_forward(y, h, w, w)
    for a, b in zip(big, small):
        assert torch.equal(a[-3:], b)
    assert not bool(big[0][: rows - 3].any())
    dx = torch.zeros_like(y)
    dx[-3:] = torch.randn(3, dim, device=dev).to(torch.bfloat16)
    gb = nq.residual_norm_backward(dx, None, y, big[0], big[2], w, big[3], w)
    gs = nq.residual_norm_backward(dx[-3:].contiguous(), None, y[-3:].contiguous(), small[0], small[2], w, small[3], w)
    assert torch.equal(gb[0][-3:], gs[0]) and torch.equal(gb[1][-3:], gs[1])
    # the sums of three rows and of zeros, in another order: 4 u of their terms
    for a, b in zip(gb[2:4], gs[2:4]):
        assert bool(((a - b).abs() <= 1e-5 * b.abs().max()).all())
