"""A small language model trained the QLoRA way on one GPU: every operator of a
training step is the library's.

    python3 examples/qlora_training.py [--steps 60] [--moments 8|32] [--dim 512]

token embedding -> blocks of (norm, NF4 + LoRA up projection, activation, NF4 +
LoRA down projection, norm, gate, residual addition) -> tied output projection.
The 4-bit bases are frozen; adapters, norms, gates and the table train. The text
is synthetic: each token follows from the one before it by a fixed table, with
some noise, so a model that trains reaches a loss near the noise's entropy.
"""
import argparse
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402
import torch.nn.functional as F  # noqa: E402

import nf4_quantize_amd as nq  # noqa: E402


class Block(torch.nn.Module):
    """z = down(silu(up(x))); the caller adds it to the residual stream."""

    def __init__(self, dim, hidden, rank, g):
        super().__init__()
        linear = nq.make_lora_linear_module()

        def base(n, k):
            w = torch.randn(n, k, generator=g, device="cuda") / math.sqrt(k)
            return w.to(torch.bfloat16)

        self.up = linear(base(hidden, dim), r=rank, alpha=rank, generator=g)
        self.down = linear(base(dim, hidden), r=rank, alpha=rank, generator=g)
        self.norm_after = torch.nn.Parameter(torch.ones(dim, device="cuda"))
        self.norm_before_next = torch.nn.Parameter(torch.ones(dim, device="cuda"))
        self.gate = torch.nn.Parameter(torch.full((dim,), 0.5, device="cuda"))

    def forward(self, x):
        return self.down(F.silu(self.up(x)))


class Model(torch.nn.Module):
    def __init__(self, vocab=1024, dim=512, hidden=1024, blocks=2, rank=16, seed=0):
        super().__init__()
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.scale = math.sqrt(dim)
        self.alpha = 1.0 / math.sqrt(blocks)
        table = torch.randn(vocab, dim, generator=g, device="cuda") / self.scale
        self.table = torch.nn.Parameter(table.to(torch.bfloat16))
        self.norm_in = torch.nn.Parameter(torch.ones(dim, device="cuda"))
        self.blocks = torch.nn.ModuleList(Block(dim, hidden, rank, g) for _ in range(blocks))

    def forward(self, ids):
        h = nq.nf4_embedding(ids, self.table, self.scale)
        h, x = nq.residual_norm(None, h, self.norm_in)
        for b in self.blocks:
            h, x = nq.residual_norm(b(x), h, b.norm_before_next, b.norm_after, b.gate, alpha=self.alpha)
        return F.linear(x, self.table)


def batches(vocab, batch, length, noise, seed):
    """Sequences in which token t + 1 is next[token t], or, with probability
    `noise`, any token."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    following = torch.randperm(vocab, generator=g, device="cuda")
    while True:
        ids = torch.empty(batch, length, dtype=torch.int64, device="cuda")
        ids[:, 0] = torch.randint(0, vocab, (batch,), generator=g, device="cuda")
        other = torch.randint(0, vocab, (batch, length), generator=g, device="cuda")
        stray = torch.rand(batch, length, generator=g, device="cuda") < noise
        for t in range(1, length):
            ids[:, t] = torch.where(stray[:, t], other[:, t], following[ids[:, t - 1]])
        yield ids


def train(steps=60, moments=8, vocab=1024, dim=512, hidden=1024, blocks=2, rank=16, batch=16, length=64, lr=5e-3,
          noise=0.1, seed=0, report=None):
    """Trains for `steps` steps; returns the losses."""
    model = Model(vocab, dim, hidden, blocks, rank, seed)
    # bfloat16 parameters with fp32 master weights, and the fp32 norms and gates: a list
    # has one dtype, and each optimizer clips by the norm of its own list
    half = [p for p in model.parameters() if p.dtype == torch.bfloat16]
    full = [p for p in model.parameters() if p.dtype == torch.float32]
    optimizers = [nq.NF4AdamW([dict(params=half, lr=lr, weight_decay=0.0, masters=True)], state_bits=moments,
                              max_grad_norm=1.0, seed=seed),
                  nq.NF4AdamW([dict(params=full, lr=lr, weight_decay=0.0)], state_bits=32, max_grad_norm=1.0)]
    data, losses = batches(vocab, batch, length, noise, seed + 1), []
    for step in range(steps):
        ids = next(data)
        logits = model(ids[:, :-1].contiguous())
        loss = F.cross_entropy(logits.float().reshape(-1, vocab), ids[:, 1:].reshape(-1))
        loss.backward()
        for opt in optimizers:
            opt.step()
            opt.zero_grad()
        losses.append(loss.item())
        if report and (step % 10 == 0 or step + 1 == steps):
            report(f"step {step}: loss {losses[-1]:.3f}, gradient norm {float(optimizers[0].grad_norm):.3f}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--moments", type=int, choices=(8, 32), default=8)
    ap.add_argument("--dim", type=int, default=512)
    a = ap.parse_args()
    train(steps=a.steps, moments=a.moments, dim=a.dim, hidden=2 * a.dim, report=lambda s: print(s, flush=True))
