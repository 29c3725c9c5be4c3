"""A small language model trained the QLoRA way on one GPU: every operator of a
training step is the library's.

    python3 examples/qlora_training.py [--steps 60] [--moments 8|32] [--dim 512] [--heads 0]
                                       [--optimizer adamw|muon]

token embedding -> blocks of (norm, NF4 + LoRA up projection, activation, NF4 +
LoRA down projection, norm, gate, residual addition) -> tied output projection. With
--heads, causal attention comes before each up projection, its queries and keys
normed head by head and rotated by their positions; with --optimizer muon, Muon
steps the adapters and AdamW the rest. The 4-bit bases are frozen; adapters, norms,
gates and the table train. The text is synthetic: each token follows from the one before it by a fixed table, with
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


def base(n, k, g):
    w = torch.randn(n, k, generator=g, device="cuda") / math.sqrt(k)
    return w.to(torch.bfloat16)


class Attention(torch.nn.Module):
    """Causal attention, two heads of queries for one of keys and values."""

    def __init__(self, dim, heads, rank, rope, g):
        super().__init__()
        linear, self.head, self.rope = nq.make_lora_linear_module(), dim // heads, rope
        narrow = dim // 2
        self.q, self.o = (linear(base(dim, dim, g), r=rank, alpha=rank, generator=g) for _ in range(2))
        self.k, self.v = (linear(base(narrow, dim, g), r=rank, alpha=rank, generator=g) for _ in range(2))
        self.norm_q, self.norm_k = (torch.nn.Parameter(torch.ones(self.head, device="cuda")) for _ in range(2))

    def forward(self, x):
        q, k, v = (y.unflatten(-1, (-1, self.head)) for y in (self.q(x), self.k(x), self.v(x)))
        q, k = nq.rotary(q, k, None, self.rope, self.norm_q, self.norm_k)
        # [batch, heads, tokens, head]; every head of keys serves two of queries
        q, k, v = (y.transpose(1, 2).float() for y in (q, k, v))
        k, v = (y.repeat_interleave(2, 1) for y in (k, v))
        scores = q @ k.transpose(2, 3).contiguous() / math.sqrt(self.head)
        later = torch.ones(x.shape[1], x.shape[1], dtype=torch.bool, device="cuda").triu(1)
        y = scores.masked_fill(later, float("-inf")).softmax(-1) @ v
        return self.o(y.transpose(1, 2).flatten(2).to(x.dtype))


class Block(torch.nn.Module):
    """z = down(silu(up(x))), x with its attention added where there is one; the caller
    adds z to the residual stream."""

    def __init__(self, dim, hidden, rank, g, heads=0, rope=None):
        super().__init__()
        linear = nq.make_lora_linear_module()
        self.up = linear(base(hidden, dim, g), r=rank, alpha=rank, generator=g)
        self.down = linear(base(dim, hidden, g), r=rank, alpha=rank, generator=g)
        self.norm_after = torch.nn.Parameter(torch.ones(dim, device="cuda"))
        self.norm_before_next = torch.nn.Parameter(torch.ones(dim, device="cuda"))
        self.gate = torch.nn.Parameter(torch.full((dim,), 0.5, device="cuda"))
        self.attention = Attention(dim, heads, rank, rope, g) if heads else None

    def forward(self, x):
        if self.attention is not None:
            x = x + self.attention(x)
        return self.down(F.silu(self.up(x)))


class Model(torch.nn.Module):
    def __init__(self, vocab=1024, dim=512, hidden=1024, blocks=2, rank=16, seed=0, heads=0):
        super().__init__()
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.scale = math.sqrt(dim)
        self.alpha = 1.0 / math.sqrt(blocks)
        table = torch.randn(vocab, dim, generator=g, device="cuda") / self.scale
        self.table = torch.nn.Parameter(table.to(torch.bfloat16))
        self.norm_in = torch.nn.Parameter(torch.ones(dim, device="cuda"))
        rope = nq.NF4Rotary(dim // heads) if heads else None
        self.blocks = torch.nn.ModuleList(Block(dim, hidden, rank, g, heads, rope) for _ in range(blocks))

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
          noise=0.1, seed=0, report=None, heads=0, optimizer="adamw"):
    """Trains for `steps` steps; returns the losses."""
    model = Model(vocab, dim, hidden, blocks, rank, seed, heads)
    # bfloat16 parameters with fp32 master weights, and the fp32 norms and gates: a list
    # has one dtype, and each optimizer clips by the norm of its own list
    half = [p for p in model.parameters() if p.dtype == torch.bfloat16]
    full = [p for p in model.parameters() if p.dtype == torch.float32]
    adapters = [p for n, p in model.named_parameters() if n.endswith(("lora_a", "lora_b"))]
    if optimizer == "muon":  # the matrices of the adapters; the table and the fp32 norms and gates stay with AdamW
        half = [p for p in half if not any(p is a for a in adapters)]
    optimizers = [nq.NF4AdamW([dict(params=half, lr=lr, weight_decay=0.0, masters=True)], state_bits=moments,
                              max_grad_norm=1.0, seed=seed),
                  nq.NF4AdamW([dict(params=full, lr=lr, weight_decay=0.0)], state_bits=32, max_grad_norm=1.0)]
    if optimizer == "muon":
        optimizers.append(nq.NF4Muon([dict(params=adapters, lr=lr, weight_decay=0.0, masters=True)], adjust="rms"))
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
    ap.add_argument("--heads", type=int, default=0)
    ap.add_argument("--optimizer", choices=("adamw", "muon"), default="adamw")
    a = ap.parse_args()
    train(steps=a.steps, moments=a.moments, dim=a.dim, hidden=2 * a.dim, report=lambda s: print(s, flush=True), heads=a.heads,
          optimizer=a.optimizer)
