"""A training step of a one-layer language model through the library's row operators
and BF16 products: token ids to clipped gradients.

    x   = embed(ids, table)                               table [vocab, hidden], tied with the logits
    qkv = rmsnorm(x) Wqkv^T;  q, k = qk_norm_rope(qkv)
    h   = x + attention(q, k, v) Wo^T                     (attention itself in torch)
    logits = rmsnorm(h) table^T;  loss = -mean logprob of the next token - beta * mean entropy

and back, every gradient by the operators' own calls: logprobs_backward,
rmsnorm_backward, qk_norm_rope_backward, embed_backward (added to the table's gradient
from the logits, in place), clip_grads.  Tokens, hidden, heads * D and vocab are
multiples of 128 (the products' K).

    python examples/lm_step.py
"""
from __future__ import annotations

import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from mx_block_scaled_gb300 import binding as mx

EPS = 1e-6


def rope_table(positions: int, rotary: int, base: float = 10000.0):
    """cos | sin of every position, angles formed in 64 bits."""
    f = base ** (-torch.arange(rotary // 2, dtype=torch.float64, device="cuda") / (rotary // 2))
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def attention(q, k, v, sequence):
    """Causal attention inside sequences (token t attends to its own sequence's tokens up to t); [tokens, heads, D]."""
    group = q.shape[1] // k.shape[1]
    k, v = (t.repeat_interleave(group, 1).transpose(0, 1) for t in (k, v))
    s = q.transpose(0, 1) @ k.transpose(1, 2) / math.sqrt(q.shape[2])
    t = torch.arange(len(sequence), device=q.device)
    keep = (sequence[:, None] == sequence[None, :]) & (t[:, None] >= t[None, :])
    return (torch.softmax(s.masked_fill(~keep, float("-inf")), -1) @ v).transpose(0, 1)


class Model:
    def __init__(self, vocab, hidden, q_heads, k_heads, D, positions, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(shape, generator=gen, device="cuda") * scale).to(torch.bfloat16)
        self.q_heads, self.k_heads, self.D, self.positions = q_heads, k_heads, D, positions
        self.scale = math.sqrt(hidden)          # of the embedded rows
        self.rope = rope_table(positions, D)
        w = dict(table=normal(vocab, hidden, scale=hidden ** -0.5),
                 qkv=normal((q_heads + 2 * k_heads) * D, hidden, scale=hidden ** -0.5),
                 out=normal(hidden, q_heads * D, scale=(q_heads * D) ** -0.5))
        for name, n in (("norm1", hidden), ("norm2", hidden), ("q_norm", D), ("k_norm", D)):
            w[name] = 1 + normal(n, scale=0.1)
        self.w = w
        self.plans = {}

    def product(self, a, b):
        """a [M, K] times b [N, K]^T in BF16 with FP32 sums."""
        key = (a.shape[0], b.shape[0], a.shape[1])
        if key not in self.plans:
            self.plans[key] = mx.Plan(*key, mx.MXGEMM_FMT_BF16, mx.MXGEMM_OUT_BF16)
        return self.plans[key].run(a, None, b, None)

    def product_backward(self, dy, x, w):
        """Gradients of product(x, w): (dx, dw)."""
        return (self.product(dy, w.t().contiguous()),
                self.product(dy.t().contiguous(), x.t().contiguous()))

    def step(self, ids, positions, targets, sequence, beta=0.0, max_norm=1.0):
        """(loss, norm of the gradients, clipped FP32 gradients by name).

        ids, positions and sequence [tokens]; padding has id and position -1; targets outside the vocabulary do not
        count."""
        w, Q, K, D, T = self.w, self.q_heads, self.k_heads, self.D, ids.numel()
        x = mx.embed(ids, w["table"], scale=self.scale)
        n1 = mx.rmsnorm(x, w["norm1"], EPS, plain=True)
        qkv = self.product(n1.y, w["qkv"]).view(T, Q + 2 * K, D)
        qk = mx.qk_norm_rope(qkv[:, :Q + K], Q, w["q_norm"], w["k_norm"], EPS, rope=self.rope, positions=positions)
        q, k, v = (t.float().requires_grad_() for t in (qk.y[:, :Q], qk.y[:, Q:], qkv[:, Q + K:]))
        a = attention(q, k, v, sequence)
        ab = a.detach().to(torch.bfloat16).reshape(T, Q * D)
        n2 = mx.rmsnorm(self.product(ab, w["out"]), w["norm2"], EPS, residual=x, plain=True)
        logits = self.product(n2.y, w["table"])
        lp = mx.logprobs(logits, targets, entropy=beta != 0.0)
        counted = (targets >= 0) & (targets < logits.shape[1])
        count = counted.sum()
        loss = -lp.logprob.sum() / count
        dlp = torch.full((T,), -1.0, device="cuda") / count
        if beta != 0.0:
            loss = loss - beta * (lp.entropy * counted).sum() / count
            dent = -beta * counted.float() / count

        g = {}
        dlogits = mx.logprobs_backward(logits, targets, lp.stats, dlp, entropy=lp.entropy,
                                       dentropy=dent if beta != 0.0 else None, dlogits=logits)
        dn2, dhead = self.product_backward(dlogits, n2.y, w["table"])
        dh, g["norm2"] = mx.rmsnorm_backward(dn2, n2.h, n2.rstd, w["norm2"])
        dab, dout = self.product_backward(dh, ab, w["out"])
        dq, dk, dv = torch.autograd.grad(a, (q, k, v), dab.float().view(T, Q, D))
        dqkv = torch.empty_like(qkv)
        dqkv[:, :Q + K] = torch.cat([dq, dk], 1)
        dqkv[:, Q + K:] = dv
        _, g["q_norm"], g["k_norm"] = mx.qk_norm_rope_backward(
            dqkv[:, :Q + K], qkv[:, :Q + K], qk.rstd, Q, w["q_norm"], w["k_norm"], rope=self.rope, positions=positions,
            dx=dqkv[:, :Q + K])
        dn1, dwqkv = self.product_backward(dqkv.view(T, -1), n1.y, w["qkv"])
        dx, g["norm1"] = mx.rmsnorm_backward(dn1, x, n1.rstd, w["norm1"], dh=dh)
        g["table"] = mx.embed_backward(dx, ids, w["table"].shape[0], scale=self.scale, add=dhead, dtable=dhead)
        g["qkv"], g["out"] = dwqkv, dout
        clipped = {name: torch.empty(t.shape, dtype=torch.float32, device="cuda") for name, t in g.items()}
        norm, _ = mx.clip_grads(list(g.values()), max_norm, out=list(clipped.values()))
        return loss, norm, clipped


def main():
    model = Model(vocab=1024, hidden=256, q_heads=4, k_heads=2, D=64, positions=256)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    ids = torch.randint(0, 1024, (512,), generator=gen, device="cuda")
    sequence = torch.arange(512, device="cuda") // 200           # two sequences of 200 tokens and one of 112
    positions = torch.arange(512, device="cuda") % 200
    targets = torch.where(positions < 199, torch.roll(ids, -1), -100)
    masters = {k: v.float() for k, v in model.w.items()}
    for i in range(10):
        loss, norm, grads = model.step(ids, positions, targets, sequence)
        for k, m in masters.items():
            m.sub_(grads[k], alpha=0.3)
            model.w[k].copy_(m)
        print(f"step {i}: loss {loss.item():.4f}, gradient norm {norm.item():.4f}")


if __name__ == "__main__":
    main()
