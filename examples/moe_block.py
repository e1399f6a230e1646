"""A mixture-of-experts feed-forward block, forward and backward, on one GB300.

    h = x + r;  y = rmsnorm(h);  ids, weights = softmax of the top-k router logits
    out = h + sum over a token's experts of  weight * W2 (silu(G) * U),  [G | U] = W1 y

Every step but the router's small product runs in the library: norm, expert
sort and dispatch (which writes the MXFP8 operand of the first product), two
grouped MXFP8 products, the gated activation (which writes the operand of the
second and keeps its own inputs as an 8-bit checkpoint), and the weighted return
with the residual.  The backward pass goes the same way back to the gradients of
x, of the norm's weight and of the router's weight, through the transposed expert
weights.  The experts' own weight gradients need a product over tokens, which the
library does not offer.

    python examples/moe_block.py [--tokens 4096 --hidden 4096 --inner 14336 --experts 8 --topk 2]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mx_block_scaled_gb300 import binding as mx  # noqa: E402

FP8, BF16 = mx.MXGEMM_FMT_MXFP8_E4M3, mx.MXGEMM_OUT_BF16


class Weight:
    """Expert weights [experts, N, K] as one MXFP8 operand, scales in the GEMM's layout."""

    def __init__(self, w):
        e, n, k = w.shape
        self.codes, self.scales = mx.quantize(w.reshape(e * n, k).contiguous(), FP8, tiled=True)


class MoeBlock:
    """Weights in BF16: norm [H], router [E, H] (FP32), w1 [E, 2F, H], w2 [E, H, F]."""

    def __init__(self, norm, router, w1, w2, topk: int, eps: float = 1e-5):
        self.norm, self.router, self.topk, self.eps = norm, router, topk, eps
        self.experts, self.inner, self.hidden = w1.shape[0], w1.shape[1] // 2, w1.shape[2]
        self.w1, self.w2 = Weight(w1), Weight(w2)
        # the backward products contract over the other axis, so the transposes are quantised along it
        self.w1t, self.w2t = Weight(w1.transpose(1, 2)), Weight(w2.transpose(1, 2))
        self.plans = {}

    def product(self, offsets, codes, scales, weight, N, K):
        """Grouped product of expert-ordered rows with each expert's [N, K] weight."""
        rows = codes.shape[0]
        plan = self.plans.get((rows, N, K))
        if plan is None:
            plan = self.plans[rows, N, K] = mx.GroupedPlan(self.experts, rows, N, K, FP8, BF16)
        return plan.run(offsets, codes, scales, weight.codes, weight.scales, run_flags=mx.MXGEMM_RUN_SB_PRELAYOUT)

    def forward(self, x, r):
        """(out, what the backward pass needs)."""
        H, F, k = self.hidden, self.inner, self.topk
        n = mx.rmsnorm(x, self.norm, self.eps, residual=r, plain=True)
        top, ids = torch.topk(n.y.float() @ self.router.T, k, dim=1)
        weights = torch.softmax(top, dim=1)
        offsets, slot, _ = mx.moe_sort(ids, self.experts)
        codes, scales = mx.moe_dispatch(n.y, slot, FP8)
        gu = self.product(offsets, codes, scales, self.w1, 2 * F, H)
        a = mx.glu(gu[:, :F], gu[:, F:], mx.MXGEMM_ACT_SILU, fmt=FP8, keep=True)
        z = self.product(offsets, a.codes, a.scales, self.w2, H, F)
        out = mx.moe_combine(z, slot, k, weights=weights, add=n.h)
        return out, (n, ids, weights, offsets, slot, a.kept_codes, a.kept_scales, z)

    def backward(self, dout, saved):
        """Gradients of x (and of r), of the norm's weight and of the router's weight."""
        n, ids, weights, offsets, slot, kept_codes, kept_scales, z = saved
        H, F, k = self.hidden, self.inner, self.topk
        dz, dweights = mx.moe_combine_backward(dout, z, slot, weights)
        codes, scales = mx.quantize(dz, FP8)
        da = self.product(offsets, codes, scales, self.w2t, F, H)
        g = mx.glu_backward(da, mx.MXGEMM_ACT_SILU, kept_codes=kept_codes, kept_scales=kept_scales, fmt=FP8,
                            plain=False)
        drows = self.product(offsets, g.codes, g.scales, self.w1t, H, 2 * F)
        dy = mx.moe_combine(drows, slot, k)
        # the router: softmax over the chosen logits, then its product
        dtop = weights * (dweights - (dweights * weights).sum(1, keepdim=True))
        dlogits = torch.zeros((dout.shape[0], self.experts), device=dout.device).scatter_(1, ids, dtop)
        drouter = dlogits.T @ n.y.float()
        dy = (dy.float() + dlogits @ self.router).to(dy.dtype)
        dx, dnorm = mx.rmsnorm_backward(dy, n.h, n.rstd, self.norm, dh=dout)
        return dx, dnorm, drouter


def make_block(hidden, inner, experts, topk, seed=0, device="cuda"):
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)

    def normal(*shape, scale):
        return torch.randn(shape, generator=gen, device=device) * scale

    w1 = torch.stack([normal(2 * inner, hidden, scale=hidden ** -0.5).to(torch.bfloat16) for _ in range(experts)])
    w2 = torch.stack([normal(hidden, inner, scale=inner ** -0.5).to(torch.bfloat16) for _ in range(experts)])
    return MoeBlock((1 + normal(hidden, scale=0.1)).to(torch.bfloat16), normal(experts, hidden, scale=hidden ** -0.5),
                    w1, w2, topk), w1, w2


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--inner", type=int, default=14336)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--topk", type=int, default=2)
    a = ap.parse_args()
    block, _, _ = make_block(a.hidden, a.inner, a.experts, a.topk)
    x, r, dout = (torch.randn((a.tokens, a.hidden), device="cuda").to(torch.bfloat16) for _ in range(3))

    def step():
        out, saved = block.forward(x, r)
        return out, block.backward(dout, saved)

    for _ in range(3):
        step()
    t = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
    torch.cuda.synchronize()
    t[0].record()
    out, saved = block.forward(x, r)
    t[1].record()
    dx, dnorm, drouter = block.backward(dout, saved)
    t[2].record()
    mx.check_device_status()
    print(f"{a.tokens} tokens, hidden {a.hidden}, {a.experts} experts of {a.inner}, top {a.topk}: "
          f"forward {t[0].elapsed_time(t[1]):.3f} ms, backward {t[1].elapsed_time(t[2]):.3f} ms; "
          f"|out| {out.float().norm():.4g}, |dx| {dx.float().norm():.4g}, |dnorm| {dnorm.norm():.4g}, "
          f"|drouter| {drouter.norm():.4g}")


if __name__ == "__main__":
    main()
