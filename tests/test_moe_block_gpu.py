"""The example's mixture-of-experts block against a 64-bit computation of the same
steps (rounded to BF16 and MXFP8 where the block stores those)."""
import os
import sys

import numpy as np
import pytest

from gpu_util import lib

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _mx(v):
    """64-bit values of the MXFP8 encoding along the last axis."""
    import torch
    b = v.reshape(*v.shape[:-1], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    s = torch.where(amax > 0, torch.frexp(amax).exponent - 9, 0).double()
    t = b * torch.exp2(-s)
    q = torch.exp2(((torch.frexp(t).exponent - 1).clamp(min=-6) - 3).double())
    return ((torch.round(t / q) * q).clamp(-448, 448) * torch.exp2(s)).reshape(v.shape)


def _bf(v):
    import torch
    return v.to(torch.bfloat16).double()


def _rel(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("tokens,hidden,inner,experts,topk", [(1, 256, 128, 4, 2), (300, 512, 256, 8, 2),
                                                              (77, 256, 384, 64, 8)])
def test_block(tokens, hidden, inner, experts, topk):
    import torch
    lib()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import moe_block
    block, w1, w2 = moe_block.make_block(hidden, inner, experts, topk, seed=tokens)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(tokens)
    x, r, dout = (torch.randn((tokens, hidden), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(3))
    out, saved = block.forward(x, r)
    dx, dnorm, drouter = block.backward(dout, saved)
    moe_block.mx.check_device_status()
    ids, weights = saved[1], saved[2].double()

    F = inner
    h = x.double() + r.double()
    rstd = (h.pow(2).mean(1, keepdim=True) + block.eps).rsqrt()
    y = _bf(h * rstd * block.norm.double())
    want = torch.zeros_like(h)
    dy, dw = torch.zeros_like(h), torch.zeros_like(weights)
    yq, hs = _mx(y), _bf(h)
    m1, m2 = _mx(w1.double()), _mx(w2.double())
    m1t, m2t = _mx(w1.double().transpose(1, 2).contiguous()), _mx(w2.double().transpose(1, 2).contiguous())
    for t in range(tokens):
        for j in range(topk):
            e, d = int(ids[t, j]), dout[t].double()
            gu = _bf(m1[e] @ yq[t])
            q = torch.sigmoid(gu[:F])
            z = _bf(m2[e] @ _mx(gu[:F] * q * gu[F:]))
            want[t] += weights[t, j] * z
            dw[t, j] = d @ z
            da = _bf(m2t[e] @ _mx(_bf(weights[t, j] * d)))
            kept = _mx(gu)
            g, u = kept[:F], kept[F:]
            q = torch.sigmoid(g)
            dgu = torch.cat([da * u * (q + g * q * (1 - q)), da * g * q])
            dy[t] += _bf(m1t[e] @ _mx(dgu))
    want = want + h
    dtop = weights * (dw - (dw * weights).sum(1, keepdim=True))
    dlogits = torch.zeros((tokens, experts), dtype=torch.float64, device="cuda").scatter_(1, ids, dtop)
    p = (_bf(dy) + dlogits @ block.router.double()) * block.norm.double()
    wdx = rstd * p - hs * rstd ** 3 * (p * hs).mean(1, keepdim=True) + dout.double()
    wdn = ((_bf(dy) + dlogits @ block.router.double()) * hs * rstd).sum(0)
    # BF16 results are off by half an ulp, 2^-9 on average.  An FP32 sum's last bits (2^-20 of a value) turn a BF16
    # rounding (step 2^-8) with a chance of 2^-12, by 2^-8 of the value, and that an E4M3 rounding (step 2^-3) with a
    # chance of 2^-5 more, by 2^-3: the root mean square of either is below 2^-11.
    assert _rel(out, want) < 2.0 ** -8
    assert _rel(dx, wdx) < 2.0 ** -7
    assert _rel(dnorm, wdn) < 2.0 ** -7
    assert _rel(drouter, dlogits.T @ y) < 2.0 ** -7
