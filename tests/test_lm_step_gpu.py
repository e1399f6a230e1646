"""The example's training step, ids to clipped gradients, against 64-bit autograd of the
same model."""
import os
import sys

import pytest

from gpu_util import lib

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _loss(m, w, ids, positions, targets, sequence, beta, attention):
    """The example's loss from 64-bit weights, in elementary torch operations."""
    import torch
    Q, K, D, T = m.q_heads, m.k_heads, m.D, ids.numel()
    real = ids >= 0

    def norm(x, weight):
        return x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + 1e-6) * weight
    x = torch.where(real[:, None], w["table"][torch.where(real, ids, 0)], 0.0) * m.scale
    qkv = (norm(x, w["norm1"]) @ w["qkv"].T).view(T, Q + 2 * K, D)
    qk = torch.cat([norm(qkv[:, :Q], w["q_norm"]), norm(qkv[:, Q:Q + K], w["k_norm"])], 1)
    placed = positions >= 0
    angles = m.rope.double()[torch.where(placed, positions, 0)][:, None]
    cos, sin = angles[..., :D // 2], angles[..., D // 2:]
    a, b = qk[..., :D // 2], qk[..., D // 2:]
    qk = torch.where(placed[:, None, None], torch.cat([a * cos - b * sin, b * cos + a * sin], -1), 0.0)
    h = x + attention(qk[:, :Q], qk[:, Q:], qkv[:, Q + K:], sequence).reshape(T, Q * D) @ w["out"].T
    logp = torch.log_softmax(norm(h, w["norm2"]) @ w["table"].T, -1)
    counted = (targets >= 0) & (targets < logp.shape[1])
    count = counted.sum()
    lp = torch.where(counted, logp.gather(1, torch.where(counted, targets, 0)[:, None])[:, 0], 0.0)
    entropy = -(logp.exp() * logp).sum(-1)
    return -lp.sum() / count - beta * (entropy * counted).sum() / count


@pytest.mark.parametrize("tokens,vocab,hidden,Q,K,D,beta", [(256, 512, 256, 4, 2, 64, 0.0), (128, 1024, 128, 1, 1, 128, 0.1),
                                                            (384, 384, 384, 6, 2, 64, 0.05)])
def test_step_gradients(tokens, vocab, hidden, Q, K, D, beta):
    import torch
    lib()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import lm_step
    m = lm_step.Model(vocab, hidden, Q, K, D, positions=tokens, seed=tokens)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(tokens)
    ids = torch.randint(0, vocab, (tokens,), generator=gen, device="cuda")
    ids[:40] = 7                                            # one token many times
    sequence = torch.arange(tokens, device="cuda") // 100
    positions = torch.arange(tokens, device="cuda") % 100
    targets = torch.where(positions < 99, torch.roll(ids, -1), -100)
    ids[-9:], positions[-9:], targets[-10:], sequence[-9:] = -1, -1, -100, 1 << 20     # padding
    loss, norm, grads = m.step(ids, positions, targets, sequence, beta=beta, max_norm=0.5)
    lm_step.mx.check_device_status()

    w = {k: v.double().requires_grad_() for k, v in m.w.items()}
    want = _loss(m, w, ids, positions, targets, sequence, beta, lm_step.attention)
    want.backward()
    total = torch.sqrt(sum(v.grad.pow(2).sum() for v in w.values()))
    factor = min(1.0, 0.5 / (float(total) + 1e-6))
    # Every stored BF16 tensor is off by at most half an ulp, 2^-9 of its values in the root mean square.  A gradient's
    # path crosses at most sixteen of them (eight forwards, eight back), which are independent: 4 * 2^-9, and twice that for
    # what products and softmax make of it.  The loss averages over tokens.
    assert abs(float(loss) - float(want)) < 2.0 ** -6 * abs(float(want))
    assert abs(float(norm) - float(total)) < 2.0 ** -6 * float(total)
    for k, v in w.items():
        err = float((grads[k].double() - v.grad * factor).norm() / (v.grad * factor).norm())
        assert err < 2.0 ** -6, (k, err)


def test_example_runs():
    lib()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import lm_step
    lm_step.main()
