"""The 64-bit references of the model's row operators: gradients against differences,
values against plain formulas (no GPU)."""
import numpy as np
import pytest

import model_ops_ref as ref


def _difference(f, x, d, eps=1e-6):
    return (f(x + eps * d) - f(x - eps * d)) / (2 * eps)


def test_embed_gradient_is_the_transpose():
    rng = np.random.default_rng(0)
    table, dy = rng.standard_normal((7, 4)), rng.standard_normal((9, 4))
    ids = np.array([0, 6, 6, -1, 3, 7, 6, 2, 0])
    out, _ = ref.embed(table, ids, 1.7)
    d, _ = ref.embed_backward(dy, ids, 7, 1.7)
    assert np.isclose((out * dy).sum(), (table * d).sum())
    assert (out[[3, 5]] == 0).all() and (d[[1, 4, 5]] == 0).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm,rotary", [(True, 16), (True, 32), (False, 16), (True, 0)])
def test_heads_gradient_against_differences(interleaved, norm, rotary):
    rng = np.random.default_rng(rotary)
    T, Q, K, D = 5, 2, 1, 32
    x, dy = rng.standard_normal((T, Q + K, D)), rng.standard_normal((T, Q + K, D))
    qw, kw = (rng.standard_normal(D), rng.standard_normal(D)) if norm else (None, None)
    a = rng.standard_normal((11, max(rotary, 2) // 2))
    rope = np.concatenate([np.cos(a), np.sin(a)], 1) if rotary else None
    pos = np.array([0, 10, -1, 3, 11])

    def f(x, qw, kw):
        return (ref.qk_norm_rope(x, Q, qw, kw, 1e-5, rope, pos, interleaved)[0] * dy).sum()
    rstd = ref.qk_norm_rope(x, Q, qw, kw, 1e-5, None, pos, interleaved)[2]
    dx, _, dq, _, dk, _ = ref.qk_norm_rope_backward(dy, x if norm else None, rstd, Q, qw, kw, rope, pos, interleaved)
    d = rng.standard_normal(x.shape)
    assert np.isclose(_difference(lambda v: f(v, qw, kw), x, d), (dx * d).sum(), rtol=1e-5)
    if norm:
        d = rng.standard_normal(D)
        assert np.isclose(_difference(lambda v: f(x, v, kw), qw, d), (dq * d).sum(), rtol=1e-5)
        assert np.isclose(_difference(lambda v: f(x, qw, v), kw, d), (dk * d).sum(), rtol=1e-5)


def test_logprobs_gradient_against_differences():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((6, 23)) * 3
    x[1, 4:9] = -np.inf
    t = np.array([0, 2, 22, -100, 5, 23])
    g, h = rng.standard_normal(6), rng.standard_normal(6)

    def f(x):
        r = ref.logprobs(x, t, 0.7)
        return (r["logprob"] * g + r["entropy"] * h).sum()
    r = ref.logprobs(x, t, 0.7)
    dx, _ = ref.logprobs_backward(x, t, np.stack([r["m"], r["log"]], 1), 0.7, g, r["entropy"], h)
    d = rng.standard_normal(x.shape)
    assert np.isclose(_difference(f, x, np.where(np.isfinite(x), d, 0)), (dx * d)[np.isfinite(x)].sum(), rtol=1e-5)
    assert (dx[1, 4:9] == 0).all()


def test_logprobs_of_masked_rows():
    x = np.full((3, 5), -np.inf)
    x[1, 3] = 2.0
    x[2] = -3e38
    r = ref.logprobs(x, np.array([1, 3, 0]), 1.0)
    assert r["logprob"][0] == -np.inf and r["logprob"][1] == 0 and np.isclose(r["logprob"][2], -np.log(5))
    assert r["entropy"][0] == 0 and r["entropy"][1] == 0 and np.isclose(r["entropy"][2], np.log(5))
    ids, lp = ref.top(x, r["z"], r["lns"], 3)
    assert ids.tolist() == [[-1, -1, -1], [3, -1, -1], [0, 1, 2]] and lp[1, 0] == 0
