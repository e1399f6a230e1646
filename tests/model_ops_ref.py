"""64-bit references (numpy) of the row operators at a model's ends and between its
products, and how far a kernel may be from them.

Every function takes 64-bit arrays holding exactly what the kernel was given and
returns the definition's value with an error bound that counts the roundings on the
kernel's path (``U``: FP32's unit roundoff), so none is fitted to a result.
"""
from __future__ import annotations

import numpy as np

from row_ops_ref import U


# ---- embedding --------------------------------------------------------------------

def embed(table, ids, scale):
    """(out, bound): one FP32 product."""
    real = (ids >= 0) & (ids < table.shape[0])
    out = np.where(real[:, None], table[np.where(real, ids, 0)] * scale, 0.0)
    return out, U * np.abs(out)


def embed_backward(dy, ids, vocab, scale, add=None):
    """(dtable, bound): an id's n rows are added one by one or in parts, n roundings at most, then one fused
    multiply-add."""
    real = (ids >= 0) & (ids < vocab)
    out, size = np.zeros((vocab, dy.shape[1])), np.zeros((vocab, dy.shape[1]))
    np.add.at(out, ids[real], dy[real])
    np.add.at(size, ids[real], np.abs(dy[real]))
    n = np.bincount(ids[real], minlength=vocab)[:, None]
    out, size = out * scale, size * abs(scale) * (n + 1) * U
    return (out, size) if add is None else (out + add, size + U * np.abs(out + add))


# ---- norm and rotation of heads -----------------------------------------------------

def _turn(x, cos, sin, rotary, interleaved):
    """(x turned, |terms|): a cos - b sin, b cos + a sin."""
    i = np.arange(rotary // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)
    y, size = x.copy(), np.abs(x)
    y[..., a], y[..., b] = x[..., a] * cos - x[..., b] * sin, x[..., b] * cos + x[..., a] * sin
    size[..., a] = np.abs(x[..., a] * cos) + np.abs(x[..., b] * sin)
    size[..., b] = np.abs(x[..., b] * cos) + np.abs(x[..., a] * sin)
    return y, size


def _angles(rope, positions, rotary):
    real = (positions >= 0) & (positions < rope.shape[0])
    a = rope[np.where(real, positions, 0)][:, None]
    return real, a[..., :rotary // 2], a[..., rotary // 2:]


def _weights(q_weight, k_weight, q_heads, heads, D):
    w = np.ones((heads, D))
    if q_weight is not None:
        w[:q_heads] = q_weight
    if k_weight is not None:
        w[q_heads:] = k_weight
    return w


# sums of squares or products: eight in a chain, two halves, five levels of a tree
HEAD_CHAIN = 8 + 1 + 5


def qk_norm_rope(x, q_heads, q_weight, k_weight, eps, rope, positions, interleaved):
    """(y, bound, rstd, relative bound of rstd).  x [tokens, heads, D].

    rstd: half of the sum's relative error, the three roundings before the root, the root's two units in the last
    place (4 U).  y: rstd's, two products, then a product and a fused multiply-add."""
    T, H, D = x.shape
    rstd, rel = None, 0.0
    v = x
    if q_weight is not None or k_weight is not None:
        rstd = 1.0 / np.sqrt((x * x).mean(2) + eps)
        rel = ((HEAD_CHAIN + 3) / 2 + 4) * U
        v = x * rstd[..., None] * _weights(q_weight, k_weight, q_heads, H, D)
    size = np.abs(v)
    if rope is not None:
        real, cos, sin = _angles(rope, positions, rope.shape[1])
        v, size = _turn(v, cos, sin, rope.shape[1], interleaved)
        v, size = np.where(real[:, None, None], v, 0.0), np.where(real[:, None, None], size, 0.0)
        if rstd is not None:
            rstd = np.where(real[:, None], rstd, 0.0)
    return v, (rel + 4 * U) * size, rstd, rel


def qk_norm_rope_backward(dy, x, rstd, q_heads, q_weight, k_weight, rope, positions, interleaved):
    """(dx, bound, dq, bound, dk, bound); x and rstd None for the rotation alone."""
    T, H, D = dy.shape
    g, size = dy, np.abs(dy)
    real = np.ones(T, bool)
    if rope is not None:
        real, cos, sin = _angles(rope, positions, rope.shape[1])
        g, size = _turn(dy, cos, -sin, rope.shape[1], interleaved)
        g, size = np.where(real[:, None, None], g, 0.0), np.where(real[:, None, None], size, 0.0)
    eg = 2 * U * size
    if x is None:
        return g, eg, None, None, None, None
    w = _weights(q_weight, k_weight, q_heads, H, D)
    r = np.where(real[:, None], rstd, 0.0)[..., None]
    n = np.where(real[:, None, None], x, 0.0) * r
    gw = g * w
    dot = (gw * n).mean(2, keepdims=True)
    # the dot product's terms carry g's error and three roundings, its sum the chain's, the mean two more
    edot = (np.abs(w * n) * eg + np.abs(gw * n) * (HEAD_CHAIN + 5) * U).mean(2, keepdims=True)
    dx = r * (gw - n * dot)
    edx = r * (np.abs(w) * eg + np.abs(gw) * 3 * U + np.abs(n) * edot + np.abs(n * dot) * 4 * U)
    t, et = g * n, np.abs(n) * eg + np.abs(g * n) * 2 * U
    terms = np.abs(t)

    def part(s):
        count = T * max(1, t[:, s].shape[1])  # no sum takes more roundings than it has terms
        return t[:, s].sum((0, 1)), et[:, s].sum((0, 1)) + (count + 40) * U * terms[:, s].sum((0, 1))
    return dx, edx, *part(slice(0, q_heads)), *part(slice(q_heads, H))


# ---- log probabilities ---------------------------------------------------------------

MARGIN = 3.0  # of a thread's reference, in powers of two


def _exponents(z, chain):
    """(p, ln S, relative bound of S) for z = scale (x - max).

    Every 2^t is off by ex2's two units in the last place (4 U) and its argument by 4 U of itself (the factor's two
    roundings, the difference, the product); the sum is rebased at most five times (a thread's moves, the warp, the
    block, the row), each time by such a factor, of an exponent no further off than the term's own and the margin."""
    with np.errstate(invalid="ignore"):
        e = np.where(z > -np.inf, np.exp(z), 0.0)
    S = e.sum(1, keepdims=True)
    p = e / S
    t = np.where(p > 0, np.abs(np.where(z > -np.inf, z, 0.0)), 0.0)
    mean_t = (p * t).sum(1, keepdims=True)
    rel = U * (chain + 5 * (4 + 4 * MARGIN) + 6 * 4 * mean_t)
    return p, np.log(S), rel, t


def logprobs(x, targets, scale, chain=None):
    """dict of logprob, entropy, stats and their bounds; rows without a value above -inf included (not NaN or +inf)."""
    rows, V = x.shape
    chain = V / 64 + 24 if chain is None else chain
    m = x.max(1, keepdims=True)
    none = ~(m > -np.inf)
    with np.errstate(invalid="ignore"):
        z = np.where(x > -np.inf, (x - np.where(none, 0.0, m)) * scale, -np.inf)
        p, lns, rel, t = _exponents(np.where(none, 0.0, z), chain)
    lns = np.where(none, 0.0, lns)
    real = (targets >= 0) & (targets < V)
    zt = z[np.arange(rows), np.where(real, targets, 0)]
    logp = np.where(real, np.where(none[:, 0], -np.inf, zt - lns[:, 0]), 0.0)
    q, q2 = (p * t).sum(1), (p * t * t).sum(1)
    entropy = np.where(none[:, 0], 0.0, lns[:, 0] + q)
    log_err = rel[:, 0] + 2 * U * np.abs(lns[:, 0])
    with np.errstate(invalid="ignore"):
        lp_err = np.where(np.isfinite(logp), log_err + 2 * U * np.abs(zt) + U * np.abs(logp), 0.0)
    # the mean of z: its terms' errors (the exponents' weigh by z again), the sums', the rebased differences
    en_err = log_err + 24 * U * q2 + q * (2 * rel[:, 0] + 8 * U) + U * 10 * MARGIN + U * entropy
    return dict(logprob=logp, logprob_err=lp_err, entropy=entropy, entropy_err=en_err,
                m=m[:, 0], log=lns[:, 0], log_err=log_err, z=z, lns=lns)


def top(x, z, lns, count):
    """ids and log probabilities of the largest, equal ones by id; -1 and -inf past those with a probability."""
    order = np.argsort(np.where(np.isnan(x), np.inf, -x), axis=1, kind="stable")[:, :count]
    v = np.take_along_axis(x, order, 1)
    ok = (v > -np.inf) & ~np.isnan(v)
    ids = np.full((x.shape[0], count), -1, np.int64)
    lp = np.full((x.shape[0], count), -np.inf)
    ids[:, :order.shape[1]] = np.where(ok, order, -1)
    lp[:, :order.shape[1]] = np.where(ok, np.take_along_axis(z, order, 1) - lns, -np.inf)
    return ids, lp


def logprobs_backward(x, targets, stats, scale, dlogprob=None, entropy=None, dentropy=None):
    """(dlogits, bound)."""
    rows, V = x.shape
    m, lns = stats[:, :1], stats[:, 1:]
    none = ~(m > -np.inf)
    with np.errstate(invalid="ignore"):
        z = np.where(x > -np.inf, (x - np.where(none, 0.0, m)) * scale, -np.inf)
    logp = z - lns
    p = np.where(none, 0.0, np.exp(np.where(none, 0.0, logp)))
    zf, lf = np.where(np.isfinite(z), z, 0.0), np.where(np.isfinite(logp), logp, 0.0)
    et = U * (4 * np.abs(zf) + 3 * np.abs(lns) + np.abs(lf))           # of ln p
    rp = et + 4 * U                                                    # relative, of p
    out, err = np.zeros_like(x), np.zeros_like(x)
    g = np.zeros((rows, 1))
    if dlogprob is not None:
        real = (targets >= 0) & (targets < V)
        g = np.where(real, dlogprob, 0.0)[:, None]
        out -= g * p
        hit = (np.arange(V) == np.where(real, targets, -1)[:, None]) & ~none
        out += np.where(hit, g, 0.0)
        err += np.where(hit, 2 * U * np.abs(g), 0.0)
    err += np.abs(g * p) * (rp + 4 * U)
    if dentropy is not None:
        h, H = dentropy[:, None], entropy[:, None]
        out -= np.where(p > 0, h * p * (lf + H), 0.0)
        err += np.abs(h) * p * ((np.abs(lf) + np.abs(H)) * (rp + 6 * U) + et)
    # a probability below 2^-126 is 0
    return out * scale, scale * (err + U * np.abs(out) + 2.0 ** -126 * (np.abs(g) + 200.0 * (dentropy is not None)))


# ---- norm and clipping ---------------------------------------------------------------

# sixteen squares in a chain and two halves at most, on in 64 bits; the root halves that, rounds once, the sum twice before
NORM_REL = ((16 + 1) / 2 + 3) * U


def clip(grads, max_norm):
    """(norm, factor, relative bound of the factor)."""
    norm = np.sqrt(sum(float((g.astype(np.float64) ** 2).sum()) for g in grads))
    return norm, min(1.0, max_norm / (norm + 1e-6)), NORM_REL + 3 * U
