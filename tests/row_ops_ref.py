"""64-bit references (numpy) of the row operators, and how far a kernel may be from them.

Every function takes 64-bit arrays holding exactly what the kernel was given
and returns the definition's value, with an error bound where it sums or
exponentiates: ``U`` is FP32's unit roundoff and each bound counts the roundings
on the kernel's path, so none is fitted to a result.
"""
from __future__ import annotations

import math

import numpy as np

U = 2.0 ** -24          # FP32 unit roundoff
UB = 2.0 ** -8          # BF16's (8-bit significand)
TINY_F32 = 2.0 ** -149
TINY_BF16 = 2.0 ** -133
ACT_SILU, ACT_GELU = 1, 2


def stored(err, value, bf16):
    """Bound after the final rounding: nothing more in FP32 (already counted), half an ulp in BF16."""
    return err + (UB * (np.abs(value) + err) + TINY_BF16 if bf16 else U * np.abs(value) + TINY_F32)


def assert_near(got, want, err, bf16, what):
    got = np.asarray(got, np.float64)
    lim = stored(err, want, bf16)
    same = np.isnan(got) & np.isnan(want) | (got == want)
    bad = ~same & ~(np.abs(got - want) <= lim)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} out of bounds, first at {i}: {got[i]!r} for "
                             f"{want[i]!r} (limit {lim[i]:.3g})")


# ---- MX ---------------------------------------------------------------------------

def grid_round(v, fmt):
    """Nearest E4M3 (fmt 1) or E2M1 (fmt 2) value of v, ties to even, saturating."""
    low, bits, most = (-6, 3, 448.0) if fmt == 1 else (0, 1, 6.0)
    _, e = np.frexp(v)
    q = np.maximum(e - 1, low) - bits
    return np.clip(np.ldexp(np.rint(np.ldexp(v, -q)), q), -most, most)


def decode_codes(codes, fmt):
    if fmt == 1:
        c = codes.astype(np.int64)
        m, e, s = c & 7, (c >> 3) & 15, np.where(c & 128, -1.0, 1.0)
        v = np.where(e > 0, (8 + m) * np.exp2(e - 10.0), m * 2.0 ** -9)
        return np.where((c & 127) == 127, np.nan, s * v)
    n = np.empty((codes.shape[0], codes.shape[1] * 2), np.int64)
    n[:, 0::2], n[:, 1::2] = codes & 15, codes >> 4
    mag = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])[n & 7]
    return np.where(n & 8, -mag, mag)


def untile(tiled, rows, K):
    """Row-major [rows, K/32] scales of the 512-byte tile layout; the padding rows must hold 127."""
    t = np.asarray(tiled).reshape(-1, K // 128, 32, 4, 4)       # block, K-tile, p, q, c
    r = t.transpose(0, 3, 2, 1, 4).reshape(-1, K // 32)         # row 128R + 32q + p, block 4T + c
    assert (r[rows:] == 127).all(), "padding rows of the tile layout"
    return r[:rows]


def assert_mx(codes, scales, value, err, fmt, what):
    """codes and scales are the MX encoding of some x with |x - value| <= err.

    The scale code must be that of an amax within the bound, and given the scale,
    rounding is monotone: every element lies between the encodings of value - err
    and value + err.
    """
    rows, K = value.shape
    emax = 8 if fmt == 1 else 2
    v, b = value.reshape(rows, -1, 32), np.broadcast_to(err, value.shape).reshape(rows, -1, 32)
    finite = np.isfinite(v).all(-1)
    scales = np.asarray(scales).astype(np.int64)
    assert (scales[~finite] == 255).all(), f"{what}: scale of a block with a NaN or an infinity"

    def code_of(amax):
        e = np.frexp(amax)[1] - 1
        return np.where(amax > 0, np.maximum(e - emax, -127) + 127, 127)

    mag = np.abs(np.where(finite[..., None], v, 0.0))
    hi, lo = code_of((mag + b).max(-1)), code_of(np.maximum(mag - b, 0).max(-1))
    ok = ~finite | (scales >= np.minimum(lo, hi)) & (scales <= np.maximum(lo, hi))
    assert ok.all(), f"{what}: scale {scales[~ok][0]} outside {lo[~ok][0]}..{hi[~ok][0]} at {np.argwhere(~ok)[0]}"
    step = np.ldexp(1.0, np.where(finite, scales, 127) - 127)[..., None]
    got = decode_codes(np.asarray(codes), fmt).reshape(rows, -1, 32)
    assert (got[~finite] == 0).all(), f"{what}: codes of a block with a NaN or an infinity"
    vz = np.where(finite[..., None], v, 0.0)
    low, high = grid_round((vz - b) / step, fmt), grid_round((vz + b) / step, fmt)
    bad = finite[..., None] & ~((got >= low) & (got <= high))
    assert not bad.any(), (f"{what}: {bad.sum()} codes outside their bounds, first {got[bad][0]} not in "
                           f"{low[bad][0]}..{high[bad][0]} at {np.argwhere(bad)[0]}")


# ---- RMS norm ---------------------------------------------------------------------

def rmsnorm(x, w, eps, r=None):
    """(h, rstd, y)."""
    h = x if r is None else x + r
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h, rstd, h * rstd[:, None] * w


def rmsnorm_rel():
    """Relative error of rstd and of y.  A thread sums at most 64 values in a chain,
    then come at most twelve tree steps; all terms are positive, each square
    carries h's rounding twice; the root halves the sum's error; division by K, the
    addition of eps, the root, and y's two products round once each."""
    chain = 64 + 12
    rstd = (chain + 2 + 2) / 2 * U + U
    return rstd, rstd + 3 * U


def rmsnorm_backward(dy, h, rstd, w, dh=None):
    """(dx, error bound of dx, dw, sum of |terms| of dw)."""
    p, r = dy * w, rstd[:, None]
    m = (p * h).mean(1, keepdims=True)
    dx = r * p - h * r ** 3 * m
    # p*h: one rounding each and chains as in the forward; rstd^3/K: four roundings; the last subtraction and addition
    chain = 64 + 12
    err = (np.abs(r * p) * 4 + np.abs(h) * r ** 3 * np.abs(p * h).mean(1, keepdims=True) * (chain + 8)) * U
    if dh is not None:
        dx = dx + dh
        err = err + 2 * U * np.abs(dh)
    err = err + 2 * U * np.abs(dx)
    t = dy * h * r
    return dx, err, t.sum(0), np.abs(t).sum(0)


# ---- gated activation -------------------------------------------------------------

def _gate(g, act):
    """(q, the activation's inner argument t, dt/dg): act(g) = g q, q = 1 / (1 + exp(-t))."""
    c = math.sqrt(8 / math.pi)
    t = g if act == ACT_SILU else c * (g + 0.044715 * g ** 3)
    slope = np.ones_like(g) if act == ACT_SILU else c * (1 + 0.134145 * g * g)
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-t)), t, slope


def _gate_rel(q, t):
    """q's relative error: t has six roundings (constants included), which move exp by |t| as much and q by 1 - q of
    that; exp is within two ulps, then an addition and a division."""
    return (8 + 7 * np.abs(t) * (1 - q)) * U


# exp(-t) overflows FP32 where q < 2^-127: q is then 0, off by less than this
Q_FLOOR = 2.0 ** -126


def glu(g, u, act):
    """(a, error bound)."""
    q, t, _ = _gate(g, act)
    a = g * q * u
    return a, (_gate_rel(q, t) + 3 * U) * np.abs(a) + Q_FLOOR * np.abs(g * u)


def glu_backward(dy, g, u, act):
    """(dg, bound, du, bound)."""
    q, t, slope = _gate(g, act)
    f, rel = g * q, _gate_rel(q, t)
    part = np.abs(f) * slope
    dg = dy * u * (q + f * (1 - q) * slope)
    # 1 - q is off by q's own error and one rounding; the products and the addition by a few more
    edg = np.abs(dy * u) * (q * (rel + 4 * U) + part * (1 - q) * (rel + 10 * U) + part * (q * rel + U)
                            + Q_FLOOR * (1 + 2 * np.abs(g) * slope))
    du = dy * f
    return dg, edg, du, (rel + 3 * U) * np.abs(du) + Q_FLOOR * np.abs(dy * g)


# ---- expert routing ---------------------------------------------------------------

def moe_sort(ids, groups):
    """(offsets, row_of_slot, slot_of_row)."""
    flat = np.asarray(ids).reshape(-1)
    key = np.where((flat >= 0) & (flat < groups), flat, groups)
    order = np.argsort(key, kind="stable")
    row = np.empty(flat.size, np.int64)
    row[order] = np.arange(flat.size)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=groups + 1)[:groups])])
    return offsets, np.where(key < groups, row, -1 - row), order


def moe_combine(y, row_of_slot, topk, weights=None, add=None):
    """(out, error bound)."""
    s = row_of_slot.reshape(-1, topk)
    live = s >= 0
    w = np.where(live, 1.0 if weights is None else weights.reshape(s.shape), 0.0)
    t = np.where(live[..., None], y[np.where(live, s, 0)], 0.0) * w[..., None]
    out, size = t.sum(1), np.abs(t).sum(1)
    if add is not None:
        out, size = out + add, size + np.abs(add)
    return out, (topk + 2) * U * size


def moe_combine_backward(dout, y, row_of_slot, weights):
    """(dy, dweights, dweights' bound)."""
    topk = row_of_slot.size // dout.shape[0]
    s = row_of_slot.reshape(-1)
    live, tok = s >= 0, np.arange(s.size) // topk
    row = np.where(live, s, -1 - s)
    dy = np.zeros_like(y)
    dy[row[live]] = weights.reshape(-1, 1)[live] * dout[tok[live]]
    t = np.zeros((s.size, dout.shape[1]))
    t[live] = dout[tok[live]] * y[row[live]]
    return dy, t.sum(1), (dout.shape[1] / 32 + 8) * U * np.abs(t).sum(1)
