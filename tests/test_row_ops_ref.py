"""The 64-bit references of the row operators, pinned without a GPU: the gradients
against central differences, the MX check against the oracle's quantiser."""
import numpy as np
import pytest

import row_ops_ref as ref


def _slope(f, x, v, step=1e-6):
    """Central difference of the scalar f along v."""
    return (f(x + step * v) - f(x - step * v)) / (2 * step)


def _close(a, b):
    assert abs(a - b) <= 1e-7 * max(1.0, abs(a), abs(b)), (a, b)


@pytest.mark.parametrize("K", [32, 96])
def test_rmsnorm_gradient_against_differences(K):
    rng = np.random.default_rng(K)
    x, r, w = rng.standard_normal((5, K)), rng.standard_normal((5, K)), 1 + rng.standard_normal(K) / 5
    dy, dh = rng.standard_normal((5, K)), rng.standard_normal((5, K))

    def loss(x, w):
        h, _, y = ref.rmsnorm(x, w, 1e-5, r)
        return (y * dy).sum() + (h * dh).sum()

    h, rstd, _ = ref.rmsnorm(x, w, 1e-5, r)
    dx, _, dw, _ = ref.rmsnorm_backward(dy, h, rstd, w, dh)
    v, vw = rng.standard_normal(x.shape), rng.standard_normal(K)
    _close(_slope(lambda z: loss(z, w), x, v), (dx * v).sum())
    _close(_slope(lambda z: loss(x, z), w, vw), (dw * vw).sum())


@pytest.mark.parametrize("act", [ref.ACT_SILU, ref.ACT_GELU])
def test_glu_gradient_against_differences(act):
    rng = np.random.default_rng(act)
    g, u, dy = (rng.standard_normal((4, 64)) * 2 for _ in range(3))
    dg, _, du, _ = ref.glu_backward(dy, g, u, act)
    v = rng.standard_normal(g.shape)
    _close(_slope(lambda z: (ref.glu(z, u, act)[0] * dy).sum(), g, v), (dg * v).sum())
    _close(_slope(lambda z: (ref.glu(g, z, act)[0] * dy).sum(), u, v), (du * v).sum())


def test_glu_against_torch():
    torch = pytest.importorskip("torch")
    g = torch.linspace(-9, 9, 257, dtype=torch.float64)
    one = np.ones(257)
    for act, f in ((ref.ACT_SILU, torch.nn.functional.silu),
                   (ref.ACT_GELU, lambda z: torch.nn.functional.gelu(z, approximate="tanh"))):
        assert np.allclose(ref.glu(g.numpy(), one, act)[0], f(g).numpy(), rtol=1e-13, atol=1e-15)


def test_combine_gradient_against_differences():
    rng = np.random.default_rng(3)
    T, k, G, N = 7, 3, 4, 32
    ids = rng.integers(-1, G, (T, k))
    _, slot, _ = ref.moe_sort(ids, G)
    y, w, dout = rng.standard_normal((T * k, N)), rng.random((T, k)), rng.standard_normal((T, N))
    dy, dw, _ = ref.moe_combine_backward(dout, y, slot, w)
    vy, vw = rng.standard_normal(y.shape), rng.standard_normal(w.shape)
    _close(_slope(lambda z: (ref.moe_combine(z, slot, k, w)[0] * dout).sum(), y, vy), (dy * vy).sum())
    _close(_slope(lambda z: (ref.moe_combine(y, slot, k, z)[0] * dout).sum(), w, vw), (dw.reshape(w.shape) * vw).sum())


def test_dispatch_is_the_transpose_of_combine_without_weights():
    rng = np.random.default_rng(4)
    T, k, G, N = 9, 2, 5, 32
    _, slot, _ = ref.moe_sort(rng.integers(-1, G, (T, k)), G)
    x, y = rng.standard_normal((T, N)), rng.standard_normal((T * k, N))
    sent = np.zeros_like(y)
    for s, row in enumerate(slot):
        if row >= 0:
            sent[row] = x[s // k]
    _close((sent * y).sum(), (x * ref.moe_combine(y, slot, k)[0]).sum())


@pytest.mark.parametrize("fmt", [1, 2])
def test_mx_check_accepts_the_oracle_and_rejects_a_changed_code(oracle_mod, fmt):
    rng = np.random.default_rng(fmt)
    x = (rng.standard_normal((6, 256)) * np.exp2(rng.integers(-40, 40, (6, 1)))).astype(np.float32)
    x[2, 64:96] = 0
    x[4, 7] = np.nan
    codes, scales = oracle_mod.quantize(fmt, x, oracle_mod.IN_F32)
    ref.assert_mx(codes, scales, x.astype(np.float64), 0.0, fmt, "oracle")
    planted = codes.copy()
    planted[3, 5] ^= 1
    with pytest.raises(AssertionError):
        ref.assert_mx(planted, scales, x.astype(np.float64), 0.0, fmt, "planted")
    planted = scales.copy()
    planted[1, 3] += 1
    with pytest.raises(AssertionError):
        ref.assert_mx(codes, planted, x.astype(np.float64), 0.0, fmt, "planted")


def test_sort_reference_by_hand():
    offsets, row, slot = ref.moe_sort(np.array([[2, 0], [-1, 2], [0, 7]]), 3)
    assert offsets.tolist() == [0, 2, 2, 4]
    assert row.tolist() == [2, 0, -5, 3, 1, -6]     # slots 2 (id -1) and 5 (id 7) are dropped
    assert slot.tolist() == [1, 4, 0, 3, 2, 5]
