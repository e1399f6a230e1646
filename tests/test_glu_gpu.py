"""Gated activation with MX output and 8-bit checkpoint, and its gradient, on the
GPU against the 64-bit definition (row_ops_ref.py), through the binding."""
import numpy as np
import pytest

import row_ops_ref as ref
from gpu_util import lib
from test_rmsnorm_gpu import _dtype, _make, _np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    lib()


def _scales(t, tiled, rows, K):
    s = t.cpu().numpy()
    return ref.untile(s, rows, K) if tiled else s


@pytest.mark.parametrize("act", [ref.ACT_SILU, ref.ACT_GELU])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt,tiled", [(0, False), (1, False), (1, True), (2, False), (2, True)])
@pytest.mark.parametrize("rows,F,keep", [(1, 128, True), (5, 640, False), (131, 384, True), (2, 14336, True)])
def test_forward(oracle_mod, act, dtype, fmt, tiled, rows, F, keep):
    b = lib()
    rng = np.random.default_rng([rows, F, fmt, act])
    gu, gu64 = _make(rng, (rows, 2 * F), _dtype(dtype), 3.0)
    plain = fmt == 0 or rows == 5
    out = b.glu(gu[:, :F], gu[:, F:], act, fmt=fmt, tiled=tiled, plain=plain, keep=keep)
    a, err = ref.glu(gu64[:, :F], gu64[:, F:], act)
    if plain:
        ref.assert_near(_np(out.y), a, err, dtype == "bf16", "a")
    if fmt:
        ref.assert_mx(out.codes.cpu().numpy(), _scales(out.scales, tiled, rows, F), a, err + ref.TINY_F32, fmt, "MX(a)")
    if keep:  # the checkpoint is the quantiser on the inputs, bit for bit
        codes, scales = oracle_mod.quantize(1, gu.float().cpu().numpy(), oracle_mod.IN_F32)
        assert (out.kept_codes.cpu().numpy() == codes).all() and (out.kept_scales.cpu().numpy() == scales).all()


@pytest.mark.parametrize("F", [32, 96, 160, 1568])
def test_forward_without_whole_tiles(F):
    b = lib()
    rng = np.random.default_rng(F)
    gu, gu64 = _make(rng, (19, 2 * F), _dtype("bf16"), 2.0)
    for fmt in (1, 2):
        out = b.glu(gu[:, :F], gu[:, F:], ref.ACT_SILU, fmt=fmt, keep=True)
        a, err = ref.glu(gu64[:, :F], gu64[:, F:], ref.ACT_SILU)
        ref.assert_mx(out.codes.cpu().numpy(), out.scales.cpu().numpy(), a, err, fmt, "MX(a)")


@pytest.mark.parametrize("act", [ref.ACT_SILU, ref.ACT_GELU])
def test_far_arguments(act):
    """Gates far to both sides, where the exponential leaves FP32, and non-finite ones."""
    import torch
    b = lib()
    g = np.zeros((2, 64), np.float32)
    g[0] = np.concatenate([np.linspace(-120, 120, 56), [1e4, -1e4, 1e19, -1e19, 1e25, -1e25, -0.0, 0.0]])
    g[1, :3] = [np.nan, np.inf, -np.inf]
    u = np.ones((2, 64), np.float32)
    gd, ud = torch.from_numpy(g).cuda(), torch.from_numpy(u).cuda()
    out = b.glu(gd, ud, act, plain=True)
    with np.errstate(all="ignore"):
        a, err = ref.glu(g.astype(np.float64), u.astype(np.float64), act)
    ref.assert_near(_np(out.y)[0], a[0], err[0], False, "a")
    got = _np(out.y)[1]
    assert np.isnan(got[0]) and got[1] == np.inf and (got[3:] == 0).all()  # -inf * 0 is NaN or -0
    dgu = _np(b.glu_backward(ud, act, gate=gd, up=ud).dgu)
    far = np.abs(g[0]) >= 1e4
    assert np.array_equal(dgu[0, :64][far], (g[0][far] > 0).astype(float)), "slopes far out are 0 and 1"
    with np.errstate(all="ignore"):
        dg, e, du, ed = ref.glu_backward(u[:1].astype(np.float64), g[:1].astype(np.float64), u[:1].astype(np.float64),
                                         act)
    near = ~far
    ref.assert_near(dgu[0, :64][near], dg[0][near], e[0][near], False, "dgate")
    ref.assert_near(dgu[0, 64:][near], du[0][near], ed[0][near], False, "dup")


@pytest.mark.parametrize("act", [ref.ACT_SILU, ref.ACT_GELU])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("fmt,tiled,rows,F", [
    (0, False, 1, 32), (0, False, 7, 608), (1, False, 33, 96), (1, True, 130, 192), (1, True, 3, 1024),
    (2, False, 6, 160), (2, True, 129, 64), (2, False, 5, 512),
])
def test_backward(act, dtype, kept, fmt, tiled, rows, F):
    b = lib()
    rng = np.random.default_rng([rows, F, fmt, act])
    dt, bf16 = _dtype(dtype), dtype == "bf16"
    gu, gu64 = _make(rng, (rows, 2 * F), dt, 2.0)
    dy, dy64 = _make(rng, (rows, F), dt)
    src = dict(gate=gu[:, :F], up=gu[:, F:])
    if kept:
        f = b.glu(gu[:, :F], gu[:, F:], act, keep=True)
        src = dict(kept_codes=f.kept_codes, kept_scales=f.kept_scales)
        sc = np.exp2(f.kept_scales.cpu().numpy().astype(np.float64) - 127)
        gu64 = ref.decode_codes(f.kept_codes.cpu().numpy(), 1) * np.repeat(sc, 32, axis=1)
    g64, u64 = gu64[:, :F], gu64[:, F:]
    out = b.glu_backward(dy, act, fmt=fmt, tiled=tiled, recompute=True, **src)
    dg, edg, du, edu = ref.glu_backward(dy64, g64, u64, act)
    ref.assert_near(_np(out.dgu)[:, :F], dg, edg, bf16, "dgate")
    ref.assert_near(_np(out.dgu)[:, F:], du, edu, bf16, "dup")
    a, ea = ref.glu(g64, u64, act)
    ref.assert_near(_np(out.a), a, ea, bf16, "a")
    if fmt:
        both, err = np.concatenate([dg, du], 1), np.concatenate([edg, edu], 1) + ref.TINY_F32
        ref.assert_mx(out.codes.cpu().numpy(), _scales(out.scales, tiled, rows, 2 * F), both, err, fmt, "MX(dgu)")
        only = b.glu_backward(dy, act, fmt=fmt, tiled=tiled, plain=False, **src)
        assert only.dgu is None and (only.codes == out.codes).all() and (only.scales == out.scales).all()


@pytest.mark.parametrize("act", [ref.ACT_SILU, ref.ACT_GELU])
def test_gradient_against_differences(act):
    b = lib()
    rng = np.random.default_rng(act)
    F = 96
    gu, gu64 = _make(rng, (4, 2 * F), _dtype("f32"), 2.0)
    dy, dy64 = _make(rng, (4, F), _dtype("f32"))
    dgu = _np(b.glu_backward(dy, act, gate=gu[:, :F], up=gu[:, F:]).dgu)
    v, e = rng.standard_normal((4, 2 * F)), 1e-5
    loss = lambda z: (ref.glu(z[:, :F], z[:, F:], act)[0] * dy64).sum()  # noqa: E731
    _, edg, _, edu = ref.glu_backward(dy64, gu64[:, :F], gu64[:, F:], act)
    lim = (np.concatenate([edg, edu], 1) * np.abs(v)).sum() + ref.U * np.abs(dgu * v).sum() + 1e-8 * v.size
    assert abs((loss(gu64 + e * v) - loss(gu64 - e * v)) / (2 * e) - (dgu * v).sum()) < lim


def test_checkpoint_gradient_is_near_the_exact_one():
    """E4M3 keeps each input to within half an ulp (2^-4 of its magnitude, or of its
    block's largest where that is subnormal): the gradient moves by the slopes times that."""
    b = lib()
    rng = np.random.default_rng(12)
    F = 512
    gu, gu64 = _make(rng, (16, 2 * F), _dtype("bf16"))
    dy, dy64 = _make(rng, (16, F), _dtype("bf16"))
    f = b.glu(gu[:, :F], gu[:, F:], ref.ACT_SILU, keep=True)
    got = _np(b.glu_backward(dy, ref.ACT_SILU, kept_codes=f.kept_codes, kept_scales=f.kept_scales).dgu)
    dg, _, du, _ = ref.glu_backward(dy64, gu64[:, :F], gu64[:, F:], ref.ACT_SILU)
    want = np.concatenate([dg, du], 1)
    # |act'| <= 1.1, |act''| <= 0.5: relative to |dy| (|u| + |g|) an eighth of 2^-1
    assert np.linalg.norm(got - want) < 2.0 ** -4 * 1.6 * np.linalg.norm(
        np.concatenate([np.abs(dy64) * (np.abs(gu64[:, F:]) + np.abs(gu64[:, :F] * gu64[:, F:])),
                        np.abs(dy64 * gu64[:, :F])], 1))


def test_separate_tensors_strides_and_guards():
    import torch
    b = lib()
    rng = np.random.default_rng(3)
    rows, F = 11, 224
    gw, gw64 = _make(rng, (rows, F + 160), _dtype("bf16"))
    uw, uw64 = _make(rng, (rows, F + 160), _dtype("bf16"))
    pad = 64
    codes = torch.full((rows * F + 2 * pad,), 0xA5, dtype=torch.uint8, device="cuda")
    kept = torch.full((rows * 2 * F + 2 * pad,), 0xA5, dtype=torch.uint8, device="cuda")
    out = b.glu(gw[:, 32:32 + F], uw[:, 160:], ref.ACT_SILU, fmt=1, codes=codes[pad:-pad].view(rows, F), keep=True,
                kept_codes=kept[pad:-pad].view(rows, 2 * F))
    a, err = ref.glu(gw64[:, 32:32 + F], uw64[:, 160:], ref.ACT_SILU)
    ref.assert_mx(out.codes.cpu().numpy(), out.scales.cpu().numpy(), a, err, 1, "MX(a)")
    for t in (codes, kept):
        assert (t[:pad] == 0xA5).all() and (t[-pad:] == 0xA5).all()
    with pytest.raises(ValueError):
        b.glu(gw[:, :F], uw[:, :F].contiguous(), ref.ACT_SILU, plain=True)     # two strides


def test_offsets_past_32_bits():
    import torch
    b = lib()
    rows, F = (1 << 31) // (2 * 14336) + 9, 14336
    gu = torch.full((rows, 2 * F), 0.5, dtype=torch.bfloat16, device="cuda")
    gu[-8:] = torch.randn((8, 2 * F), device="cuda").to(torch.bfloat16)
    out = b.glu(gu[:, :F], gu[:, F:], ref.ACT_SILU, fmt=1, keep=True)
    tail = b.glu(gu[-8:, :F], gu[-8:, F:], ref.ACT_SILU, fmt=1, keep=True)
    for name in ("codes", "scales", "kept_codes", "kept_scales"):
        assert torch.equal(getattr(out, name)[-8:], getattr(tail, name)), name
    dy = torch.ones((rows, F), dtype=torch.bfloat16, device="cuda")
    full = b.glu_backward(dy, ref.ACT_SILU, kept_codes=out.kept_codes, kept_scales=out.kept_scales)
    part = b.glu_backward(dy[-8:], ref.ACT_SILU, kept_codes=tail.kept_codes, kept_scales=tail.kept_scales)
    assert torch.equal(full.dgu[-8:], part.dgu)


@pytest.mark.parametrize("rows,F", [(3, 96), (700, 4096)])
def test_outputs_over_inputs(rows, F):
    """y over a dense gate, dgu over the halves, a over dy; overlaps of other kinds are refused."""
    import torch
    b = lib()
    rng = np.random.default_rng(rows)
    gu = _make(rng, (rows, 2 * F), _dtype("bf16"))[0]
    dy = _make(rng, (rows, F), _dtype("bf16"))[0]
    want = b.glu(gu[:, :F], gu[:, F:], ref.ACT_SILU, plain=True, keep=True)
    grad = b.glu_backward(dy, ref.ACT_SILU, gate=gu[:, :F], up=gu[:, F:], recompute=True, fmt=1)
    for kw in (dict(dgu=gu, gate=gu[:, F:], up=gu[:, :F]), dict(a=gu.view(2 * rows, F)[:rows], gate=gu[:, :F], up=gu[:, F:])):
        with pytest.raises(b.MxGemmError) as e:
            b.glu_backward(dy, ref.ACT_SILU, **kw)
        assert e.value.status == b.MXGEMM_ERR_ARG
    g, u = gu[:, :F].contiguous(), gu[:, F:].contiguous()
    got = b.glu(g, u, ref.ACT_SILU, plain=True, keep=True, y=g)
    assert got.y is g and torch.equal(g, want.y) and torch.equal(got.kept_codes, want.kept_codes)
    got = b.glu_backward(dy, ref.ACT_SILU, gate=gu[:, :F], up=gu[:, F:], recompute=True, fmt=1, dgu=gu, a=dy)
    assert got.dgu is gu and got.a is dy
    assert all(torch.equal(p, q) for p, q in zip(got, grad))


@pytest.mark.parametrize("act", [ref.ACT_SILU, ref.ACT_GELU])
def test_float32_keeps_its_precision(act):
    """FP32 operands: the exponential's argument is not rounded on the way (SiLU) and nothing is flushed.  exp is
    within two ulps, then an addition, a reciprocal within an ulp and a product: 8 roundings of q and of 1 - q.  GELU's
    argument has seven, which move q by |t| (1 - q) and 1 - q by |t| q as much.  Below 2^-126 q is off by a few 2^-149."""
    import torch
    b = lib()
    rng = np.random.default_rng(40 + act)
    F, floor = 2080, 2.0 ** -147
    g = rng.standard_normal((4, F)) * np.array([[1], [3], [30], [1]])
    g[0] = np.linspace(-104, 104, F)
    gu = np.concatenate([g, rng.standard_normal((4, F)) * 1e3], 1).astype(np.float32)
    dy = rng.standard_normal((4, F)).astype(np.float32)
    gd, dyd = torch.from_numpy(gu).cuda(), torch.from_numpy(dy).cuda()
    y = _np(b.glu(gd[:, :F], gd[:, F:], act, plain=True).y)
    back = b.glu_backward(dyd, act, gate=gd[:, :F], up=gd[:, F:], recompute=True)
    g, u, dy = gu[:, :F].astype(np.float64), gu[:, F:].astype(np.float64), dy.astype(np.float64)
    with np.errstate(over="ignore"):
        q, t, slope = ref._gate(g, act)
        rest = 1 / (1 + np.exp(t))
    arg = 0 if act == ref.ACT_SILU else 7 * np.abs(t)
    f, eq, er = g * q, (8 + arg * rest) * ref.U, (8 + arg * q) * ref.U
    err = (eq + 3 * ref.U) * np.abs(f * u) + floor * np.abs(g * u)
    ref.assert_near(y, f * u, err, False, "a")
    ref.assert_near(_np(back.a), f * u, err, False, "a again")
    part = np.abs(f) * rest * slope
    dg = dy * u * (q + f * rest * slope)
    edg = np.abs(dy * u) * (q * eq + part * (eq + er + 8 * ref.U) + floor * (1 + np.abs(g) * slope)) + 4 * ref.U * np.abs(dg)
    ref.assert_near(_np(back.dgu)[:, :F], dg, edg, False, "dgate")
    ref.assert_near(_np(back.dgu)[:, F:], dy * f, (eq + 3 * ref.U) * np.abs(dy * f) + floor * np.abs(dy * g), False, "dup")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt,tiled", [(1, True), (2, True), (1, False), (2, False)])
@pytest.mark.parametrize("rows,F", [(1501, 1664), (2501, 1088), (900, 4096)])
def test_many_rows(oracle_mod, dtype, fmt, tiled, rows, F):
    """Several chunks to every warp, both directions, the gradient from the checkpoint."""
    b = lib()
    rng = np.random.default_rng([rows, F])
    bf16 = dtype == "bf16"
    tiled = tiled and F % 128 == 0
    gu, gu64 = _make(rng, (rows, 2 * F), _dtype(dtype), 2.0)
    dy, dy64 = _make(rng, (rows, F), _dtype(dtype))
    out = b.glu(gu[:, :F], gu[:, F:], ref.ACT_SILU, fmt=fmt, tiled=tiled, plain=True, keep=True)
    a, err = ref.glu(gu64[:, :F], gu64[:, F:], ref.ACT_SILU)
    ref.assert_near(_np(out.y), a, err, bf16, "a")
    ref.assert_mx(out.codes.cpu().numpy(), _scales(out.scales, tiled, rows, F), a, err + ref.TINY_F32, fmt, "MX(a)")
    codes, scales = oracle_mod.quantize(1, gu.float().cpu().numpy(), oracle_mod.IN_F32)
    assert (out.kept_codes.cpu().numpy() == codes).all() and (out.kept_scales.cpu().numpy() == scales).all()
    sc = np.exp2(scales.astype(np.float64) - 127)
    kept64 = ref.decode_codes(codes, 1) * np.repeat(sc, 32, axis=1)
    for src, v64 in ((dict(kept_codes=out.kept_codes, kept_scales=out.kept_scales), kept64),
                     (dict(gate=gu[:, :F], up=gu[:, F:]), gu64)):
        back = b.glu_backward(dy, ref.ACT_SILU, fmt=fmt, tiled=tiled, recompute=True, **src)
        dg, edg, du, edu = ref.glu_backward(dy64, v64[:, :F], v64[:, F:], ref.ACT_SILU)
        ref.assert_near(_np(back.dgu)[:, :F], dg, edg, bf16, "dgate")
        ref.assert_near(_np(back.dgu)[:, F:], du, edu, bf16, "dup")
        a, ea = ref.glu(v64[:, :F], v64[:, F:], ref.ACT_SILU)
        ref.assert_near(_np(back.a), a, ea, bf16, "a again")
        both, e = np.concatenate([dg, du], 1), np.concatenate([edg, edu], 1) + ref.TINY_F32
        ref.assert_mx(back.codes.cpu().numpy(), _scales(back.scales, tiled, rows, 2 * F), both, e, fmt, "MX(dgu)")


def test_flags_and_numbers_that_are_none():
    """A flag without a truth value raises its own error; a format past 32 bits is no format."""
    import torch
    b = lib()
    x, w = torch.ones((4, 64), device="cuda"), torch.ones(64, device="cuda")
    both = torch.tensor([True, False])
    for call in (lambda: b.glu(x, x, ref.ACT_SILU, plain=both), lambda: b.glu(x, x, ref.ACT_SILU, fmt=1, tiled=both),
                 lambda: b.glu(x, x, ref.ACT_SILU, keep=both), lambda: b.rmsnorm(x, w, 1e-5, plain=both),
                 lambda: b.glu_backward(x, ref.ACT_SILU, gate=x, up=x, recompute=both)):
        with pytest.raises(RuntimeError, match="Boolean value"):
            call()
    for call in (lambda: b.glu(x, x, ref.ACT_SILU, fmt=(1 << 32) + 1), lambda: b.glu(x, x, (1 << 32) + 1, plain=True),
                 lambda: b.rmsnorm(x, w, 1e-5, fmt=(1 << 32) + 1),
                 lambda: b.moe_dispatch(x, torch.arange(4, dtype=torch.int32, device="cuda"), (1 << 32) + 3)):
        with pytest.raises(b.MxGemmError) as e:
            call()
        assert e.value.status == b.MXGEMM_ERR_ARG
