"""Norm and rotation of heads and their gradients on the GPU against the 64-bit
definition (model_ops_ref.py), through the binding."""
import numpy as np
import pytest

import model_ops_ref as ref
from gpu_util import lib
from row_ops_ref import assert_near

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    lib()


def _dt(name):
    import torch
    return dict(bf16=torch.bfloat16, f32=torch.float32)[name]


def _make(rng, shape, dtype, scale=1.0):
    import torch
    t = torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).cuda().to(_dt(dtype))
    return t, t.double().cpu().numpy()


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _rope(rows, rotary):
    """cos | sin of every position, formed in 64 bits, as a device tensor and the values it holds."""
    import torch
    a = np.arange(rows)[:, None] * 10000.0 ** (-np.arange(rotary // 2) / (rotary // 2))
    t = torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)).cuda()
    return t, _np(t)


def _case(tokens, Q, H, D, rotary, dtype, wt, norm=True, seed=0, wide=True, rows=500):
    import torch
    rng = np.random.default_rng([tokens, H, D, rotary, seed])
    x, x64 = _make(rng, (tokens, H, D), dtype, 1.5)
    qw, qw64 = _make(rng, (D,), wt) if norm and Q else (None, None)
    kw, kw64 = _make(rng, (D,), wt) if norm and Q < H else (None, None)
    rope, rope64 = _rope(rows, rotary) if rotary else (None, None)
    pos = rng.integers(0, rows, tokens)
    pos[rng.random(tokens) < 0.1] = -1
    pos[rng.random(tokens) < 0.05] = rows
    pos_dev = torch.from_numpy(pos.astype(np.int64 if wide else np.int32)).cuda() if rotary else None
    return dict(x=x, x64=x64, qw=qw, kw=kw, qw64=qw64, kw64=kw64, rope=rope, rope64=rope64, pos=pos, pos_dev=pos_dev, Q=Q,
                dtype=dtype, rng=rng)


def _forward(c, interleaved, **more):
    b = lib()
    got = b.qk_norm_rope(more.pop("x", c["x"]), c["Q"], c["qw"], c["kw"], EPS, rope=c["rope"], positions=c["pos_dev"],
                         interleaved=interleaved, **more)
    y, err, rstd, rel = ref.qk_norm_rope(c["x64"], c["Q"], c["qw64"], c["kw64"], EPS, c["rope64"], c["pos"], interleaved)
    assert_near(_np(got.y), y, err, c["dtype"] == "bf16", "y")
    if rstd is None:
        assert got.rstd is None
    else:
        assert_near(_np(got.rstd), rstd, rel * rstd, False, "rstd")
    return got


def _backward(c, interleaved, rstd, **more):
    b = lib()
    shape = c["x"].shape
    dy, dy64 = _make(c["rng"], shape, c["dtype"])
    norm = rstd is not None
    if "dy" in more:
        more["dy"].copy_(dy)
        dy = more.pop("dy")
    if more.pop("over", False):
        more["dx"] = dy
    got = b.qk_norm_rope_backward(dy, more.pop("x", c["x"]) if norm else None, rstd, c["Q"], c["qw"], c["kw"], rope=c["rope"],
                                  positions=c["pos_dev"], interleaved=interleaved, **more)
    dx, edx, dq, edq, dk, edk = ref.qk_norm_rope_backward(dy64, c["x64"] if norm else None, _np(rstd), c["Q"], c["qw64"],
                                                          c["kw64"], c["rope64"], c["pos"], interleaved)
    assert_near(_np(got[0]), dx, edx, c["dtype"] == "bf16", "dx")
    for g, w, e, what in ((got[1], dq, edq, "dq"), (got[2], dk, edk, "dk")):
        if g is not None:
            assert_near(_np(g), w, e, False, what)
    return got


SIZES = [  # tokens, query heads, heads, D, rotary
    (1, 1, 1, 16, 16), (1, 4, 6, 128, 128), (3, 2, 3, 32, 16), (7, 0, 2, 64, 64), (5, 5, 5, 48, 32), (33, 3, 4, 80, 80),
    (20, 8, 10, 96, 48), (64, 12, 16, 128, 64), (9, 2, 3, 192, 192), (6, 3, 5, 256, 128), (4, 1, 2, 512, 512),
    (2, 1, 2, 496, 240), (130, 7, 9, 64, 32), (1000, 5, 7, 128, 128), (37, 40, 48, 128, 0), (300, 33, 44, 16, 16),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,wt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("tokens,Q,H,D,rotary", SIZES)
def test_both_directions(tokens, Q, H, D, rotary, dtype, wt, interleaved):
    c = _case(tokens, Q, H, D, rotary, dtype, wt, wide=H % 2 == 0)
    got = _forward(c, interleaved)
    dead = (c["pos"] < 0) | (c["pos"] >= 500)
    if rotary:
        assert (_np(got.y)[dead] == 0).all() and (_np(got.rstd)[dead] == 0).all()
    _backward(c, interleaved, got.rstd)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,Q,H,D,rotary", [(1, 1, 1, 16, 16), (50, 4, 6, 128, 128), (9, 3, 3, 80, 16), (5, 0, 7, 512, 256)])
def test_rotation_alone(tokens, Q, H, D, rotary, dtype, interleaved):
    c = _case(tokens, Q, H, D, rotary, dtype, "f32", norm=False)
    c["x"][0, 0, -1] = float("inf")     # a value that is not turned is left as it is
    c["x64"][0, 0, -1] = np.inf
    if rotary < D and 0 <= c["pos"][0] < 500:
        _forward(c, interleaved)
    c["x"][0, 0, -1] = 1.0
    c["x64"][0, 0, -1] = 1.0
    _forward(c, interleaved)
    _backward(c, interleaved, None)


def test_rotation_undoes_itself_and_matches_the_angle():
    """One pair by a quarter turn; the gradient's rotation is the inverse."""
    import torch
    b = lib()
    rope = torch.zeros((2, 16), device="cuda")
    rope[0, :8] = 1.0                   # position 0: as it is
    rope[1, 8:] = 1.0                   # position 1: a quarter turn
    x = torch.arange(2 * 16, dtype=torch.float32, device="cuda").view(2, 1, 16)
    pos = torch.tensor([0, 1], device="cuda")
    y = b.qk_norm_rope(x, 1, rope=rope, positions=pos).y
    assert (y[0] == x[0]).all() and (y[1, 0, :8] == -x[1, 0, 8:]).all() and (y[1, 0, 8:] == x[1, 0, :8]).all()
    y = b.qk_norm_rope(x, 1, rope=rope, positions=pos, interleaved=True).y
    assert (y[1, 0, 0::2] == -x[1, 0, 1::2]).all() and (y[1, 0, 1::2] == x[1, 0, 0::2]).all()
    assert torch.equal(b.qk_norm_rope_backward(y, None, None, 1, rope=rope, positions=pos, interleaved=True)[0], x)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["inside", "heads first", "in place", "in place inside"])
def test_layouts(dtype, layout):
    """Heads inside a q|k|v product's rows, [heads, tokens, D], in place; nothing else is written."""
    import torch
    T, Q, H, D = 21, 4, 6, 64
    c = _case(T, Q, H, D, 32, dtype, "f32", seed=3)
    if layout == "heads first":
        x = c["x"].transpose(0, 1).contiguous().transpose(0, 1)
        y = torch.empty((H, T, D), dtype=_dt(dtype), device="cuda").transpose(0, 1)
        got = _forward(c, False, x=x, y=y)
        assert got.y is y
        dy = torch.empty((H, T, D), dtype=_dt(dtype), device="cuda").transpose(0, 1)
        _backward(c, False, got.rstd, x=x, dy=dy, over=True)
        return
    if layout == "in place":
        x = c["x"].clone()
        got = _forward(c, True, x=x, y=x)
        _backward(c, True, got.rstd, over=True)
        x = c["x"].clone()
        _backward(c, True, got.rstd, x=x, dx=x)
        return
    rows = torch.full((T, H + 3, D), 7.0, dtype=_dt(dtype), device="cuda")
    x = rows[:, 1:1 + H]
    x.copy_(c["x"])
    got = _forward(c, False, x=x, y=x if layout == "in place inside" else None)
    if layout == "inside":
        assert torch.equal(x, c["x"])
        drows = torch.full((T, H + 2, D), 5.0, dtype=_dt(dtype), device="cuda")
        _backward(c, False, got.rstd, x=x, dx=drows[:, 2:])
        assert (drows[:, :2] == 5).all()
    assert (rows[:, 0] == 7).all() and (rows[:, 1 + H:] == 7).all()


def test_padding_may_hold_anything():
    import torch
    c = _case(40, 2, 3, 64, 64, "f32", "f32", seed=5)
    dead = torch.from_numpy((c["pos"] < 0) | (c["pos"] >= 500)).cuda()
    assert dead.any()
    c["x"][dead] = float("nan")
    c["x64"][dead.cpu().numpy()] = 0
    got = _forward(c, False)
    got.rstd[dead] = float("nan")
    b, dy = lib(), torch.ones_like(c["x"])
    dy[dead] = float("inf")
    dx, dq, dk = b.qk_norm_rope_backward(dy, c["x"], got.rstd, 2, c["qw"], c["kw"], rope=c["rope"], positions=c["pos_dev"])
    assert (dx[dead] == 0).all() and torch.isfinite(dx).all() and torch.isfinite(dq).all() and torch.isfinite(dk).all()


def test_rows_of_extreme_scale():
    c = _case(6, 1, 2, 128, 128, "f32", "f32", seed=7)
    for i, s in enumerate((0.0, 1e-12, 1e13, 1e-4, 1e17)):
        c["x"][i] *= s
    c["x64"] = _np(c["x"])
    got = _forward(c, False)
    _backward(c, False, got.rstd)


def test_stream_graphs_and_many_tokens():
    """More tokens than a pass of the grid, a side stream, two captured gradients replayed in turn."""
    import torch
    b = lib()
    c = _case(9001, 2, 3, 32, 32, "bf16", "bf16", seed=9, rows=500)
    got = _forward(c, False)
    _backward(c, False, got.rstd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = b.qk_norm_rope(c["x"], 2, c["qw"], c["kw"], EPS, rope=c["rope"], positions=c["pos_dev"], stream=side).y
    side.synchronize()
    assert torch.equal(y, got.y)
    args = (c["x"], got.rstd, 2, c["qw"], c["kw"])
    graphs = []
    for s in (1.0, -2.0):
        dy = torch.full_like(c["x"], s)
        want = b.qk_norm_rope_backward(dy, *args, rope=c["rope"], positions=c["pos_dev"])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = b.qk_norm_rope_backward(dy, *args, rope=c["rope"], positions=c["pos_dev"])
        graphs.append((g, out, want, dy))                  # the gradient that the graph reads stays alive
    for g, *_ in graphs:
        g.replay()
    for _, out, want, _ in graphs:
        assert all(torch.equal(o, w) for o, w in zip(out, want))


def test_offsets_past_32_bits():
    import torch
    b = lib()
    T = 3
    big = torch.empty((T, (1 << 30) + 64), dtype=torch.bfloat16, device="cuda")   # tokens 2 GB apart
    x = big[:, :512].view(T, 4, 128)
    x.normal_()
    w = torch.ones(128, device="cuda")
    got = b.qk_norm_rope(x, 3, w, w, EPS)
    assert torch.equal(got.y, b.qk_norm_rope(x.contiguous(), 3, w, w, EPS).y)


def test_refusals():
    import torch
    b = lib()
    x = torch.ones((4, 3, 64), device="cuda")
    w, rope, pos = torch.ones(64, device="cuda"), torch.ones((9, 32), device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    for bad in (dict(q_weight=w[:32]), dict(rope=rope, positions=pos[:3]), dict(rope=rope.double(), positions=pos),
                dict(k_weight=w.bfloat16()), dict(y=torch.ones((4, 3, 32), device="cuda"))):
        with pytest.raises(ValueError):
            b.qk_norm_rope(x, 2, **{**dict(q_weight=w, k_weight=w), **bad})
    for bad in (dict(rope=rope), dict(positions=pos), dict(k_weight=None), dict(eps=-1.0), dict(q_heads=4),
                dict(rope=torch.ones((9, 80), device="cuda"), positions=pos), dict(rope=rope[:, :8].contiguous(), positions=pos)):
        args = {**dict(q_heads=2, q_weight=w, k_weight=w, eps=EPS), **bad}
        with pytest.raises(b.MxGemmError):
            b.qk_norm_rope(x, **args)
    with pytest.raises(b.MxGemmError):
        b.qk_norm_rope(x, 2)                               # neither weights nor angles
    with pytest.raises(b.MxGemmError):
        b.qk_norm_rope_backward(x, None, None, 2, w, w)
