"""RMS norm with residual and MX output, and its gradient, on the GPU against the
64-bit definition (row_ops_ref.py), through the binding."""
import numpy as np
import pytest

import row_ops_ref as ref
from gpu_util import lib

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    lib()


def _make(rng, shape, dtype, scale=1.0):
    """Device tensor and the 64-bit values it holds."""
    import torch
    t = torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).cuda().to(dtype)
    return t, t.double().cpu().numpy()


def _dtype(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float32


def _np(t):
    return t.double().cpu().numpy()


def _check_forward(b, out, want, fmt, tiled, bf16, has_residual, plain):
    h, rstd, y = want
    rr, ry = ref.rmsnorm_rel()
    rows, K = y.shape
    if has_residual:
        ref.assert_near(_np(out.h), h, ref.U * np.abs(h), bf16, "h")
    ref.assert_near(_np(out.rstd), rstd, rr * rstd, False, "rstd")
    err = ry * np.abs(y) + ref.TINY_F32
    if plain:
        ref.assert_near(_np(out.y), y, err, bf16, "y")
    if fmt:
        scales = out.scales.cpu().numpy()
        ref.assert_mx(out.codes.cpu().numpy(), ref.untile(scales, rows, K) if tiled else scales, y, err, fmt, "MX(y)")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt,tiled", [(0, False), (1, False), (1, True), (2, False), (2, True)])
@pytest.mark.parametrize("rows,K,residual,plain", [
    (1, 128, True, False), (3, 384, False, True), (130, 512, True, True), (7, 640, True, False),
    (5, 4096, True, True), (2, 8192, False, False), (3, 8320, True, False), (2, 16384, True, False),
    (2, 16512, False, True), (1, 32768, True, False),
])
def test_forward(dtype, fmt, tiled, rows, K, residual, plain):
    b = lib()
    rng = np.random.default_rng([rows, K, fmt])
    dt = _dtype(dtype)
    x, x64 = _make(rng, (rows, K), dt, 3.0)
    r, r64 = _make(rng, (rows, K), dt) if residual else (None, None)
    w, w64 = _make(rng, (K,), dt)
    out = b.rmsnorm(x, w, EPS, residual=r, fmt=fmt, tiled=tiled, plain=plain or fmt == 0)
    _check_forward(b, out, ref.rmsnorm(x64, w64, EPS, r64), fmt, tiled, dtype == "bf16", residual, plain or fmt == 0)


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("K", [32, 96, 160, 1056, 5152])
def test_forward_without_whole_tiles(fmt, K):
    """K a multiple of 32 only: row-major scales that are not whole words."""
    b = lib()
    rng = np.random.default_rng(K)
    x, x64 = _make(rng, (37, K), _dtype("bf16"))
    w, w64 = _make(rng, (K,), _dtype("f32"))     # weight of another type
    out = b.rmsnorm(x, w, EPS, fmt=fmt, plain=True)
    _check_forward(b, out, ref.rmsnorm(x64, w64, EPS), fmt, False, True, False, True)


def test_forward_extreme_rows():
    """A row of zeros, one of tiny and one of huge values, and rows with a NaN or an infinity."""
    import torch
    b = lib()
    rng = np.random.default_rng(1)
    x = rng.standard_normal((7, 256)).astype(np.float32)
    x[0] = 0
    x[1] *= 1e-18
    x[2] *= 1e15
    x[3, 17] = np.nan
    x[4, 200] = np.inf
    x[5] = -0.0
    w = rng.standard_normal(256).astype(np.float32)
    xd, wd = torch.from_numpy(x).cuda(), torch.from_numpy(w).cuda()
    out = b.rmsnorm(xd, wd, EPS, fmt=1, plain=True)
    with np.errstate(invalid="ignore"):
        _, rstd, y = ref.rmsnorm(x.astype(np.float64), w.astype(np.float64), EPS)
    fin = [0, 1, 2, 5, 6]
    rr, ry = ref.rmsnorm_rel()
    ref.assert_near(_np(out.rstd)[fin], rstd[fin], rr * rstd[fin], False, "rstd")
    err = ry * np.abs(y[fin]) + ref.TINY_F32
    ref.assert_near(_np(out.y)[fin], y[fin], err, False, "y")
    ref.assert_mx(out.codes.cpu().numpy()[fin], out.scales.cpu().numpy()[fin], y[fin], err, 1, "MX")
    got = _np(out.y)
    assert np.isnan(got[3]).all()                                  # the sum is NaN
    assert np.isnan(got[4, 200]) and (np.delete(got[4], 200) == 0).all()  # 1/inf = 0, inf * 0 = NaN
    sc = out.scales.cpu().numpy()
    assert (sc[3] == 255).all() and sc[4, 200 // 32] == 255 and (np.delete(sc[4], 200 // 32) == 127).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_inputs_in_place_h_and_guards(dtype):
    """Rows of wider matrices; h written over the residual; nothing written around the outputs."""
    import torch
    b = lib()
    rng = np.random.default_rng(8)
    rows, K, dt = 9, 672, _dtype(dtype)
    wide, wide64 = _make(rng, (rows, K + 64), dt)
    x, x64 = wide[:, 32:32 + K], wide64[:, 32:32 + K]
    r, r64 = _make(rng, (rows, K), dt)
    w, w64 = _make(rng, (K,), dt)
    pad = 64
    buf = torch.full((rows * K + 2 * pad,), 77.0, dtype=dt, device="cuda")
    codes = torch.full((rows * K + 2 * pad,), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows * K // 32 + 2 * pad,), 0xA5, dtype=torch.uint8, device="cuda")
    out = b.rmsnorm(x, w, EPS, residual=r, fmt=1, h=r, y=buf[pad:-pad].view(rows, K),
                    codes=codes[pad:-pad].view(rows, K), scales=scales[pad:-pad].view(rows, K // 32))
    assert out.h is r
    _check_forward(b, out, ref.rmsnorm(x64, w64, EPS, r64), 1, False, dtype == "bf16", True, True)
    for t, v in ((buf, 77.0), (codes, 0xA5), (scales, 0xA5)):
        assert (t[:pad] == v).all() and (t[-pad:] == v).all()
    assert (_np(wide) == wide64).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,K,dh", [
    (1, 32, True), (2, 160, False), (33, 512, True), (400, 1056, True), (700, 128, False), (19, 4096, True),
    (40, 8192, False), (3, 8224, True), (5, 16384, True), (2, 16416, False), (3, 32768, True),
    (1024, 96, True), (1025, 32, True), (1300, 160, False), (2000, 1056, True), (1100, 2080, True), (1030, 4096, False),
    (1025, 8192, True),
])
def test_backward(dtype, rows, K, dh):
    import torch
    b = lib()
    rng = np.random.default_rng([rows, K, 5])
    dt, bf16 = _dtype(dtype), dtype == "bf16"
    h, h64 = _make(rng, (rows, K), dt, 2.0)
    dy, dy64 = _make(rng, (rows, K), dt)
    g, g64 = _make(rng, (rows, K), dt) if dh else (None, None)
    w, w64 = _make(rng, (K,), dt)
    rstd = torch.from_numpy((1 / np.sqrt((h64 * h64).mean(1) + EPS)).astype(np.float32)).cuda()
    dx, dw = b.rmsnorm_backward(dy, h, rstd, w, dh=g)
    want, err, wdw, size = ref.rmsnorm_backward(dy64, h64, _np(rstd), w64, g64)
    ref.assert_near(_np(dx), want, err, bf16, "dx")
    ref.assert_near(_np(dw), wdw, (rows + 64) * ref.U * size, False, "dw")
    again = b.rmsnorm_backward(dy, h, rstd, w, dh=g)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw), "two runs differ"


def test_backward_in_place_strided_and_mixed_weight():
    """dx over dh, rows of wider matrices, a weight of another type, workspace from the caller."""
    import torch
    b = lib()
    rng = np.random.default_rng(21)
    rows, K = 1200, 288
    hw, hw64 = _make(rng, (rows, 2 * K), _dtype("bf16"))
    dyw, dyw64 = _make(rng, (rows, K + 96), _dtype("bf16"))
    dh, dh64 = _make(rng, (rows, K), _dtype("bf16"))
    w, w64 = _make(rng, (K,), _dtype("f32"))
    h64, dy64 = hw64[:, K:], dyw64[:, :K]
    rstd = torch.from_numpy((1 / np.sqrt((h64 * h64).mean(1) + EPS)).astype(np.float32)).cuda()
    need = b.mxgemm_rmsnorm_backward_workspace_bytes(rows, K)
    ws = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    dx, dw = b.rmsnorm_backward(dyw[:, :K], hw[:, K:], rstd, w, dh=dh, dx=dh, workspace=ws)
    want, err, wdw, size = ref.rmsnorm_backward(dy64, h64, _np(rstd), w64, dh64)
    ref.assert_near(_np(dx), want, err, True, "dx")
    ref.assert_near(_np(dw), wdw, (rows + 64) * ref.U * size, False, "dw")
    assert (ws[need:] == 0xA5).all()
    with pytest.raises(b.MxGemmError) as e:
        b.rmsnorm_backward(dyw[:, :K], hw[:, K:], rstd, w, workspace=ws[: need - 32])
    assert e.value.status == b.MXGEMM_ERR_WORKSPACE


def test_gradient_against_differences():
    """The kernel's FP32 gradient along random directions against central differences of the 64-bit forward."""
    import torch
    b = lib()
    rng = np.random.default_rng(4)
    rows, K = 6, 256
    x, x64 = _make(rng, (rows, K), _dtype("f32"))
    w, w64 = _make(rng, (K,), _dtype("f32"))
    dy, dy64 = _make(rng, (rows, K), _dtype("f32"))
    out = b.rmsnorm(x, w, EPS, plain=True)
    dx, dw = b.rmsnorm_backward(dy, x, out.rstd, w)
    f = lambda x_, w_: (ref.rmsnorm(x_, w_, EPS)[2] * dy64).sum()  # noqa: E731
    v, vw, e = rng.standard_normal((rows, K)), rng.standard_normal(K), 1e-5
    # FP32 gradients: the bound of each term summed over the direction, with rstd's own error
    lim = (ref.rmsnorm_backward(dy64, x64, _np(out.rstd), w64)[1] * np.abs(v)).sum() * 4 + 1e-8 * rows * K
    assert abs((f(x64 + e * v, w64) - f(x64 - e * v, w64)) / (2 * e) - (_np(dx) * v).sum()) < lim
    size = ref.rmsnorm_backward(dy64, x64, _np(out.rstd), w64)[3]
    lim = ((rows + 64 + 40) * ref.U * size * np.abs(vw)).sum() + 1e-8 * rows * K
    assert abs((f(x64, w64 + e * vw) - f(x64, w64 - e * vw)) / (2 * e) - (_np(dw) * vw).sum()) < lim


def test_side_stream_and_graph_replay():
    """On a stream of its own, ordered only by an event; and captured in a graph and replayed on new inputs."""
    import torch
    b = lib()
    rng = np.random.default_rng(6)
    x, x64 = _make(rng, (64, 1024), _dtype("bf16"))
    w, w64 = _make(rng, (1024,), _dtype("bf16"))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = b.rmsnorm(x, w, EPS, fmt=1, plain=True, stream=s)
    s.synchronize()
    _check_forward(b, out, ref.rmsnorm(x64, w64, EPS), 1, False, True, False, True)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.rmsnorm(x, w, EPS, fmt=1, y=out.y, codes=out.codes, scales=out.scales, rstd=out.rstd)
    x2, x264 = _make(rng, (64, 1024), _dtype("bf16"))
    x.copy_(x2)
    g.replay()
    torch.cuda.synchronize()
    _check_forward(b, out, ref.rmsnorm(x264, w64, EPS), 1, False, True, False, True)


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last rows of a call equal those rows on their own."""
    import torch
    b = lib()
    rows, K = (1 << 31) // 8192 + 37, 8192
    x = torch.empty((rows, K), dtype=torch.bfloat16, device="cuda")
    x[:-64].fill_(1.0)
    x[-64:] = torch.randn((64, K), device="cuda").to(torch.bfloat16)
    w = torch.randn((K,), device="cuda")
    out = b.rmsnorm(x, w, EPS, fmt=1, plain=True)
    tail = b.rmsnorm(x[-64:], w, EPS, fmt=1, plain=True)
    assert torch.equal(out.y[-64:], tail.y) and torch.equal(out.codes[-64:], tail.codes)
    assert torch.equal(out.scales[-64:], tail.scales) and torch.equal(out.rstd[-64:], tail.rstd)
    dx, _ = b.rmsnorm_backward(out.y, x, out.rstd, w)
    dt, _ = b.rmsnorm_backward(tail.y, x[-64:], tail.rstd, w)
    assert torch.equal(dx[-64:], dt)


@pytest.mark.parametrize("rows", [5, 1100])
def test_outputs_over_inputs(rows):
    """y over x and h over the residual give what apart outputs give; dx over dy is refused."""
    import torch
    b = lib()
    rng = np.random.default_rng(rows)
    x, r, dy = (_make(rng, (rows, 512), _dtype("bf16"))[0] for _ in range(3))
    w = _make(rng, (512,), _dtype("bf16"))[0]
    want = b.rmsnorm(x, w, EPS, residual=r, plain=True, fmt=1)
    grads = b.rmsnorm_backward(dy, want.h, want.rstd, w, dh=x.clone())
    for kw in (dict(dx=dy), dict(dx=want.h)):
        with pytest.raises(b.MxGemmError) as e:
            b.rmsnorm_backward(dy, want.h, want.rstd, w, dh=x.clone(), **kw)
        assert e.value.status == b.MXGEMM_ERR_ARG
    xc = x.clone()
    over = b.rmsnorm_backward(dy, want.h, want.rstd, w, dh=xc, dx=xc)
    assert torch.equal(over[0], grads[0]) and torch.equal(over[1], grads[1])
    got = b.rmsnorm(x, w, EPS, residual=r, plain=True, fmt=1, h=r, y=x)
    assert got.y is x and got.h is r
    assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("rows,K", [(4096, 96), (4099, 512), (4098, 544), (4097, 1024)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("residual", [False, True])
def test_many_narrow_rows(rows, K, dtype, residual):
    """Rows that share a block: the same results as in calls of few rows, nothing past the last one."""
    import torch
    b = lib()
    rng = np.random.default_rng([rows, K])
    x, r = (_make(rng, (rows, K), _dtype(dtype))[0] for _ in range(2))
    w = _make(rng, (K,), _dtype(dtype))[0]
    tiled, pad = K % 128 == 0, 64
    buf = torch.full((rows * K + 2 * pad,), 3.0, dtype=x.dtype, device="cuda")
    y = buf[pad:-pad].view(rows, K)
    got = b.rmsnorm(x, w, EPS, residual=r if residual else None, plain=True, fmt=1, tiled=tiled, y=y)
    for at in range(0, rows, 2048):
        few = slice(at, min(at + 2048, rows))
        want = b.rmsnorm(x[few], w, EPS, residual=r[few] if residual else None, plain=True, fmt=1)
        for name in ("h", "y", "codes", "rstd"):
            if getattr(got, name) is not None:
                assert torch.equal(getattr(got, name)[few], getattr(want, name)), name
        scales = got.scales.cpu().numpy()
        scales = ref.untile(scales, rows, K) if tiled else scales
        assert np.array_equal(scales[few], want.scales.cpu().numpy())
    assert (buf[:pad] == 3.0).all() and (buf[-pad:] == 3.0).all()
    if tiled:  # rows up to the tile's end hold 1.0
        padded = (rows + 127) // 128 * 128
        assert (ref.untile(got.scales.cpu().numpy(), padded, K)[rows:] == 127).all()


@pytest.mark.parametrize("rows,K", [(1025, 96), (1301, 512), (2437, 544), (3000, 1024)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dh", [False, True])
def test_backward_many_narrow_rows(rows, K, dtype, dh):
    """Rows that share a block: dx as in calls of few rows, dw within the sum's bound, the same from run to run."""
    import torch
    b = lib()
    rng = np.random.default_rng([rows, K])
    dt, bf16 = _dtype(dtype), dtype == "bf16"
    h, h64 = _make(rng, (rows, K), dt)
    dy, dy64 = _make(rng, (rows, K), dt)
    g, g64 = _make(rng, (rows, K), dt) if dh else (None, None)
    w, w64 = _make(rng, (K,), dt)
    rstd = torch.from_numpy((1 / np.sqrt((h64 * h64).mean(1) + EPS)).astype(np.float32)).cuda()
    dx, dw = b.rmsnorm_backward(dy, h, rstd, w, dh=g)
    want, err, wdw, size = ref.rmsnorm_backward(dy64, h64, _np(rstd), w64, g64)
    ref.assert_near(_np(dx), want, err, bf16, "dx")
    ref.assert_near(_np(dw), wdw, (rows + 64) * ref.U * size, False, "dw")
    for at in range(0, rows, 1000):
        few = slice(at, min(at + 1000, rows))
        part = b.rmsnorm_backward(dy[few], h[few], rstd[few], w, dh=g[few] if dh else None)
        assert torch.equal(part[0], dx[few])
    again = b.rmsnorm_backward(dy, h, rstd, w, dh=g)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw), "two runs differ"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,K,dh", [(12, 512, False), (12, 96, True), (1100, 512, True), (1100, 2080, False),
                                       (12, 8224, True), (12, 16384, False)])
def test_backward_of_extreme_rows(dtype, rows, K, dh):
    """Rows whose rstd is far from 1, where its powers leave FP32 and dx does not; a row of zeros with a tiny eps."""
    import torch
    b = lib()
    rng = np.random.default_rng([rows, K, 7])
    dt = _dtype(dtype)
    scale = np.ones((rows, 1), np.float32)
    scale[:12, 0] = [1, 1e4, 1e12, 1e13, 1e15, 1e17, 1e-4, 1e-10, 1e-13, 1e-15, 1e-17, 0]
    h = torch.from_numpy((rng.standard_normal((rows, K)) * scale).astype(np.float32)).cuda().to(dt)
    h64 = _np(h)
    dy, dy64 = _make(rng, (rows, K), dt)
    w, w64 = _make(rng, (K,), dt)
    g = g64 = None
    rstd = torch.from_numpy((1 / np.sqrt((h64 * h64).mean(1) + (scale[:, 0] == 0) * 1e-30)).astype(np.float32)).cuda()
    if dh:  # of dx's own size, so that it hides nothing
        g = (torch.from_numpy(rng.standard_normal((rows, K)).astype(np.float32)).cuda() * rstd[:, None]).to(dt)
        g64 = _np(g)
    dx, dw = b.rmsnorm_backward(dy, h, rstd, w, dh=g)
    want, err, wdw, size = ref.rmsnorm_backward(dy64, h64, _np(rstd), w64, g64)
    ref.assert_near(_np(dx), want, err, dtype == "bf16", "dx")
    ref.assert_near(_np(dw), wdw, (rows + 64) * ref.U * size, False, "dw")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,K,dh", [
    (8001, 96, True), (8001, 96, False), (7999, 512, True), (7999, 512, False), (9001, 544, True), (4000, 992, False),
    (5000, 2080, True), (3001, 4096, True), (1500, 8192, False), (700, 8224, True), (311, 16384, False), (320, 32768, True),
])
def test_backward_of_many_rows(dtype, rows, K, dh):
    """Several rows to every block: the ring past its depth, rows side by side, the last rows of some blocks missing."""
    import torch
    b = lib()
    rng = np.random.default_rng([rows, K, 11])
    dt = _dtype(dtype)
    h, h64 = _make(rng, (rows, K), dt, 2.0)
    dy, dy64 = _make(rng, (rows, K), dt)
    g, g64 = _make(rng, (rows, K), dt) if dh else (None, None)
    w, w64 = _make(rng, (K,), dt)
    rstd = torch.from_numpy((1 / np.sqrt((h64 * h64).mean(1) + EPS)).astype(np.float32)).cuda()
    dx, dw = b.rmsnorm_backward(dy, h, rstd, w, dh=g)
    want, err, wdw, size = ref.rmsnorm_backward(dy64, h64, _np(rstd), w64, g64)
    ref.assert_near(_np(dx), want, err, dtype == "bf16", "dx")
    ref.assert_near(_np(dw), wdw, (rows + 64) * ref.U * size, False, "dw")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,K,residual", [(5001, 96, True), (4500, 544, False), (4100, 1024, True), (3000, 2016, False)])
def test_forward_of_many_rows(dtype, rows, K, residual):
    b = lib()
    rng = np.random.default_rng([rows, K])
    dt = _dtype(dtype)
    x, x64 = _make(rng, (rows, K), dt, 3.0)
    r, r64 = _make(rng, (rows, K), dt) if residual else (None, None)
    w, w64 = _make(rng, (K,), dt)
    want = ref.rmsnorm(x64, w64, EPS, r64)
    for fmt in (1, 2):
        out = b.rmsnorm(x, w, EPS, residual=r, fmt=fmt, tiled=K % 128 == 0, plain=True)
        _check_forward(b, out, want, fmt, K % 128 == 0, dtype == "bf16", residual, True)
