"""The norm of many gradients and their clipping on the GPU against the 64-bit
definition (model_ops_ref.py), through the binding."""
import numpy as np
import pytest

import model_ops_ref as ref
from gpu_util import lib
from row_ops_ref import TINY_F32, assert_near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    lib()


def _dt(name):
    import torch
    return dict(bf16=torch.bfloat16, f32=torch.float32)[name]


def _grads(rng, shapes, dtypes, scale=1.0):
    import torch
    t = [torch.from_numpy(np.asarray(rng.standard_normal(s) * scale, np.float32)).cuda().to(_dt(d)) for s, d in zip(shapes, dtypes)]
    return t, [x.double().cpu().numpy() for x in t]


def _check(grads, g64, max_norm, out_dtypes=None, out=None):
    import torch
    b = lib()
    norm, factor, rel = ref.clip(g64, max_norm)
    only = b.grad_norm(grads)
    assert_near(only.cpu().numpy(), np.array([norm]), np.array([ref.NORM_REL * norm]), False, "norm")
    if out is None and out_dtypes is not None:
        out = [torch.empty_like(g, dtype=_dt(d)) for g, d in zip(grads, out_dtypes)]
    got, res = b.clip_grads(grads, max_norm, out=out)
    assert torch.equal(got, only) and res is (grads if out is None else out)
    for i, (r, g) in enumerate(zip(res, g64)):
        assert_near(r.double().cpu().numpy(), g * factor, rel * np.abs(g * factor) + TINY_F32, r.dtype == torch.bfloat16,
                    f"tensor {i}")
    return res


SHAPES = [[(1,)], [(7,)], [(8,)], [(4095,)], [(4096,)], [(4097,)], [(3, 5), (1,), (0,), (2, 2, 2)], [(0,)], [(0,), (9,), (0,)],
          [(100, 333), (4096,), (8192, 3), (1,)], [(1_000_003,)], [(17,)] * 40, [(257,)] * 300, [(33,)] * 1000, [(5,)] * 2000]


@pytest.mark.parametrize("form", ["in place", "f32", "bf16"])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_lists(i, form):
    """One tensor to two thousand (a table a launch takes up to 32, 256 or 896), mixed types, clipped and not."""
    rng = np.random.default_rng(i)
    shapes = SHAPES[i]
    dtypes = [["f32", "bf16"][(i + j) % 2] for j in range(len(shapes))]
    for max_norm in (0.1, 1e6):
        grads, g64 = _grads(rng, shapes, dtypes)
        _check(grads, g64, max_norm, None if form == "in place" else [form] * len(shapes))


@pytest.mark.parametrize("src", ["f32", "bf16"])
@pytest.mark.parametrize("dst", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 9, 1000, 30_000, 5_000_000])
def test_types_and_alignment(n, src, dst):
    """Tensors that start on any boundary of their type, and outputs that do."""
    import torch
    rng = np.random.default_rng(n)
    for at, to in ((0, 0), (1, 0), (0, 3), (5, 2)):
        (base,), (b64,) = _grads(rng, [(n + 16,)], [src])
        obase = torch.full((n + 16,), 7.0, dtype=_dt(dst), device="cuda")
        _check([base[at:at + n]], [b64[at:at + n]], 0.5, out=[obase[to:to + n]])
        assert (obase[:to] == 7).all() and (obase[to + n:] == 7).all()
        assert np.array_equal(base.double().cpu().numpy(), b64)


def test_empty_list_and_layouts():
    import torch
    b, rng = lib(), np.random.default_rng(1)
    assert b.grad_norm([]).tolist() == [0.0]
    norm, out = b.clip_grads([], 1.0)
    assert norm.tolist() == [0.0] and out == []
    (g,), (g64,) = _grads(rng, [(64, 48)], ["f32"])
    t = g.t()                                              # dense, in another order
    _check((t,), [g64.T], 0.3)
    assert np.allclose(g.double().cpu().numpy(), t.t().double().cpu().numpy())
    # the same tensor twice counts twice in the norm
    (h,), (h64,) = _grads(rng, [(100,)], ["f32"])
    assert_near(b.grad_norm([h, h]).cpu().numpy(), np.array([np.sqrt(2 * (h64 ** 2).sum())]),
                np.array([ref.NORM_REL * np.sqrt(2 * (h64 ** 2).sum())]), False, "norm")


@pytest.mark.parametrize("scale", [1e-30, 1e-25, 1e-15, 1e10, 1e18, 3e37])
def test_extreme_scales(scale):
    """Squares outside FP32's range, beside ordinary tensors and alone; zeros in between."""
    rng = np.random.default_rng(3)
    shapes = [(5000,), (4096,), (77,)]
    grads, g64 = _grads(rng, shapes, ["f32", "bf16", "f32"], scale)
    grads[1].zero_()
    g64[1][:] = 0
    if scale < 1e30:
        _check(grads, g64, 1e-3 * scale if scale > 1 else 1.0, ["f32"] * 3)
    else:   # the norm may pass FP32's largest value: its clipped gradients do not
        norm, factor, rel = ref.clip(g64, 1.0)
        import torch
        out = [torch.empty_like(g, dtype=torch.float32) for g in grads]
        lib().clip_grads(grads, 1.0, out=out)
        for o, g in zip(out, g64):
            assert_near(o.double().cpu().numpy(), g * factor, (rel + 2 * ref.U) * np.abs(g * factor) + TINY_F32, False, "out")
    mixed, m64 = _grads(rng, [(3000,), (3000,)], ["f32", "f32"])
    mixed[0] *= scale
    m64[0] = mixed[0].double().cpu().numpy()
    if scale < 1e30:
        norm = np.sqrt(sum((m ** 2).sum() for m in m64))
        assert_near(lib().grad_norm(mixed).cpu().numpy(), np.array([norm]), np.array([ref.NORM_REL * norm]), False, "norm")


def test_not_finite():
    import torch
    b = lib()
    g = [torch.ones(100, device="cuda"), torch.ones(50, dtype=torch.bfloat16, device="cuda")]
    g[0][7] = float("inf")
    out = [torch.empty_like(x) for x in g]
    norm, _ = b.clip_grads(g, 1.0, out=out)
    assert norm.item() == float("inf") and torch.isnan(out[0][7]) and (out[0][:7] == 0).all() and (out[1] == 0).all()
    g[0][7] = float("nan")
    norm, _ = b.clip_grads(g, 1.0)
    assert torch.isnan(norm).all() and torch.isnan(g[0]).all() and torch.isnan(g[1]).all()


def test_zero_norm_and_zero_limit():
    import torch
    b = lib()
    g = [torch.zeros(5000, device="cuda")]
    norm, _ = b.clip_grads(g, 0.0)
    assert norm.item() == 0 and (g[0] == 0).all()
    g = [torch.ones(5000, device="cuda")]
    norm, _ = b.clip_grads(g, 0.0)
    assert (g[0] == 0).all()


def test_large_stream_and_graph():
    """A tensor past 2^31 values; a side stream; two captured calls, each with its own table and workspace."""
    import torch
    b = lib()
    n = (1 << 31) + 4099
    big = torch.full((n,), 0.5, dtype=torch.bfloat16, device="cuda")
    big[-1] = 3.0
    norm, _ = b.clip_grads([big], 1.0)
    want = np.sqrt(0.25 * (n - 1) + 9.0)
    assert abs(norm.item() - want) <= ref.NORM_REL * want + ref.U * want
    f = torch.tensor(3.0 / want, dtype=torch.bfloat16).item()
    assert abs(big[-1].item() - 3.0 / want) <= 2 ** -8 * 3.0 / want and abs(f - big[-1].item()) <= 2 ** -7 * f
    assert (big[:7] == big[1 << 31]).all() and big[0].item() > 0
    del big
    rng = np.random.default_rng(9)
    grads, g64 = _grads(rng, [(5000,), (123,)], ["f32", "bf16"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = b.grad_norm(grads, stream=side)
    side.synchronize()
    assert torch.equal(got, b.grad_norm(grads))
    graphs = []
    for lim in (0.5, 0.25):
        out = [torch.empty_like(x) for x in grads]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            norm, _ = b.clip_grads(list(grads), lim, out=out)
        graphs.append((g, lim, norm, out))
    grads[0].mul_(3)
    g64[0] = grads[0].double().cpu().numpy()
    for g, *_ in graphs:
        g.replay()
    for _, lim, norm, out in graphs:
        n, factor, rel = ref.clip(g64, lim)
        assert_near(norm.cpu().numpy(), np.array([n]), np.array([ref.NORM_REL * n]), False, "norm")
        for o, x in zip(out, g64):
            assert_near(o.double().cpu().numpy(), x * factor, rel * np.abs(x * factor), o.dtype == torch.bfloat16, "out")


def test_refusals():
    import torch
    b = lib()
    g = torch.ones((8, 8), device="cuda")
    for bad in (lambda: b.grad_norm([g.half()]), lambda: b.grad_norm([g[:, ::2]]), lambda: b.grad_norm([g, None]),
                lambda: b.grad_norm(g), lambda: b.clip_grads([g], 1.0, out=[]), lambda: b.clip_grads([g], 1.0, out=[g[0]]),
                lambda: b.clip_grads([g], 1.0, out=[torch.ones((8, 8), device="cuda").t()])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: b.clip_grads([g], -1.0), lambda: b.clip_grads([g, g], 1.0), lambda: b.clip_grads([g, g[1]], 1.0),
                lambda: b.grad_norm([g], norm=g.view(-1)[:1])):
        with pytest.raises(b.MxGemmError):
            bad()
    assert (g == 1).all()
