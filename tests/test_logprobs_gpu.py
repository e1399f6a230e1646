"""Log probabilities, entropy, the most probable tokens and the logits' gradient on the
GPU against the 64-bit definition (model_ops_ref.py), through the binding."""
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


def _np(t):
    return t.double().cpu().numpy()


def _logits(rng, rows, V, dtype, how="model"):
    import torch
    x = rng.standard_normal((rows, V)) * 2.5
    if how == "peaked":
        x[np.arange(rows), rng.integers(0, V, rows)] += 30
    elif how == "masked":
        x[rng.random((rows, V)) < np.linspace(0, 1, rows)[:, None]] = -np.inf
    elif how == "lowest":                       # masked by the type's lowest value, and one row by nothing else
        low = float(torch.finfo(_dt(dtype)).min)
        x[rng.random((rows, V)) < np.linspace(0.2, 1.2, rows)[:, None]] = low
    elif how == "equal":
        x[:] = rng.standard_normal((rows, 1))
    elif how == "steps":
        x = np.round(x)
    elif how == "rising":                       # every value exceeds all before it
        x = np.sort(x, 1)
    elif how == "block":                        # all large values next to each other
        x[:, V // 3: V // 3 + V // 8 + 1] += 40
    elif how == "far":
        x += rng.choice([-1e4, 1e4, 3e5], rows)[:, None]
    t = torch.from_numpy(x.astype(np.float32)).cuda().to(_dt(dtype))
    return t, _np(t)


def _targets(rng, rows, V, wide):
    import torch
    t = rng.integers(0, V, rows)
    t[rng.random(rows) < 0.1] = -100
    t[rng.random(rows) < 0.05] = V
    return torch.from_numpy(t.astype(np.int64 if wide else np.int32)).cuda(), t


def _check(x, x64, rng, scale=1.0, top=5, wide=True, stream=None):
    import torch
    b = lib()
    rows, V = x64.shape
    t, t64 = _targets(rng, rows, V, wide)
    got = b.logprobs(x, t, scale=scale, top=top, entropy=True, stream=stream)
    if stream is not None:
        stream.synchronize()
    r = ref.logprobs(x64, t64, float(np.float32(scale)))
    assert_near(_np(got.logprob), r["logprob"], r["logprob_err"], False, "logprob")
    assert_near(_np(got.entropy), r["entropy"], r["entropy_err"], False, "entropy")
    st = _np(got.stats)
    assert np.array_equal(st[:, 0], r["m"])
    assert_near(st[:, 1], r["log"], r["log_err"], False, "log of the sum")
    if top:
        ids, lp = ref.top(x64, r["z"], r["lns"], top)
        assert np.array_equal(got.top_ids.cpu().numpy(), ids)
        at = np.where(ids >= 0, np.take_along_axis(r["z"], np.maximum(ids, 0), 1), 0.0)
        assert_near(_np(got.top_logprobs), lp, np.where(ids >= 0, r["log_err"][:, None] + 3 * ref.U * np.abs(at), 0), False,
                    "top")
    again = b.logprobs(x, t, scale=scale, top=top, entropy=True)
    for a, c in zip(got, again):
        assert a is c is None or torch.equal(a, c)     # the same sums in every run
    return got, t, t64, r


SIZES = [(1, 1), (2, 2), (3, 15), (5, 16), (4, 17), (7, 31), (2, 47), (9, 100), (3, 513), (33, 1000), (6, 4096), (2, 8200),
         (3, 32000), (1, 50257), (5, 50257), (2, 131072), (1, 262147), (1, 1_000_003)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("top", [0, 1, 5, 32])
@pytest.mark.parametrize("rows,V", SIZES)
def test_sizes(rows, V, dtype, top):
    rng = np.random.default_rng([rows, V, top])
    x, x64 = _logits(rng, rows, V, dtype)
    _check(x, x64, rng, scale=[1.0, 0.7][V % 2], top=top, wide=rows % 2 == 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("how", ["peaked", "masked", "lowest", "equal", "steps", "rising", "block", "far"])
@pytest.mark.parametrize("rows,V,top", [(40, 300, 20), (12, 5000, 32), (6, 40000, 20), (700, 1100, 5), (3, 128256, 32)])
def test_shapes_of_rows(rows, V, top, how, dtype):
    rng = np.random.default_rng([rows, V])
    x, x64 = _logits(rng, rows, V, dtype, how)
    _check(x, x64, rng, top=top)


@pytest.mark.parametrize("rows,V,dtype,top,how", [(700, 9000, "bf16", 20, "model"), (900, 9001, "f32", 32, "masked"),
                                                  (900, 9000, "f32", 0, "model"), (1100, 9000, "bf16", 7, "steps"),
                                                  (1250, 33000, "f32", 20, "model")])
def test_rows_of_a_part_of_a_wave(rows, V, dtype, top, how):
    """Blocks of 192, 160, 128 and 96 threads."""
    rng = np.random.default_rng(rows + top)
    x, x64 = _logits(rng, rows, V, dtype, how)
    _check(x, x64, rng, top=top)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("outside", ["-inf", "lower", "steps"])
@pytest.mark.parametrize("rows,V,first,n", [(3, 128256, 40000, 1000), (2, 128256, 127000, 1256), (160, 60000, 4096, 2048),
                                            (160, 60001, 0, 700), (700, 5000, 513, 900), (5, 1_000_003, 500_000, 40_000)])
def test_one_range_of_tokens(rows, V, first, n, outside, dtype):
    """The largest logits are a range's, which few threads hold; then in steps, many of them equal."""
    rng = np.random.default_rng([rows, first])
    x, _ = _logits(rng, rows, V, dtype, "steps" if outside == "steps" else "model")
    x[:, first:first + n] += 40
    if outside == "-inf":
        x[:, :first] = x[:, first + n:] = -float("inf")
    for top in (1, 20, 32):
        _check(x, _np(x), rng, top=top)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [2, 160])
def test_most_probable_tokens_of_two_threads(rows, dtype):
    """More of them than are ranked at once, at the places of two threads of a block of 256."""
    rng = np.random.default_rng(rows)
    V, values = 65536 * (2 if rows > 100 else 8), 16 if dtype == "bf16" else 8
    x, _ = _logits(rng, rows, V, dtype)
    x[:, (np.arange(V) // values % 256 == 9) | (np.arange(V) // values % 256 == 201)] += 40
    for top in (5, 20):
        _check(x, _np(x), rng, top=top)


@pytest.mark.parametrize("rows,V,threads", [(2500, 500, 32), (2500, 5000, 32), (2600, 20000, 128), (400, 9000, 256)])
def test_many_rows(rows, V, threads):
    """Enough rows for every rule on a block's size."""
    rng = np.random.default_rng(rows)
    x, x64 = _logits(rng, rows, V, "bf16", "steps" if V == 500 else "model")
    _check(x, x64, rng, top=20)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,offset,stride", [(1000, 1, 1001), (1000, 3, 1007), (333, 0, 335), (50001, 5, 50016), (20, 1, 21)])
def test_rows_that_start_anywhere(V, offset, stride, dtype):
    import torch
    rng = np.random.default_rng(V)
    base, _ = _logits(rng, 1, 6 * stride + 16, dtype)
    x = torch.as_strided(base, (6, V), (stride, 1), offset)
    got, t, t64, r = _check(x, _np(x), rng, top=5)
    _backward(x, _np(x), got, t, t64, 1.0, rng, dtype)


def test_rows_without_values_and_with_too_many():
    """All -inf; one value; NaN; +inf: the header's words."""
    import torch
    b = lib()
    x = torch.full((6, 777), float("-inf"), device="cuda")
    x[1, 500] = -3.0
    x[2] = 0.5
    x[2, 7] = float("nan")
    x[3] = 0.25
    x[3, 9] = float("inf")
    x[5, :2] = torch.tensor([2.0, 2.0], device="cuda")
    for dt in (torch.float32, torch.bfloat16):
        t = torch.tensor([3, 500, 8, 9, -1, 1], device="cuda")
        got = b.logprobs(x.to(dt), t, top=3, entropy=True)
        lp, en, st = _np(got.logprob), _np(got.entropy), _np(got.stats)
        assert lp[0] == -np.inf and en[0] == 0 and st[0].tolist() == [-np.inf, 0]
        assert lp[1] == 0 and en[1] == 0 and st[1].tolist() == [-3, 0]
        assert np.isnan(lp[2]) and np.isnan(en[2]) and np.isnan(st[2, 1])
        assert np.isnan(lp[3]) and np.isnan(en[3])
        assert lp[4] == 0 and en[4] == 0
        # two equal values: ln 2 of a sum of two exact ones, rounded by logf (one unit) and where it is stored
        for v, w in ((lp[5], -np.log(2)), (en[5], np.log(2)), (st[5, 1], np.log(2))):
            assert abs(v - w) <= 4 * ref.U * np.log(2)
        ids = got.top_ids.cpu().numpy().tolist()
        assert ids[0] == [-1, -1, -1] and ids[1] == [500, -1, -1] and ids[5] == [0, 1, -1] and ids[4] == [-1, -1, -1]
        assert ids[2] == [0, 1, 2] and ids[3][0] == 9
        d = b.logprobs_backward(x.to(dt), t, got.stats, torch.ones(6, device="cuda"), entropy=got.entropy,
                                dentropy=torch.ones(6, device="cuda"))
        assert (d[[0, 4]] == 0).all() and (d[1] == 0).all() and torch.isnan(d[2]).any()


def test_parts_alone():
    import torch
    b, rng = lib(), np.random.default_rng(2)
    x, x64 = _logits(rng, 9, 3000, "f32")
    t, _ = _targets(rng, 9, 3000, True)
    whole = b.logprobs(x, t, top=4, entropy=True)
    assert b.logprobs(x).logprob is None and b.logprobs(x).entropy is None and b.logprobs(x).top_ids is None
    assert torch.equal(b.logprobs(x, t).logprob, whole.logprob) and torch.equal(b.logprobs(x).stats, whole.stats)
    assert torch.equal(b.logprobs(x, entropy=True).entropy, whole.entropy)
    assert torch.equal(b.logprobs(x, top=4).top_ids, whole.top_ids)
    out = [torch.full_like(v, 9) for v in whole]
    got = b.logprobs(x, t, top=4, logprob=out[0], entropy=out[1], stats=out[2], top_ids=out[3], top_logprobs=out[4])
    assert all(a is o and torch.equal(o, w) for a, o, w in zip(got, out, whole))


def _backward(x, x64, got, t, t64, scale, rng, dtype, parts="both", over=False):
    import torch
    b = lib()
    rows = x64.shape[0]
    g, h = rng.standard_normal(rows).astype(np.float32), rng.standard_normal(rows).astype(np.float32)
    kw = {}
    if parts != "entropy":
        kw["dlogprob"] = torch.from_numpy(g).cuda()
    if parts != "logprob":
        kw["dentropy"], kw["entropy"] = torch.from_numpy(h).cuda(), got.entropy
    d = b.logprobs_backward(x, t if parts != "entropy" else None, got.stats, scale=scale, dlogits=x if over else None, **kw)
    want, err = ref.logprobs_backward(x64, t64, _np(got.stats), float(np.float32(scale)),
                                      g.astype(np.float64) if parts != "entropy" else None,
                                      _np(got.entropy), h.astype(np.float64) if parts != "logprob" else None)
    assert_near(_np(d), want, err + TINY_F32, dtype == "bf16", "dlogits")
    return d


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("parts", ["both", "logprob", "entropy"])
@pytest.mark.parametrize("rows,V", SIZES[:-1])
def test_gradient(rows, V, parts, dtype):
    rng = np.random.default_rng([rows, V])
    x, x64 = _logits(rng, rows, V, dtype, "masked" if rows > 4 else "model")
    scale = [1.0, 1.4][V % 2]
    got, t, t64, _ = _check(x, x64, rng, scale=scale, top=0)
    _backward(x, x64, got, t, t64, scale, rng, dtype, parts)
    _backward(x, x64, got, t, t64, scale, rng, dtype, parts, over=True)


@pytest.mark.parametrize("how", ["peaked", "lowest", "far", "equal"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradient_of_shapes_of_rows(how, dtype):
    rng = np.random.default_rng(4)
    x, x64 = _logits(rng, 20, 3001, dtype, how)
    got, t, t64, _ = _check(x, x64, rng, top=0)
    _backward(x, x64, got, t, t64, 1.0, rng, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradient_of_a_padded_vocabulary(dtype):
    """Logits whose rows have columns past the vocabulary: their gradient in place, beside, and dense."""
    import torch
    b, rng = lib(), np.random.default_rng(12)
    wide, _ = _logits(rng, 9, 1024, dtype)
    keep = wide.clone()
    x = wide[:, :999]
    x64 = _np(x)
    got, t, t64, _ = _check(x, x64, rng, top=4)
    dense = b.logprobs_backward(x, t, got.stats, torch.ones(9, device="cuda"))
    beside = torch.full_like(wide, 3.0)
    assert b.logprobs_backward(x, t, got.stats, torch.ones(9, device="cuda"), dlogits=beside[:, :999]).data_ptr() == beside.data_ptr()
    assert torch.equal(beside[:, :999], dense) and (beside[:, 999:] == 3).all()
    _backward(x, x64, got, t, t64, 1.0, rng, dtype, over=True)
    assert torch.equal(wide[:, 999:], keep[:, 999:])


def test_gradient_into_other_alignment():
    """Logits off a 32-byte boundary, their gradient on one: value by value."""
    import torch
    rng = np.random.default_rng(6)
    base, _ = _logits(rng, 1, 5 * 1000 + 8, "f32")
    x = base[0, 3:5003].view(5, 1000)
    got, t, t64, _ = _check(x, _np(x), rng, top=3)
    d = _backward(x, _np(x), got, t, t64, 1.0, rng, "f32")
    assert d.data_ptr() % 32 == 0 and x.data_ptr() % 32 == 12


def test_stream_and_graphs():
    import torch
    b, rng = lib(), np.random.default_rng(8)
    x, x64 = _logits(rng, 16, 9000, "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    _check(x, x64, rng, stream=side)
    t, _ = _targets(rng, 16, 9000, True)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = b.logprobs(x, t, top=20, entropy=True)
        d = b.logprobs_backward(x, t, out.stats, torch.ones(16, device="cuda"))
    y, _ = _logits(rng, 16, 9000, "bf16")
    x.copy_(y)
    g.replay()
    want = b.logprobs(y, t, top=20, entropy=True)
    assert all(torch.equal(a, c) for a, c in zip(out, want))
    assert torch.equal(d, b.logprobs_backward(y, t, want.stats, torch.ones(16, device="cuda")))


def test_offsets_past_32_bits():
    import torch
    b = lib()
    rows, V = 18, 130_001
    big = torch.empty((rows, 1 << 27), dtype=torch.bfloat16, device="cuda")     # rows 256 MB apart
    x = big[:, :V]
    x.normal_()
    t = torch.randint(0, V, (rows,), device="cuda")
    far, near = b.logprobs(x, t, top=5, entropy=True), b.logprobs(x.contiguous(), t, top=5, entropy=True)
    # rows start at other places against 32 bytes, so their sums' order is another: 8 units of 24 bits of ln S < 16
    assert torch.equal(far.top_ids, near.top_ids) and torch.equal(far.stats[:, 0], near.stats[:, 0])
    assert float((far.logprob - near.logprob).abs().max()) < 2e-5
    x = torch.zeros((40000, 60000), dtype=torch.bfloat16, device="cuda")        # 4.8 GB
    x[39999, 7] = 5.0
    t = torch.full((40000,), 7, device="cuda")
    got = b.logprobs(x, t, top=1)
    assert int(got.top_ids[39999, 0]) == 7 and int(got.top_ids[0, 0]) == 0
    d = b.logprobs_backward(x, t, got.stats, torch.ones(40000, device="cuda"), dlogits=x)
    assert float(d[39999, 7]) > 0.9 and float(d[39998, 6]) < 0


def test_refusals():
    import torch
    b = lib()
    x, t = torch.zeros((4, 100), device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    for bad in (lambda: b.logprobs(x.half(), t), lambda: b.logprobs(x, t.float()), lambda: b.logprobs(x, t[:3]),
                lambda: b.logprobs(x.t(), t), lambda: b.logprobs(x, t, entropy=torch.zeros(3, device="cuda")),
                lambda: b.logprobs_backward(x, t, torch.zeros(4, device="cuda"), torch.zeros(4, device="cuda")),
                lambda: b.logprobs(x, t, top=3, top_ids=torch.zeros((4, 3), dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    st = torch.zeros((4, 2), device="cuda")
    for bad in (lambda: b.logprobs(x, t, scale=0.0), lambda: b.logprobs(x, t, top=33), lambda: b.logprobs(x, t, top=-1),
                lambda: b.logprobs_backward(x, t, st), lambda: b.logprobs_backward(x, None, st, torch.zeros(4, device="cuda")),
                lambda: b.logprobs_backward(x, None, st, dentropy=torch.zeros(4, device="cuda")),
                lambda: b.logprobs_backward(x, t, st, torch.zeros(4, device="cuda"), scale=float("inf"))):
        with pytest.raises(b.MxGemmError):
            bad()
