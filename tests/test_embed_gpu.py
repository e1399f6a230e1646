"""Embedding rows and the table's gradient on the GPU against the 64-bit definition
(model_ops_ref.py), through the binding."""
import numpy as np
import pytest

import model_ops_ref as ref
from gpu_util import lib
from row_ops_ref import assert_near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    lib()


def _dt(name):
    import torch
    return dict(bf16=torch.bfloat16, f32=torch.float32)[name]


def _make(rng, shape, dtype):
    import torch
    t = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).cuda().to(_dt(dtype))
    return t, t.double().cpu().numpy()


def _np(t):
    return t.double().cpu().numpy()


def _ids(rng, n, vocab, how):
    if how == "one":
        return np.full(n, vocab // 2)
    if how == "none":
        return rng.choice([-1, vocab, -100, 1 << 20], n) if vocab <= 1 << 20 else np.full(n, -1)
    ids = rng.integers(0, vocab, n)
    if how == "skewed":
        ids = np.minimum((vocab * rng.random(n) ** 6).astype(np.int64), vocab - 1)
        ids[rng.random(n) < 0.1] = -1
        ids[rng.random(n) < 0.02] = vocab
    return ids


def _dev(ids, wide):
    import torch
    return torch.from_numpy(np.asarray(ids, np.int64 if wide else np.int32)).cuda()


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("tokens,K,vocab,wide", [(1, 32, 1, True), (3, 96, 50, False), (130, 512, 7, True),
                                                 (33, 1056, 1000, False), (700, 4096, 300, True)])
def test_lookup(dtype, out, tokens, K, vocab, wide):
    rng = np.random.default_rng([tokens, K])
    table, t64 = _make(rng, (vocab, K), dtype)
    ids = _ids(rng, tokens, vocab, "skewed")
    got = lib().embed(_dev(ids, wide), table, scale=1.75, dtype=_dt(out))
    want, err = ref.embed(t64, ids, 1.75)
    assert_near(_np(got), want, err, out == "bf16", "out")
    assert (_np(got)[(ids < 0) | (ids >= vocab)] == 0).all()


def test_lookup_strides_guards_and_far_ids():
    """Rows of a wider table, an id past 32 bits, a row past 2^32 bytes; nothing written around the output."""
    import torch
    b, rng = lib(), np.random.default_rng(5)
    wide, w64 = _make(rng, (40, 256), "bf16")
    ids = torch.tensor([[3, 39], [1 << 40, -(1 << 40)]], device="cuda")
    buf = torch.full((4 * 160 + 128,), 7.0, dtype=torch.bfloat16, device="cuda")
    got = b.embed(ids, wide[:, 64:224], out=buf[64:-64].view(4, 160))
    assert (_np(got)[:2] == w64[[3, 39], 64:224]).all() and (got[2:] == 0).all()
    assert (buf[:64] == 7).all() and (buf[-64:] == 7).all()
    big = torch.empty((700_000, 4096), dtype=torch.bfloat16, device="cuda")   # 5.7 GB
    big[-1] = 3.0
    big[0] = 2.0
    got = b.embed(torch.tensor([699_999, 0, 700_000], device="cuda", dtype=torch.int32), big, scale=-2.0)
    assert (got[0] == -6).all() and (got[1] == -4).all() and (got[2] == 0).all()
    assert not torch.signbit(got[2]).any()


def test_lookup_reads_named_rows_only():
    import torch
    table = torch.full((9, 64), float("nan"), device="cuda")
    table[4] = 1.0
    got = lib().embed(torch.tensor([4, -1, 9, 4], device="cuda"), table)
    assert _np(got).tolist() == [[1.0] * 64, [0.0] * 64, [0.0] * 64, [1.0] * 64]


# up to 64 tokens take no sort; the counting sort takes up to 2048 ids of tables below 2^21 - 1 rows, the radix sort the rest: one pass up to 1023 rows,
# two up to 2^20 - 1, three beyond
@pytest.mark.parametrize("tokens,vocab,K,how", [
    (1, 1, 32, "even"), (1, 50, 160, "none"), (7, 3, 96, "skewed"), (8, 9, 512, "one"), (9, 9, 512, "one"),
    (31, 40, 544, "skewed"), (64, 64, 64, "even"), (33, 5, 64, "even"), (64, 3, 4096, "one"), (64, 100, 1056, "skewed"), (65, 5, 1056, "skewed"), (1000, 300, 96, "skewed"),
    (1000, 1000, 4096, "even"), (3000, 2, 64, "one"), (8192, 5000, 64, "skewed"), (8192, 60, 32, "none"),
    (8193, 900, 64, "skewed"), (9000, 70000, 32, "even"), (20000, 5000, 96, "skewed"), (20000, 50, 32, "one"),
    (300, 600_000, 32, "even"), (33, 600_000, 32, "even"), (40000, 1_100_000, 32, "skewed"), (133, 524_287, 32, "even"), (133, 524_286, 32, "even"),
    (9000, 1023, 4096, "skewed"), (9000, 1024, 32, "skewed"), (70001, 128, 512, "skewed"),
])
@pytest.mark.parametrize("dtype,out,form", [("bf16", "f32", "plain"), ("f32", "bf16", "add"), ("f32", "f32", "in place"),
                                            ("bf16", "bf16", "in place")])
def test_gradient(tokens, vocab, K, how, dtype, out, form):
    import torch
    b, rng = lib(), np.random.default_rng([tokens, vocab])
    ids = _ids(rng, tokens, vocab, how)
    dy, d64 = _make(rng, (tokens, K), dtype)
    real = (ids >= 0) & (ids < vocab)
    dy[torch.from_numpy(~real).cuda()] = float("nan")      # rows without an id may hold anything
    d64[~real] = 0
    add, a64 = (None, None) if form == "plain" else _make(rng, (vocab, K), out)
    ids_dev = _dev(ids, tokens % 2 == 0)
    got = b.embed_backward(dy, ids_dev, vocab, scale=0.75, dtype=_dt(out), add=add, dtable=add if form == "in place" else None)
    want, err = ref.embed_backward(d64, ids, vocab, 0.75, a64)
    assert_near(_np(got), want, err, out == "bf16", "dtable")
    if form == "in place":
        assert got is add
        rest = np.setdiff1d(np.arange(vocab), ids[real])
        assert (_np(got)[rest] == a64[rest]).all()
    else:
        again = b.embed_backward(dy, ids_dev, vocab, scale=0.75, dtype=_dt(out), add=add)
        assert torch.equal(again, got)                     # the same sums in every run


@pytest.mark.parametrize("tokens,vocab,how", [(2047, 5000, "skewed"), (2048, 60, "none"), (2048, 2048, "even"), (2049, 900, "skewed"),
                                              (2049, 128256, "even"), (4100, 3, "one"), (700, 2_097_150, "skewed"),
                                              (700, 2_097_151, "skewed"), (65, 3_000_000, "even"), (2049, 3_000_000, "skewed")])
def test_gradient_around_the_rules_of_the_sort(tokens, vocab, how):
    import torch
    b, rng = lib(), np.random.default_rng([tokens, vocab])
    ids = _ids(rng, tokens, vocab, how)
    ids[tokens // 2:tokens // 2 + 2] = vocab - 1           # the last row, and ids outside the table
    ids[:2] = [vocab, -1]
    real = (ids >= 0) & (ids < vocab)
    dy, d64 = _make(rng, (tokens, 32), "f32")
    d64[~real] = 0
    # the rows that occur, and those next to them
    rows = np.unique(np.clip(np.concatenate([ids[real], ids[real] + 1, ids[real] - 1, [0, vocab - 1]]), 0, vocab - 1))
    place = np.full(tokens, -1)
    place[real] = np.searchsorted(rows, ids[real])
    got = b.embed_backward(dy, _dev(ids, tokens % 2 == 0), vocab, dtype=torch.float32)
    want, err = ref.embed_backward(d64, place, len(rows), 1.0, None)
    assert_near(_np(got[torch.from_numpy(rows).cuda()]), want, err, False, "dtable")
    assert int(got.any(1).sum()) == len(np.unique(ids[real]))


def test_gradient_strides_guards_stream_and_graph():
    """Rows inside a wider matrix, a side stream, a captured call with a workspace of its own, replayed on new ids."""
    import torch
    b, rng = lib(), np.random.default_rng(11)
    T, V, K = 300, 77, 96
    wide, w64 = _make(rng, (T, 160), "f32")
    dy, d64 = wide[:, 32:128], w64[:, 32:128]
    ids = _ids(rng, T, V, "skewed")
    ids_dev = _dev(ids, True)
    buf = torch.full((V * K + 64,), 5.0, device="cuda")
    out = buf[32:-32].view(V, K)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b.embed_backward(dy, ids_dev, V, dtable=out, stream=side)
    side.synchronize()
    assert_near(_np(out), *ref.embed_backward(d64, ids, V, 1.0), False, "dtable")
    assert (buf[:32] == 5).all() and (buf[-32:] == 5).all()
    graphs = []
    for _ in range(2):    # two captured calls, of which each has its own workspace
        g = torch.cuda.CUDAGraph()
        o = torch.empty((V, K), device="cuda")
        with torch.cuda.graph(g):
            b.embed_backward(dy, ids_dev, V, dtable=o)
        graphs.append((g, o))
    new = _ids(rng, T, V, "even")
    ids_dev.copy_(_dev(new, True))
    want = ref.embed_backward(d64, new, V, 1.0)
    for g, o in graphs:
        o.fill_(9)
        g.replay()
    for g, o in graphs:
        assert_near(_np(o), *want, False, "dtable")


def test_gradient_of_far_rows():
    """A table past 2^32 bytes, named at its ends."""
    import torch
    b = lib()
    V, K = 600_000, 4096
    dtable = torch.full((V, K), 1.0, dtype=torch.bfloat16, device="cuda")     # 4.9 GB
    dy = torch.full((5, K), 2.0, dtype=torch.bfloat16, device="cuda")
    b.embed_backward(dy, torch.tensor([V - 1, 0, V - 1, V, 17], device="cuda"), V, add=dtable, dtable=dtable)
    assert (dtable[V - 1] == 5).all() and (dtable[0] == 3).all() and (dtable[17] == 3).all() and (dtable[V - 2] == 1).all()
    b.embed_backward(dy, torch.tensor([V - 1, 0, V - 1, V, 17], device="cuda"), V, dtable=dtable)
    assert (dtable[V - 1] == 4).all() and (dtable[0] == 2).all() and (dtable[V - 2] == 0).all()
    assert int(dtable.count_nonzero()) == 3 * K


def test_refusals():
    import torch
    b = lib()
    table, ids = torch.ones((8, 64), device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        b.embed(ids.float(), table)
    with pytest.raises(ValueError):
        b.embed(ids, table.half())
    with pytest.raises(ValueError):
        b.embed(ids, table, dtype=torch.float16)
    with pytest.raises(b.MxGemmError):
        b.embed(ids, torch.ones((8, 40), device="cuda"))
    with pytest.raises(b.MxGemmError):
        b.embed(ids, table, scale=float("nan"))
    with pytest.raises((ValueError, b.MxGemmError)):
        b.embed(ids[:0], table)
    with pytest.raises(ValueError):
        b.embed_backward(table, ids, 8)                    # eight rows, four ids
    with pytest.raises((ValueError, b.MxGemmError)):
        b.embed_backward(table[:4], ids, 0)
    with pytest.raises(b.MxGemmError):
        b.embed_backward(table.repeat(20, 1), ids.repeat(40), 8, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        b.embed_backward(table[:4], ids, 9, add=table)
