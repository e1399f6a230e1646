"""Expert sort, dispatch, combine and their gradients on the GPU against the 64-bit
definition (row_ops_ref.py) and the oracle's quantiser, through the binding."""
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


def _dev(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _ids(rng, T, k, G, load="zipf", drop=0.0):
    """Expert ids [T, k]; uneven load; some outside the range; token T // 2 loses all its slots."""
    p = 1.0 / np.arange(1, G + 1) ** (1.2 if load == "zipf" else 0.0)
    ids = rng.permutation(G)[rng.choice(G, size=(T, k), p=p / p.sum())].astype(np.int64)
    if drop:
        ids[rng.random((T, k)) < drop] = -1
        ids[rng.random((T, k)) < drop] = G + 3
        ids[T // 2] = -1
    return ids


@pytest.mark.parametrize("dtype", [np.int32, np.int64])
@pytest.mark.parametrize("T,k,G", [
    (1, 1, 1), (1, 8, 64), (3, 2, 512), (31, 1, 5), (32, 8, 64), (129, 7, 60), (512, 8, 8), (513, 8, 8),
    (1000, 6, 256), (4099, 2, 8), (20011, 3, 512), (70001, 8, 64),
    (2048, 1, 4), (2049, 1, 512), (12288, 1, 300), (12289, 1, 300), (5461, 3, 64),
])
@pytest.mark.parametrize("drop", [0.0, 0.1])
def test_sort(dtype, T, k, G, drop):
    import torch
    b = lib()
    rng = np.random.default_rng([T, k, G])
    ids = _ids(rng, T, k, G, drop=drop).astype(dtype)
    guard = torch.full((G + 1 + 16,), -7, dtype=torch.int64, device="cuda")
    o, r, s = b.moe_sort(_dev(ids), G, offsets=guard[8:-8])
    wo, wr, ws = ref.moe_sort(ids, G)
    assert (o.cpu().numpy() == wo).all()
    assert (r.cpu().numpy() == wr).all()
    assert (s.cpu().numpy() == ws).all()
    assert (guard[:8] == -7).all() and (guard[-8:] == -7).all()


@pytest.mark.parametrize("value", [-1, 2, 1 << 40, -(1 << 62)])
def test_sort_one_expert_or_none(value):
    """All slots on one expert, or every one dropped (64-bit ids far outside the range among them)."""
    b = lib()
    ids = np.full((700, 2), value, np.int64)
    o, r, s = b.moe_sort(_dev(ids), 4)
    wo, wr, ws = ref.moe_sort(ids, 4)
    assert (o.cpu().numpy() == wo).all() and (r.cpu().numpy() == wr).all() and (s.cpu().numpy() == ws).all()


def test_sort_workspaces_of_streams_threads_and_graphs():
    """Sorts that overlap on two streams, in two threads and in a replayed graph do not share a workspace."""
    import threading
    import torch
    b = lib()
    rng = np.random.default_rng(77)
    T, k, G = 30000, 4, 64
    sets = [_ids(rng, T, k, G) for _ in range(4)]
    want = [ref.moe_sort(i, G) for i in sets]
    dev = [_dev(i) for i in sets]
    torch.cuda.synchronize()
    g, gs = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=gs):
        in_graph = b.moe_sort(dev[0], G)
    got, streams = {}, [torch.cuda.Stream() for _ in range(2)]

    def work(i):
        with torch.cuda.stream(streams[0]):     # both threads on one stream
            for _ in range(20):
                got[i] = b.moe_sort(dev[i], G)

    threads = [threading.Thread(target=work, args=(i,)) for i in (1, 2)]
    for t in threads:
        t.start()
    for _ in range(20):
        got[3] = b.moe_sort(dev[3], G, stream=streams[1])
        with torch.cuda.stream(gs):
            g.replay()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    got[0] = in_graph
    for i in range(4):
        for x, w in zip(got[i], want[i]):
            assert (x.cpu().numpy() == w).all(), i


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", [1, 2, 3])
@pytest.mark.parametrize("T,k,G,K,drop", [
    (1, 1, 4, 128, 0.0), (1, 8, 64, 2048, 0.0), (33, 2, 8, 384, 0.2), (200, 5, 7, 4096, 0.1), (65, 3, 16, 96, 0.1),
    (9, 40, 64, 640, 0.3), (300, 8, 64, 1056, 0.0),
])
def test_dispatch(oracle_mod, dtype, fmt, T, k, G, K, drop):
    import torch
    b = lib()
    rng = np.random.default_rng([T, k, K, fmt])
    ids = _ids(rng, T, k, G, drop=drop)
    x, x64 = _make(rng, (T, K), _dtype(dtype))
    if T > 8:  # a block with a NaN stays within its rows
        x[3, 40] = float("nan")
        x64[3, 40] = np.nan
    _, slot, source = b.moe_sort(_dev(ids), G)
    rows, scales = b.moe_dispatch(x, slot, fmt)
    offsets, _, src = ref.moe_sort(ids, G)
    live = (np.arange(T * k) < offsets[-1])[:, None]
    if fmt == 3:
        want = torch.where(_dev(live), x.to(torch.bfloat16)[_dev(src // k)], torch.zeros((), dtype=torch.bfloat16,
                                                                                        device="cuda"))
        assert torch.equal(rows.view(torch.int16), want.view(torch.int16))
        return
    codes, sc = oracle_mod.quantize(fmt, x.float().cpu().numpy(), oracle_mod.IN_F32)
    assert (rows.cpu().numpy() == np.where(live, codes[src // k], 0)).all()
    assert (scales.cpu().numpy() == np.where(live, sc[src // k], 127)).all()


def test_dispatch_of_strided_rows_guards_and_foreign_tables():
    """Rows of a wider matrix; nothing around the outputs is written; table entries that name no row write nothing."""
    import torch
    b = lib()
    rng = np.random.default_rng(2)
    T, k, K, pad = 6, 2, 160, 64
    wide, _ = _make(rng, (T, K + 96), _dtype("bf16"))
    x = wide[:, 64:64 + K]
    codes = torch.full((T * k * K + 2 * pad,), 0xA5, dtype=torch.uint8, device="cuda")
    table = torch.arange(T * k, dtype=torch.int32, device="cuda")
    table[3], table[5] = T * k, -1 - T * k      # past the end, and a dropped one past the end
    table[7], table[8] = 2 ** 31 - 1, -(2 ** 31)
    rows, scales = b.moe_dispatch(x, table, 1, rows=codes[pad:-pad].view(T * k, K))
    plain, _ = b.moe_dispatch(x.contiguous(), torch.arange(T * k, dtype=torch.int32, device="cuda"), 1)
    skipped = [3, 5, 7, 8]
    keep = [i for i in range(T * k) if i not in skipped]
    assert torch.equal(rows[keep], plain[keep]) and (rows[skipped] == 0xA5).all()
    assert (codes[:pad] == 0xA5).all() and (codes[-pad:] == 0xA5).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("T,k,G,N,add,drop", [
    (1, 1, 1, 32, False, 0.0), (1, 8, 64, 2048, True, 0.0), (37, 2, 8, 672, True, 0.2), (100, 8, 16, 4096, False, 0.1),
    (5, 40, 64, 512, True, 0.2), (513, 3, 5, 96, False, 0.0),
])
def test_combine(dtype, weighted, T, k, G, N, add, drop):
    import torch
    b = lib()
    rng = np.random.default_rng([T, k, N])
    dt, bf16 = _dtype(dtype), dtype == "bf16"
    ids = _ids(rng, T, k, G, drop=drop)
    offsets, slot, _ = ref.moe_sort(ids, G)
    y, y64 = _make(rng, (T * k, N), dt)
    y[offsets[-1]:] = float("nan")      # the rows of dropped slots are whatever the memory held
    w = rng.random((T, k)).astype(np.float32)
    w[(slot < 0).reshape(T, k)] = np.nan
    r, r64 = _make(rng, (T, N), dt) if add else (None, None)
    out = b.moe_combine(y, _dev(slot.astype(np.int32)), k, weights=_dev(w) if weighted else None, add=r)
    want, err = ref.moe_combine(y64, slot, k, w.astype(np.float64) if weighted else None, r64)
    ref.assert_near(_np(out), want, err, bf16, "out")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,G,N,drop", [
    (1, 1, 1, 32, 0.0), (1, 8, 64, 2048, 0.0), (37, 2, 8, 672, 0.2), (100, 8, 16, 4096, 0.1), (5, 40, 64, 512, 0.2),
    (513, 3, 5, 96, 0.0), (3, 1, 2, 8224, 0.0),
])
def test_combine_backward(dtype, T, k, G, N, drop):
    import torch
    b = lib()
    rng = np.random.default_rng([T, k, N, 1])
    dt, bf16 = _dtype(dtype), dtype == "bf16"
    offsets, slot, _ = ref.moe_sort(_ids(rng, T, k, G, drop=drop), G)
    y, y64 = _make(rng, (T * k, N), dt)
    y[offsets[-1]:] = float("nan")
    dout, dout64 = _make(rng, (T, N), dt)
    w = rng.random((T, k)).astype(np.float32)
    w[(slot < 0).reshape(T, k)] = np.nan
    dy, dw = b.moe_combine_backward(dout, y, _dev(slot.astype(np.int32)), _dev(w))
    wdy, wdw, err = ref.moe_combine_backward(dout64, y64, slot, w.astype(np.float64))
    ref.assert_near(_np(dy), wdy, ref.U * np.abs(wdy), bf16, "dy")
    assert dw.shape == (T, k)
    ref.assert_near(_np(dw).reshape(-1), wdw, err, False, "dweights")
    again = b.moe_combine_backward(dout, y, _dev(slot.astype(np.int32)), _dev(w))
    assert torch.equal(again[0], dy) and torch.equal(again[1], dw)


def test_combine_in_place_strided_and_guards():
    import torch
    b = lib()
    rng = np.random.default_rng(9)
    T, k, N, pad = 21, 2, 288, 64
    _, slot, _ = ref.moe_sort(_ids(rng, T, k, 4), 4)
    yw, yw64 = _make(rng, (T * k, 2 * N), _dtype("bf16"))
    buf = torch.full((T * N + 2 * pad,), 3.0, dtype=torch.bfloat16, device="cuda")
    res = buf[pad:-pad].view(T, N)
    r, r64 = _make(rng, (T, N), _dtype("bf16"))
    res.copy_(r)
    out = b.moe_combine(yw[:, N:], _dev(slot.astype(np.int32)), k, add=res, out=res)
    want, err = ref.moe_combine(yw64[:, N:], slot, k, None, r64)
    ref.assert_near(_np(out), want, err, True, "out")
    assert (buf[:pad] == 3.0).all() and (buf[-pad:] == 3.0).all()


def test_gradients_against_differences():
    """combine's kernel gradients along random directions against differences of the 64-bit forward."""
    b = lib()
    rng = np.random.default_rng(5)
    T, k, G, N = 8, 3, 4, 64
    _, slot, _ = ref.moe_sort(_ids(rng, T, k, G, drop=0.2), G)
    y, y64 = _make(rng, (T * k, N), _dtype("f32"))
    dout, dout64 = _make(rng, (T, N), _dtype("f32"))
    w = rng.random((T, k)).astype(np.float32)
    dy, dw = b.moe_combine_backward(dout, y, _dev(slot.astype(np.int32)), _dev(w))
    f = lambda y_, w_: (ref.moe_combine(y_, slot, k, w_)[0] * dout64).sum()  # noqa: E731
    vy, vw, e, w64 = rng.standard_normal(y64.shape), rng.standard_normal((T, k)), 1e-4, w.astype(np.float64)
    # the forward is bilinear: central differences are exact up to 64-bit rounding
    lim = 2 * ref.U * np.abs(_np(dy) * vy).sum() + 1e-9
    assert abs((f(y64 + e * vy, w64) - f(y64 - e * vy, w64)) / (2 * e) - (_np(dy) * vy).sum()) < lim
    size = np.abs(ref.moe_combine_backward(np.abs(dout64), np.abs(y64), slot, w64)[1].reshape(T, k) * vw).sum()
    assert abs((f(y64, w64 + e * vw) - f(y64, w64 - e * vw)) / (2 * e) - (_np(dw) * vw).sum()) < 12 * ref.U * size + 1e-9


def test_dispatch_feeds_the_grouped_gemm(oracle_mod):
    """sort -> dispatch -> grouped GEMM on one side stream: each kept slot's row is its token times its expert's weight."""
    import torch
    from gpu_util import small_int_codes
    b = lib()
    rng = np.random.default_rng(11)
    T, k, G, N, K = 50, 2, 6, 256, 512
    ids = _ids(rng, T, k, G, drop=0.1)
    x = rng.integers(-2, 3, (T, K)).astype(np.float32)       # exact in E4M3, exact sums
    B, SB = small_int_codes(rng, G * N, K, 1)
    dB, dSB, dx, dids = _dev(B), _dev(SB), _dev(x).to(torch.bfloat16), _dev(ids)
    plan = b.GroupedPlan(G, T * k, N, K, 1, b.MXGEMM_OUT_F32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        offs, slot, _ = b.moe_sort(dids, G)
        rows, scales = b.moe_dispatch(dx, slot, 1)
        C = plan.run(offs, rows, scales, dB, dSB)
    s.synchronize()
    b.check_device_status()
    codes, sc = oracle_mod.quantize(1, x, oracle_mod.IN_F32)
    got, table = C.cpu().numpy(), slot.cpu().numpy()
    for t in range(T):
        for j in range(k):
            e, row = ids[t, j], table[t * k + j]
            if 0 <= e < G:
                want, _ = oracle_mod.gemm(1, codes[t:t + 1], sc[t:t + 1], B[e * N:(e + 1) * N], SB[e * N:(e + 1) * N], K)
                assert (got[row] == want[0]).all()


def test_offsets_past_32_bits():
    """Rows whose bytes and elements pass 2^31: the last token's rows and sums are those of the token alone."""
    import torch
    b = lib()
    T, k, K = (1 << 31) // (8 * 4096) + 5, 8, 4096
    x = torch.full((T, K), 0.25, dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn((3, K), device="cuda").to(torch.bfloat16)
    table = torch.arange(T * k, dtype=torch.int32, device="cuda")
    small = torch.arange(3 * k, dtype=torch.int32, device="cuda")
    rows, scales = b.moe_dispatch(x, table, 3)
    part, _ = b.moe_dispatch(x[-3:], small, 3)
    assert torch.equal(rows[-3 * k:], part)
    out = b.moe_combine(rows, table, k)
    assert torch.equal(out[-3:], b.moe_combine(part, small, k))
    w = torch.rand((T, k), device="cuda")
    dy, dw = b.moe_combine_backward(x, rows, table, w)
    pdy, pdw = b.moe_combine_backward(x[-3:], part, small, w[-3:].contiguous())
    assert torch.equal(dy[-3 * k:], pdy) and torch.equal(dw[-3:], pdw)


@pytest.mark.parametrize("T", [6, 900])
def test_outputs_over_inputs(T):
    """dy over y gives what an apart output gives; outputs over other inputs are refused."""
    import torch
    b = lib()
    rng = np.random.default_rng(T)
    k, N = 2, 1056
    _, slot, _ = ref.moe_sort(_ids(rng, T, k, 4, drop=0.2), 4)
    slot = _dev(slot.astype(np.int32))
    y, dout = (_make(rng, (n, N), _dtype("bf16"))[0] for n in (T * k, T))
    w = _dev(rng.random((T, k)).astype(np.float32))
    want = b.moe_combine_backward(dout, y, slot, w)
    for call in (lambda: b.moe_combine(y, slot, k, out=y[:T]),
                 lambda: b.moe_dispatch(y[:T], slot, b.MXGEMM_FMT_BF16, rows=y),
                 lambda: b.moe_combine_backward(y[:T], y.clone(), slot, w, dy=y)):
        with pytest.raises(b.MxGemmError) as e:
            call()
        assert e.value.status == b.MXGEMM_ERR_ARG
    got = b.moe_combine_backward(dout, y, slot, w, dy=y)
    assert got[0] is y and torch.equal(y, want[0]) and torch.equal(got[1], want[1])


def test_weight_gradient_over_the_weights():
    """dweights over weights gives what an apart output gives, also where a warp takes several slots."""
    import torch
    b = lib()
    rng = np.random.default_rng(31)
    for T, k in ((5, 3), (9000, 4)):
        _, slot, _ = ref.moe_sort(_ids(rng, T, k, 8, drop=0.1), 8)
        slot = _dev(slot.astype(np.int32))
        y, dout = (_make(rng, (n, 96), _dtype("bf16"))[0] for n in (T * k, T))
        w = _dev(rng.random((T, k)).astype(np.float32))
        want = b.moe_combine_backward(dout, y, slot, w)
        got = b.moe_combine_backward(dout, y, slot, w, dweights=w)
        assert got[1] is w and torch.equal(w, want[1]) and torch.equal(got[0], want[0])


# Calls with more units than sixteen warps a multiprocessor take other kernels, or several slots a warp.

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", [1, 2, 3])
@pytest.mark.parametrize("T,k,K", [(5000, 2, 672), (3001, 3, 1056), (2500, 1, 1536), (2600, 5, 96)])
def test_dispatch_of_many_tokens(oracle_mod, dtype, fmt, T, k, K):
    import torch
    b = lib()
    rng = np.random.default_rng([T, k, K, fmt])
    ids = _ids(rng, T, k, 16, drop=0.1)
    x, _ = _make(rng, (T, K), _dtype(dtype))
    x[3, 40] = float("nan")
    x[T - 1, K - 1] = float("inf")
    offsets, slot, src = ref.moe_sort(ids, 16)
    pad = 64
    width = K if fmt == 1 else K // 2 if fmt == 2 else K
    buf = torch.full((T * k * width + 2 * pad,), 0x25, dtype=torch.bfloat16 if fmt == 3 else torch.uint8, device="cuda")
    rows, scales = b.moe_dispatch(x, _dev(slot.astype(np.int32)), fmt, rows=buf[pad:-pad].view(T * k, width))
    live = (np.arange(T * k) < offsets[-1])[:, None]
    assert (buf[:pad] == 0x25).all() and (buf[-pad:] == 0x25).all()
    if fmt == 3:
        want = torch.where(_dev(live), x.to(torch.bfloat16)[_dev(src // k)],
                           torch.zeros((), dtype=torch.bfloat16, device="cuda"))
        assert torch.equal(rows.view(torch.int16), want.view(torch.int16))
        return
    codes, sc = oracle_mod.quantize(fmt, x.float().cpu().numpy(), oracle_mod.IN_F32)
    assert (rows.cpu().numpy() == np.where(live, codes[src // k], 0)).all()
    assert (scales.cpu().numpy() == np.where(live, sc[src // k], 127)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("weighted,add", [(True, True), (False, False), (True, False)])
@pytest.mark.parametrize("T,k,N", [(1301, 3, 1056), (2600, 1, 96), (2433, 2, 512), (1500, 5, 672), (1220, 8, 640)])
def test_combine_of_many_tokens(dtype, weighted, add, T, k, N):
    b = lib()
    rng = np.random.default_rng([T, k, N])
    dt = _dtype(dtype)
    offsets, slot, _ = ref.moe_sort(_ids(rng, T, k, 16, drop=0.15), 16)
    y, y64 = _make(rng, (T * k, N), dt)
    y[offsets[-1]:] = float("nan")
    w = rng.random((T, k)).astype(np.float32)
    w[(slot < 0).reshape(T, k)] = np.nan
    r, r64 = _make(rng, (T, N), dt) if add else (None, None)
    out = b.moe_combine(y, _dev(slot.astype(np.int32)), k, weights=_dev(w) if weighted else None, add=r)
    want, err = ref.moe_combine(y64, slot, k, w.astype(np.float64) if weighted else None, r64)
    ref.assert_near(_np(out), want, err, dtype == "bf16", "out")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,N", [(7001, 3, 96), (5000, 8, 544), (20001, 1, 512), (10000, 2, 640)])
def test_combine_backward_of_many_slots(dtype, T, k, N):
    b = lib()
    rng = np.random.default_rng([T, k, N, 1])
    dt = _dtype(dtype)
    offsets, slot, _ = ref.moe_sort(_ids(rng, T, k, 16, drop=0.1), 16)
    y, y64 = _make(rng, (T * k, N), dt)
    y[offsets[-1]:] = float("nan")
    dout, dout64 = _make(rng, (T, N), dt)
    w = rng.random((T, k)).astype(np.float32)
    w[(slot < 0).reshape(T, k)] = np.nan
    dy, dw = b.moe_combine_backward(dout, y, _dev(slot.astype(np.int32)), _dev(w))
    wdy, wdw, err = ref.moe_combine_backward(dout64, y64, slot, w.astype(np.float64))
    ref.assert_near(_np(dy), wdy, ref.U * np.abs(wdy), dtype == "bf16", "dy")
    ref.assert_near(_np(dw).reshape(-1), wdw, err, False, "dweights")
