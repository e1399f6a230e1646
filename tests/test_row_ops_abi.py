"""Refusals of the row operators' entry points: arguments are checked on the host,
before any device call (no GPU needed)."""
import pytest

ARG, SHAPE, ALIGN, WORKSPACE, UNSUPPORTED = -1, -2, -3, -4, -8


@pytest.fixture(scope="module")
def lib():
    from mx_block_scaled_gb300 import build
    build.build()
    from mx_block_scaled_gb300 import binding
    return binding


def _call(lib, name, good, change):
    args = dict(good)
    args.update(change)
    return getattr(lib._lib, name)(*args.values())


NORM = dict(in_dtype=2, x=64, x_stride=256, residual=64, residual_stride=256, weight=64, weight_dtype=2, eps=1e-5,
            rows=4, K=256, h=64, y=64, fmt=1, codes=64, scales=64, rstd=64, flags=0, stream=None)


@pytest.mark.parametrize("change,expect", [
    (dict(x=None), ARG), (dict(weight=None), ARG), (dict(in_dtype=3), ARG), (dict(weight_dtype=0), ARG),
    (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG), (dict(fmt=3), ARG), (dict(fmt=0), ARG),
    (dict(codes=None), ARG), (dict(scales=None), ARG), (dict(flags=2), ARG),
    (dict(h=None, y=None, fmt=0, codes=None, scales=None, rstd=None), ARG),
    (dict(rows=0), SHAPE), (dict(rows=1 << 31), SHAPE), (dict(K=40), SHAPE), (dict(K=0), SHAPE),
    (dict(x_stride=255), SHAPE), (dict(residual_stride=0), SHAPE), (dict(K=96, flags=1), SHAPE),
    (dict(x=80), ALIGN), (dict(x_stride=264), ALIGN), (dict(residual=16), ALIGN), (dict(weight=48), ALIGN),
    (dict(h=48), ALIGN), (dict(y=48), ALIGN), (dict(codes=8), ALIGN), (dict(scales=4), ALIGN), (dict(rstd=2), ALIGN),
    (dict(K=32768 + 32, x_stride=1 << 16, residual_stride=1 << 16), UNSUPPORTED),
])
def test_rmsnorm(lib, change, expect):
    assert _call(lib, "mxgemm_rmsnorm", NORM, change) == expect


BACK = dict(in_dtype=1, dy=64, dy_stride=256, h=64, h_stride=256, rstd=64, weight=64, weight_dtype=1, dh=64,
            dh_stride=256, rows=1500, K=256, dx=64, dweight=64, workspace=64, ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("change,expect", [
    (dict(dy=None), ARG), (dict(h=None), ARG), (dict(rstd=None), ARG), (dict(weight=None), ARG), (dict(dx=None), ARG),
    (dict(dweight=None), ARG), (dict(in_dtype=0), ARG), (dict(weight_dtype=7), ARG),
    (dict(rows=-1), SHAPE), (dict(K=33), SHAPE), (dict(dh_stride=8), SHAPE), (dict(h_stride=255), SHAPE),
    (dict(dy=48), ALIGN), (dict(dh_stride=260), ALIGN), (dict(dx=16), ALIGN), (dict(dweight=16), ALIGN),
    (dict(workspace=16), ALIGN),
    (dict(workspace=None), WORKSPACE), (dict(ws_bytes=608 * 256 * 4 - 1), WORKSPACE),
    (dict(K=65536, dy_stride=65536, h_stride=65536, dh_stride=65536, ws_bytes=1 << 30), UNSUPPORTED),
])
def test_rmsnorm_backward(lib, change, expect):
    assert _call(lib, "mxgemm_rmsnorm_backward", BACK, change) == expect


def test_rmsnorm_backward_workspace(lib):
    f = lib.mxgemm_rmsnorm_backward_workspace_bytes
    assert f(4, 256) == f(1024, 8192) == 0          # one launch, no partial sums
    assert f(1500, 256) == 608 * 256 * 4 and f(4, 16384) == 4 * 16384 * 4
    assert f(0, 256) == f(4, 40) == f(4, 65536) == 0
    assert f(1 << 20, 8192) == f(1 << 21, 8192) <= 1 << 24


GLU = dict(act=1, in_dtype=2, gate=64, up=64, stride=512, rows=4, F=256, y=64, fmt=2, codes=64, scales=64, flags=1,
           kept_codes=64, kept_scales=64, stream=None)


@pytest.mark.parametrize("change,expect", [
    (dict(gate=None), ARG), (dict(up=None), ARG), (dict(act=0), ARG), (dict(act=3), ARG), (dict(in_dtype=9), ARG),
    (dict(kept_codes=None), ARG), (dict(kept_scales=None), ARG), (dict(fmt=0), ARG), (dict(flags=4), ARG),
    (dict(y=None, fmt=0, codes=None, scales=None, flags=0, kept_codes=None, kept_scales=None), ARG),
    (dict(rows=0), SHAPE), (dict(F=16), SHAPE), (dict(F=96), SHAPE), (dict(stride=255), SHAPE),
    (dict(gate=48), ALIGN), (dict(up=48), ALIGN), (dict(stride=520), ALIGN), (dict(y=16), ALIGN),
    (dict(kept_codes=8), ALIGN), (dict(kept_scales=8), ALIGN), (dict(codes=8), ALIGN),
])
def test_glu(lib, change, expect):
    assert _call(lib, "mxgemm_glu", GLU, change) == expect


GLUB = dict(act=2, in_dtype=2, dy=64, dy_stride=256, gate=None, up=None, stride=0, kept_codes=64, kept_scales=64,
            rows=4, F=256, dgu=64, fmt=1, codes=64, scales=64, flags=1, a=64, stream=None)


@pytest.mark.parametrize("change,expect", [
    (dict(dy=None), ARG), (dict(act=5), ARG), (dict(in_dtype=0), ARG), (dict(kept_scales=None), ARG),
    (dict(gate=64, up=64, stride=512), ARG),                    # both forms of the inputs
    (dict(kept_codes=None, kept_scales=None), ARG),             # neither
    (dict(kept_codes=None, kept_scales=None, gate=64, stride=512), ARG),
    (dict(fmt=7), ARG), (dict(dgu=None, fmt=0, codes=None, scales=None, flags=0, a=None), ARG),
    (dict(F=32 + 64), SHAPE),                                   # 2F = 192: no whole tiles
    (dict(F=8), SHAPE), (dict(rows=0), SHAPE), (dict(dy_stride=8), SHAPE),
    (dict(kept_codes=None, kept_scales=None, gate=64, up=64, stride=255), SHAPE),
    (dict(dy=16), ALIGN), (dict(dgu=16), ALIGN), (dict(a=16), ALIGN), (dict(kept_codes=4), ALIGN),
    (dict(dy_stride=257), ALIGN),
])
def test_glu_backward(lib, change, expect):
    assert _call(lib, "mxgemm_glu_backward", GLUB, change) == expect


SORT = dict(expert_ids=64, id_bytes=8, slots=16, groups=4, offsets=64, row_of_slot=64, slot_of_row=64,
            workspace=None, ws_bytes=0, stream=None)


@pytest.mark.parametrize("change,expect", [
    (dict(expert_ids=None), ARG), (dict(offsets=None), ARG), (dict(row_of_slot=None), ARG), (dict(id_bytes=2), ARG),
    (dict(slots=0), SHAPE), (dict(slots=1 << 31), SHAPE), (dict(groups=0), SHAPE), (dict(groups=513), SHAPE),
    (dict(expert_ids=68), ALIGN), (dict(offsets=4), ALIGN), (dict(row_of_slot=66), ALIGN), (dict(slot_of_row=1), ALIGN),
    (dict(workspace=8), ALIGN), (dict(slots=1 << 20), WORKSPACE), (dict(slots=1 << 20, workspace=64, ws_bytes=64), WORKSPACE),
])
def test_moe_sort(lib, change, expect):
    assert _call(lib, "mxgemm_moe_sort", SORT, change) == expect


def test_moe_sort_workspace(lib):
    f = lib.mxgemm_moe_sort_workspace_bytes
    assert f(16, 4) == 0 and f(0, 4) == 0 and f(1 << 20, 513) == 0
    assert 0 < f(1 << 20, 64) <= 1 << 20 and 0 < f((1 << 31) - 1, 512) <= 1 << 20


SEND = dict(in_dtype=2, x=64, x_stride=256, tokens=4, topk=2, K=256, row_of_slot=64, fmt=1, rows=64, scales=64,
            stream=None)


@pytest.mark.parametrize("change,expect", [
    (dict(x=None), ARG), (dict(row_of_slot=None), ARG), (dict(rows=None), ARG), (dict(fmt=0), ARG), (dict(fmt=4), ARG),
    (dict(scales=None), ARG), (dict(fmt=3), ARG), (dict(in_dtype=3), ARG),
    (dict(tokens=0), SHAPE), (dict(topk=0), SHAPE), (dict(tokens=1 << 20, topk=1 << 12), SHAPE), (dict(tokens=1, topk=(1 << 20) + 1), SHAPE),
    (dict(K=48), SHAPE),
    (dict(x_stride=128), SHAPE),
    (dict(x=16), ALIGN), (dict(x_stride=257), ALIGN), (dict(row_of_slot=2), ALIGN), (dict(rows=8), ALIGN),
    (dict(scales=8), ALIGN), (dict(fmt=3, scales=None, rows=16), ALIGN),
    (dict(tokens=1 << 29, K=8192, x_stride=8192), UNSUPPORTED),
])
def test_moe_dispatch(lib, change, expect):
    assert _call(lib, "mxgemm_moe_dispatch", SEND, change) == expect


COMB = dict(in_dtype=2, y=64, y_stride=256, tokens=4, topk=2, N=256, row_of_slot=64, weights=64, add=64,
            add_stride=256, out=64, stream=None)


@pytest.mark.parametrize("change,expect", [
    (dict(y=None), ARG), (dict(row_of_slot=None), ARG), (dict(out=None), ARG), (dict(in_dtype=0), ARG),
    (dict(tokens=0), SHAPE), (dict(topk=-1), SHAPE), (dict(tokens=1, topk=1 << 30), SHAPE), (dict(N=250), SHAPE), (dict(y_stride=0), SHAPE),
    (dict(add_stride=100), SHAPE),
    (dict(y=16), ALIGN), (dict(add=16), ALIGN), (dict(out=16), ALIGN), (dict(weights=2), ALIGN),
    (dict(y_stride=260), ALIGN), (dict(tokens=1 << 29, N=8192, y_stride=8192, add_stride=8192), UNSUPPORTED),
])
def test_moe_combine(lib, change, expect):
    assert _call(lib, "mxgemm_moe_combine", COMB, change) == expect


COMBB = dict(in_dtype=2, dout=64, dout_stride=256, y=64, y_stride=256, tokens=4, topk=2, N=256, row_of_slot=64,
             weights=64, dy=64, dweights=64, stream=None)


@pytest.mark.parametrize("change,expect", [
    (dict(dout=None), ARG), (dict(y=None), ARG), (dict(row_of_slot=None), ARG), (dict(weights=None), ARG),
    (dict(dy=None), ARG), (dict(dweights=None), ARG), (dict(in_dtype=8), ARG),
    (dict(tokens=0), SHAPE), (dict(N=0), SHAPE), (dict(dout_stride=8), SHAPE), (dict(y_stride=8), SHAPE),
    (dict(dout=16), ALIGN), (dict(dy=16), ALIGN), (dict(dweights=2), ALIGN), (dict(dout_stride=260), ALIGN),
])
def test_moe_combine_backward(lib, change, expect):
    assert _call(lib, "mxgemm_moe_combine_backward", COMBB, change) == expect


def test_binding_refuses_host_tensors_and_wrong_shapes(lib):
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(4, 256), torch.ones(256)
    ids = torch.zeros(4, 2, dtype=torch.int64)
    with pytest.raises(ValueError):
        lib.rmsnorm(x, w, 1e-5)
    with pytest.raises(ValueError):
        lib.rmsnorm_backward(x, x, torch.ones(4), w)
    with pytest.raises(ValueError):
        lib.glu(x, x, lib.MXGEMM_ACT_SILU, plain=True)
    with pytest.raises(ValueError):
        lib.glu_backward(x, lib.MXGEMM_ACT_SILU, gate=x, up=x)
    with pytest.raises(ValueError):
        lib.moe_sort(ids, 4)
    with pytest.raises(ValueError):
        lib.moe_dispatch(x, ids.int(), lib.MXGEMM_FMT_MXFP8_E4M3)
    with pytest.raises(ValueError):
        lib.moe_combine(x, ids.int(), 2)
    with pytest.raises(ValueError):
        lib.moe_combine_backward(x, x, ids.int(), w)


# outputs that touch an input: at 1 << 20 .. of a matrix that the good call has elsewhere
APART = dict(
    mxgemm_rmsnorm=dict(in_dtype=2, x=1 << 20, x_stride=256, residual=2 << 20, residual_stride=512, weight=64,
                        weight_dtype=2, eps=1e-5, rows=4, K=256, h=3 << 20, y=4 << 20, fmt=1, codes=5 << 20, scales=64,
                        rstd=64, flags=0, stream=None),
    mxgemm_rmsnorm_backward=dict(in_dtype=1, dy=1 << 20, dy_stride=256, h=2 << 20, h_stride=256, rstd=64, weight=64,
                                 weight_dtype=1, dh=3 << 20, dh_stride=512, rows=4, K=256, dx=4 << 20, dweight=64,
                                 workspace=None, ws_bytes=0, stream=None),
    mxgemm_glu=dict(act=1, in_dtype=2, gate=1 << 20, up=(1 << 20) + 512, stride=512, rows=4, F=256, y=2 << 20, fmt=2,
                    codes=3 << 20, scales=64, flags=1, kept_codes=4 << 20, kept_scales=64, stream=None),
    mxgemm_glu_backward=dict(act=2, in_dtype=2, dy=1 << 20, dy_stride=256, gate=2 << 20, up=(2 << 20) + 512,
                             stride=512, kept_codes=None, kept_scales=None, rows=4, F=256, dgu=3 << 20, fmt=1,
                             codes=4 << 20, scales=64, flags=1, a=5 << 20, stream=None),
    mxgemm_moe_sort=dict(expert_ids=1 << 20, id_bytes=4, slots=600, groups=8, offsets=2 << 20, row_of_slot=3 << 20,
                         slot_of_row=4 << 20, workspace=None, ws_bytes=0, stream=None),
    mxgemm_moe_dispatch=dict(in_dtype=2, x=1 << 20, x_stride=512, tokens=4, topk=2, K=256, row_of_slot=64, fmt=1,
                             rows=2 << 20, scales=64, stream=None),
    mxgemm_moe_combine=dict(in_dtype=2, y=1 << 20, y_stride=256, tokens=4, topk=2, N=256, row_of_slot=64, weights=64,
                            add=2 << 20, add_stride=512, out=3 << 20, stream=None),
    mxgemm_moe_combine_backward=dict(in_dtype=2, dout=1 << 20, dout_stride=256, y=2 << 20, y_stride=512, tokens=4,
                                     topk=2, N=256, row_of_slot=64, weights=64, dy=3 << 20, dweights=64, stream=None),
)


@pytest.mark.parametrize("name,change", [
    ("mxgemm_rmsnorm", dict(h=2 << 20)),                       # the residual itself, but with a stride
    ("mxgemm_rmsnorm", dict(y=(1 << 20) + 512)),               # x, a row on
    ("mxgemm_rmsnorm", dict(y=(1 << 20) - 4 * 512 + 32)),      # its end in x
    ("mxgemm_rmsnorm", dict(codes=(2 << 20) + 3 * 1024)),      # the residual's last row
    ("mxgemm_rmsnorm_backward", dict(dx=1 << 20)), ("mxgemm_rmsnorm_backward", dict(dx=2 << 20)),
    ("mxgemm_rmsnorm_backward", dict(dx=3 << 20)),
    ("mxgemm_rmsnorm_backward", dict(dh_stride=256, dx=(3 << 20) + 32)),
    ("mxgemm_glu", dict(y=1 << 20)), ("mxgemm_glu", dict(codes=1 << 20)), ("mxgemm_glu", dict(kept_codes=(1 << 20) + 64)),
    ("mxgemm_glu_backward", dict(dgu=1 << 20)), ("mxgemm_glu_backward", dict(dgu=(2 << 20) + 32)),
    ("mxgemm_glu_backward", dict(dgu=2 << 20, stride=1024)),
    ("mxgemm_glu_backward", dict(dgu=2 << 20, gate=(2 << 20) + 512, up=2 << 20)),  # the halves the other way round
    ("mxgemm_glu_backward", dict(a=2 << 20)), ("mxgemm_glu_backward", dict(a=(1 << 20) + 32)),
    ("mxgemm_glu_backward", dict(codes=1 << 20)),
    ("mxgemm_moe_sort", dict(row_of_slot=1 << 20)), ("mxgemm_moe_sort", dict(slot_of_row=(1 << 20) + 599 * 4)),
    ("mxgemm_moe_sort", dict(offsets=(1 << 20) - 64)), ("mxgemm_moe_sort", dict(id_bytes=8, row_of_slot=(1 << 20) + 4796)),
    ("mxgemm_moe_dispatch", dict(rows=(1 << 20) + 3 * 1024)), ("mxgemm_moe_dispatch", dict(rows=(1 << 20) - 8 * 256 + 16)),
    ("mxgemm_moe_combine", dict(out=1 << 20)), ("mxgemm_moe_combine", dict(out=2 << 20)),
    ("mxgemm_moe_combine", dict(out=(1 << 20) + 7 * 512)),
    ("mxgemm_moe_combine_backward", dict(dy=1 << 20)), ("mxgemm_moe_combine_backward", dict(dy=2 << 20)),
])
def test_outputs_apart_from_inputs(lib, name, change):
    assert _call(lib, name, APART[name], change) == ARG
