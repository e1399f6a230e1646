"""Refusals of the model's row operators: arguments are checked on the host before any
device call.  The calls run in a process that sees no device, so that one which passes
the checks ends there (no GPU needed, none used)."""
import ctypes
import json
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, ARG, SHAPE, ALIGN, WORKSPACE, CUDA, UNSUPPORTED = 0, -1, -2, -3, -4, -6, -8
MB = 1 << 20
F32, BF16 = 1, 2

# every pointer of a good call in megabytes of its own
CALLS = dict(
    mxgemm_embed=dict(in_dtype=BF16, table=1 * MB, table_stride=256, vocab=100, K=256, ids=2 * MB, id_bytes=8, tokens=9,
                      scale=1.5, out_dtype=F32, out=3 * MB, stream=None),
    mxgemm_embed_backward=dict(in_dtype=BF16, dy=1 * MB, dy_stride=256, ids=2 * MB, id_bytes=4, tokens=99, vocab=100,
                               K=256, scale=1.0, add=3 * MB, out_dtype=F32, dtable=4 * MB, workspace=5 * MB,
                               ws_bytes=MB, stream=None),
    mxgemm_qk_norm_rope=dict(in_dtype=BF16, x=1 * MB, x_token=512, x_head=64, tokens=9, q_heads=4, k_heads=2, D=64,
                             q_weight=2 * MB, k_weight=3 * MB, weight_dtype=F32, eps=1e-6, rope=4 * MB, rope_rows=50,
                             rotary=32, positions=5 * MB, position_bytes=8, flags=1, y=6 * MB, y_token=384, y_head=64,
                             rstd=7 * MB, stream=None),
    mxgemm_qk_norm_rope_backward=dict(in_dtype=F32, dy=1 * MB, dy_token=384, dy_head=64, x=2 * MB, x_token=384,
                                      x_head=64, rstd=3 * MB, tokens=300, q_heads=4, k_heads=2, D=64, q_weight=4 * MB,
                                      k_weight=5 * MB, weight_dtype=BF16, rope=6 * MB, rope_rows=50, rotary=64,
                                      positions=7 * MB, position_bytes=4, flags=0, dx=8 * MB, dx_token=384, dx_head=64,
                                      dq_weight=9 * MB, dk_weight=10 * MB, workspace=11 * MB, ws_bytes=MB, stream=None),
    mxgemm_logprobs=dict(in_dtype=F32, logits=1 * MB, stride=101, rows=9, V=100, scale=0.5, targets=2 * MB, id_bytes=8,
                         logprob=3 * MB, entropy=4 * MB, stats=5 * MB, top=5, top_ids=6 * MB, top_logprobs=7 * MB,
                         stream=None),
    mxgemm_logprobs_backward=dict(in_dtype=BF16, logits=1 * MB, stride=100, rows=9, V=100, scale=2.0, targets=2 * MB,
                                  id_bytes=4, stats=3 * MB, dlogprob=4 * MB, entropy=5 * MB, dentropy=6 * MB,
                                  dlogits=7 * MB, dlogits_stride=100, stream=None),
)
NO_NORM = dict(q_weight=None, k_weight=None, rstd=None)
NO_NORM_BACK = dict(NO_NORM, x=None, dq_weight=None, dk_weight=None, workspace=None, ws_bytes=0)

REFUSED = [
    *(("mxgemm_embed", c, e) for c, e in [
        (dict(table=None), ARG), (dict(ids=None), ARG), (dict(out=None), ARG), (dict(in_dtype=3), ARG),
        (dict(out_dtype=0), ARG), (dict(id_bytes=2), ARG), (dict(scale=float("inf")), ARG), (dict(scale=float("nan")), ARG),
        (dict(tokens=0), SHAPE), (dict(vocab=0), SHAPE), (dict(K=40), SHAPE), (dict(table_stride=255), SHAPE),
        (dict(tokens=1 << 31), SHAPE), (dict(vocab=1 << 31), SHAPE),
        (dict(table=MB + 16), ALIGN), (dict(table_stride=264), ALIGN), (dict(ids=2 * MB + 4), ALIGN),
        (dict(out=3 * MB + 16), ALIGN),
        (dict(tokens=(1 << 31) - 1, K=4096, table_stride=4096), UNSUPPORTED),
        (dict(out=MB), ARG), (dict(out=MB + 99 * 512), ARG), (dict(out=2 * MB), ARG), (dict(out=2 * MB + 64), ARG)]),
    *(("mxgemm_embed_backward", c, e) for c, e in [
        (dict(dy=None), ARG), (dict(ids=None), ARG), (dict(dtable=None), ARG), (dict(in_dtype=0), ARG),
        (dict(out_dtype=3), ARG), (dict(id_bytes=1), ARG), (dict(scale=float("nan")), ARG),
        (dict(tokens=0), SHAPE), (dict(vocab=0), SHAPE), (dict(vocab=1 << 30), SHAPE), (dict(K=16), SHAPE),
        (dict(dy_stride=200), SHAPE),
        (dict(dy=MB + 16), ALIGN), (dict(dy_stride=260), ALIGN), (dict(ids=2 * MB + 2), ALIGN), (dict(add=3 * MB + 8), ALIGN),
        (dict(dtable=4 * MB + 16), ALIGN), (dict(workspace=5 * MB + 16), ALIGN),
        (dict(workspace=None), WORKSPACE), (dict(ws_bytes=100), WORKSPACE),
        (dict(K=1 << 29, dy_stride=1 << 29), UNSUPPORTED),
        (dict(dtable=MB), ARG), (dict(dtable=3 * MB + 32), ARG), (dict(dtable=2 * MB), ARG), (dict(dtable=5 * MB + 32), ARG),
        (dict(workspace=3 * MB), ARG), (dict(workspace=MB + 32), ARG), (dict(workspace=2 * MB), ARG)]),
    *(("mxgemm_qk_norm_rope", c, e) for c, e in [
        (dict(x=None), ARG), (dict(y=None), ARG), (dict(in_dtype=5), ARG), (dict(weight_dtype=0), ARG),
        (dict(q_weight=None), ARG), (dict(k_weight=None), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG),
        (dict(rope=None), ARG), (dict(positions=None), ARG), (dict(position_bytes=2), ARG), (dict(flags=2), ARG),
        (dict(NO_NORM, rope=None, positions=None), ARG),          # nothing to do
        (dict(q_weight=None, k_weight=None), ARG),                # rstd without a norm
        (dict(tokens=0), SHAPE), (dict(q_heads=-1), SHAPE), (dict(q_heads=0, k_heads=0), SHAPE), (dict(D=24), SHAPE),
        (dict(D=8), SHAPE), (dict(rotary=8), SHAPE), (dict(rotary=80), SHAPE), (dict(rotary=24), SHAPE), (dict(rotary=0), SHAPE),
        (dict(rope_rows=0), SHAPE), (dict(x_head=63), SHAPE), (dict(x_token=320), SHAPE), (dict(y_token=383), SHAPE),
        (dict(y_head=0), SHAPE),
        (dict(x=MB + 16), ALIGN), (dict(x_token=520), ALIGN), (dict(y=6 * MB + 8), ALIGN), (dict(y_head=72, y_token=512), ALIGN),
        (dict(q_weight=2 * MB + 16), ALIGN), (dict(rope=4 * MB + 16), ALIGN), (dict(positions=5 * MB + 4), ALIGN),
        (dict(rstd=7 * MB + 2), ALIGN),
        (dict(D=528, x_head=528, x_token=8192, y_head=528, y_token=8192), UNSUPPORTED),
        (dict(tokens=(1 << 31) - 1), UNSUPPORTED),
        (dict(y=MB), ARG), (dict(y=MB + 32, y_token=512), ARG), (dict(y=2 * MB), ARG), (dict(y=4 * MB), ARG),
        (dict(y=5 * MB), ARG), (dict(y=7 * MB), ARG), (dict(rstd=MB), ARG), (dict(rstd=5 * MB), ARG)]),
    *(("mxgemm_qk_norm_rope_backward", c, e) for c, e in [
        (dict(dy=None), ARG), (dict(dx=None), ARG), (dict(x=None), ARG), (dict(rstd=None), ARG), (dict(q_weight=None), ARG),
        (dict(NO_NORM_BACK, dq_weight=9 * MB), ARG), (dict(NO_NORM_BACK, rstd=3 * MB), ARG), (dict(flags=4), ARG),
        (dict(rope=None), ARG), (dict(in_dtype=0), ARG), (dict(weight_dtype=9), ARG),
        (dict(tokens=-1), SHAPE), (dict(D=72), SHAPE), (dict(rotary=128), SHAPE), (dict(dx_token=64), SHAPE),
        (dict(dy=MB + 4), ALIGN), (dict(dx_token=388), ALIGN), (dict(dq_weight=9 * MB + 1), ALIGN),
        (dict(workspace=11 * MB + 16), ALIGN), (dict(positions=7 * MB + 2), ALIGN),
        (dict(workspace=None), WORKSPACE), (dict(ws_bytes=64), WORKSPACE),
        (dict(D=1024, dy_head=1024, dy_token=8192, x_head=1024, x_token=8192, dx_head=1024, dx_token=8192), UNSUPPORTED),
        (dict(dx=MB + 32), ARG), (dict(dx=MB, dx_token=512), ARG), (dict(dx=2 * MB + 64), ARG), (dict(dx=3 * MB), ARG),
        (dict(dx=6 * MB), ARG), (dict(dx=11 * MB), ARG), (dict(dq_weight=10 * MB), ARG), (dict(dq_weight=MB), ARG),
        (dict(dk_weight=2 * MB), ARG), (dict(workspace=7 * MB), ARG), (dict(dx=MB, dq_weight=MB), ARG),
        (dict(dx=2 * MB, workspace=2 * MB), ARG)]),
    *(("mxgemm_logprobs", c, e) for c, e in [
        (dict(logits=None), ARG), (dict(targets=None), ARG), (dict(logprob=None), ARG), (dict(in_dtype=0), ARG),
        (dict(scale=0.0), ARG), (dict(scale=-1.0), ARG), (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG),
        (dict(id_bytes=3), ARG), (dict(top=0), ARG), (dict(top_ids=None), ARG), (dict(top_logprobs=None), ARG),
        (dict(targets=None, logprob=None, entropy=None, stats=None, top=0, top_ids=None, top_logprobs=None), ARG),
        (dict(rows=0), SHAPE), (dict(V=0), SHAPE), (dict(stride=99), SHAPE), (dict(top=-1), SHAPE), (dict(rows=1 << 31), SHAPE),
        (dict(logits=MB + 2), ALIGN), (dict(targets=2 * MB + 4), ALIGN), (dict(stats=5 * MB + 4), ALIGN),
        (dict(top_ids=6 * MB + 4), ALIGN), (dict(entropy=4 * MB + 1), ALIGN),
        (dict(top=33), UNSUPPORTED), (dict(rows=1 << 29), UNSUPPORTED),
        (dict(logprob=MB), ARG), (dict(entropy=MB + 8 * 404 + 396), ARG), (dict(stats=3 * MB + 32), ARG),
        (dict(top_ids=2 * MB), ARG), (dict(top_logprobs=6 * MB), ARG)]),
    *(("mxgemm_logprobs_backward", c, e) for c, e in [
        (dict(logits=None), ARG), (dict(stats=None), ARG), (dict(dlogits=None), ARG), (dict(targets=None), ARG),
        (dict(dlogprob=None), ARG), (dict(entropy=None), ARG), (dict(in_dtype=4), ARG), (dict(scale=0.0), ARG),
        (dict(targets=None, dlogprob=None, dentropy=None), ARG),
        (dict(rows=0), SHAPE), (dict(V=0), SHAPE), (dict(stride=50), SHAPE),
        (dict(logits=MB + 1), ALIGN), (dict(dlogits=7 * MB + 1), ALIGN), (dict(stats=3 * MB + 4), ALIGN),
        (dict(dlogits_stride=99), SHAPE), (dict(dlogits=MB + 2), ARG), (dict(dlogits=MB, stride=128), ARG), (dict(dlogits=2 * MB), ARG),
        (dict(dlogits=3 * MB), ARG), (dict(dlogits=4 * MB), ARG), (dict(dlogits=5 * MB), ARG), (dict(dlogits=6 * MB), ARG)]),
]
SERVED = [(name, {}) for name in CALLS] + [
    ("mxgemm_embed", dict(tokens=1, vocab=1, table_stride=0)),
    ("mxgemm_embed_backward", dict(dtable=3 * MB)), ("mxgemm_embed_backward", dict(add=None)),
    ("mxgemm_qk_norm_rope", dict(y=MB, y_token=512)),                             # in place
    ("mxgemm_qk_norm_rope", dict(x_token=64, x_head=576)),                        # [heads, tokens, D]
    ("mxgemm_qk_norm_rope", dict(q_heads=6, k_heads=0, k_weight=None)),
    ("mxgemm_qk_norm_rope", dict(q_heads=0, k_heads=6, q_weight=None)),
    ("mxgemm_qk_norm_rope", dict(rope=None, positions=None, rope_rows=0, rotary=0)),
    ("mxgemm_qk_norm_rope", NO_NORM), ("mxgemm_qk_norm_rope", dict(rstd=None)),
    ("mxgemm_qk_norm_rope_backward", dict(dx=MB)), ("mxgemm_qk_norm_rope_backward", dict(dx=2 * MB)),
    ("mxgemm_qk_norm_rope_backward", NO_NORM_BACK), ("mxgemm_qk_norm_rope_backward", dict(NO_NORM_BACK, dx=MB)),
    ("mxgemm_qk_norm_rope_backward", dict(dq_weight=None, dk_weight=None)),
    ("mxgemm_logprobs", dict(targets=None, logprob=None)), ("mxgemm_logprobs", dict(top=0, top_ids=None, top_logprobs=None)),
    ("mxgemm_logprobs", dict(entropy=None, stats=None)), ("mxgemm_logprobs", dict(logits=MB + 4)),
    ("mxgemm_logprobs", dict(top=32, V=3)),
    ("mxgemm_logprobs_backward", dict(dlogits=MB)), ("mxgemm_logprobs_backward", dict(dlogits=MB, stride=128, dlogits_stride=128)),
    ("mxgemm_logprobs_backward", dict(stride=128, dlogits_stride=104)), ("mxgemm_logprobs_backward", dict(entropy=None, dentropy=None)),
    ("mxgemm_logprobs_backward", dict(targets=None, dlogprob=None)),
]

# (tensors as (address, elements, dtype[, out address, out dtype]), other arguments, status)
GRADS = [
    ([(MB, 1000, F32), (2 * MB, 999, BF16)], {}, CUDA),
    ([(MB, 1000, F32, 3 * MB, BF16), (2 * MB, 999, BF16, 4 * MB, F32)], {}, CUDA),
    ([(MB, 1000, F32, MB, F32), (2 * MB, 999, BF16, 4 * MB, F32)], {}, CUDA),
    ([(2 * MB, 10, F32), (MB, 10, F32), (None, 0, F32)], {}, CUDA),      # any order, an empty one
    ([], {}, CUDA),
    ([(MB, 10, F32), (None, 5, F32)], {}, ARG), ([(MB, 10, 7)], {}, ARG), ([(MB, -1, F32)], {}, SHAPE),
    ([(MB + 2, 10, F32)], {}, ALIGN), ([(MB + 1, 10, BF16)], {}, ALIGN), ([(MB, 10, F32, 2 * MB + 2, F32)], {}, ALIGN),
    ([(MB, 10, F32)], dict(max_norm=-1.0), ARG), ([(MB, 10, F32)], dict(max_norm=float("nan")), ARG),
    ([(MB, 10, F32)], dict(norm=None), ARG), ([(MB, 10, F32)], dict(workspace=None), WORKSPACE),
    ([(MB, 10, F32)], dict(ws_bytes=8), WORKSPACE), ([(MB, 10, F32)], dict(norm=9 * MB + 2), ALIGN),
    ([(MB, 1 << 41, F32)], {}, SHAPE),
    ([(MB, 100, F32), (MB, 100, F32)], {}, ARG),                          # the same tensor twice, in place
    ([(MB, 100, F32), (MB + 396, 100, F32)], {}, ARG),
    ([(MB, 100, F32, 3 * MB, F32), (MB, 100, F32, 4 * MB, F32)], {}, CUDA),   # twice, to outputs of their own
    ([(MB, 100, F32, 3 * MB, F32), (2 * MB, 100, F32, 3 * MB + 396, F32)], {}, ARG),
    ([(MB, 100, F32, 2 * MB + 4, F32), (2 * MB, 100, F32, 4 * MB, F32)], {}, ARG),
    ([(MB, 100, BF16, MB, F32)], {}, ARG),                                # another type in place
    ([(MB, 100, F32)], dict(norm=MB + 8), ARG), ([(MB, 100, F32)], dict(workspace=MB + 16), ARG),
]

CHILD = """
import ctypes, json, sys
from mx_block_scaled_gb300 import binding
d = json.load(sys.stdin)
got = [getattr(binding._lib, name)(*args) for name, args in d["calls"]]
def grads(t, more):
    n = len(t)
    p = (ctypes.c_void_p * n)(*[x[0] for x in t]); k = (ctypes.c_int64 * n)(*[x[1] for x in t])
    ty = (ctypes.c_int * n)(*[x[2] for x in t])
    out = any(len(x) > 3 for x in t)
    o = (ctypes.c_void_p * n)(*[x[3] for x in t]) if out else None
    oty = (ctypes.c_int * n)(*[x[4] for x in t]) if out else None
    a = dict(max_norm=1.0, norm=9 << 20, workspace=10 << 20, ws_bytes=1 << 20)
    a.update(more)
    return binding._lib.mxgemm_clip_grads(n, p, k, ty, o, oty, a["max_norm"], a["norm"], a["workspace"], a["ws_bytes"], None)
print(json.dumps([got, [grads(*g) for g in d["grads"]]]))
"""


def _args(name, change):
    args = dict(CALLS[name])
    assert set(change) <= set(args)
    args.update(change)
    return [name, list(args.values())]


@pytest.fixture(scope="module")
def status():
    from mx_block_scaled_gb300 import build
    build.build()
    d = dict(calls=[_args(n, c) for n, c, _ in REFUSED] + [_args(n, c) for n, c in SERVED],
             grads=[[list(t), more] for t, more, _ in GRADS])
    r = subprocess.run([sys.executable, "-c", CHILD], input=json.dumps(d), capture_output=True, text=True, cwd=ROOT,
                       env=dict(os.environ, CUDA_VISIBLE_DEVICES="", PYTHONPATH=ROOT), timeout=300)
    assert r.returncode == 0, r.stderr
    return json.loads(r.stdout.splitlines()[-1])


@pytest.mark.parametrize("i", range(len(REFUSED)), ids=lambda i: f"{REFUSED[i][0][7:]}-{i}")
def test_refused(status, i):
    assert status[0][i] == REFUSED[i][2], REFUSED[i]


@pytest.mark.parametrize("i", range(len(SERVED)), ids=lambda i: f"{SERVED[i][0][7:]}-{i}")
def test_served(status, i):
    assert status[0][len(REFUSED) + i] == CUDA, SERVED[i]    # there is no device


@pytest.mark.parametrize("i", range(len(GRADS)))
def test_lists_of_gradients(status, i):
    assert status[1][i] == GRADS[i][2], GRADS[i]


def test_workspaces():
    from mx_block_scaled_gb300 import binding as lib
    f = lib.mxgemm_embed_backward_workspace_bytes
    assert f(0, 100, 64) == f(9, 0, 64) == f(9, 100, 40) == f(9, 1 << 30, 64) == 0
    assert f(1, 100, 64) == f(64, 100, 64) == 0 and 0 < f(65, 100, 64) <= 1 << 14 and f(1 << 15, 128256, 4096) <= (1 << 19) + (1 << 10) * 2 * 4096 * 4 + 64
    g = lib.mxgemm_qk_norm_rope_backward_workspace_bytes
    assert g(0, 4, 64) == g(4, 0, 64) == g(4, 4, 24) == g(4, 4, 528) == g(1 << 30, 1 << 20, 64) == 0
    assert g(1, 1, 16) == 0 and 0 < g(1000, 40, 128) <= g(1 << 20, 40, 128) <= 1 << 20
    assert lib.mxgemm_grad_workspace_bytes(0) == 0 and 0 < lib.mxgemm_grad_workspace_bytes(1) <= 1 << 13
    assert lib.mxgemm_grad_workspace_bytes(2000) <= 1 << 15


def test_binding_refuses_what_does_not_fit():
    torch = pytest.importorskip("torch")
    from mx_block_scaled_gb300 import binding as lib
    x, ids = torch.zeros(4, 64), torch.zeros(4, dtype=torch.int64)
    for call in (lambda: lib.embed(ids, x), lambda: lib.embed_backward(x, ids, 9),
                 lambda: lib.qk_norm_rope(x.view(4, 1, 64), 1, torch.ones(64)),
                 lambda: lib.qk_norm_rope_backward(x.view(4, 1, 64), None, None, 1),
                 lambda: lib.logprobs(x, ids), lambda: lib.logprobs_backward(x, ids, torch.zeros(4, 2), torch.zeros(4)),
                 lambda: lib.grad_norm([x]), lambda: lib.clip_grads([x], 1.0), lambda: lib.grad_norm(x),
                 lambda: lib.grad_norm([None])):
        with pytest.raises((ValueError, RuntimeError)):
            call()
    assert ctypes.sizeof(ctypes.c_void_p) == 8
