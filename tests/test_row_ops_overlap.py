"""Outputs of the row operators over their inputs or over each other: refused, apart from
the in-place forms that the header names.  The calls run in a process that sees no
device, so that one which passes the checks ends there (no GPU needed, none used)."""
import json
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ARG, CUDA = -1, -6
MB = 1 << 20

# every pointer of a good call in a megabyte of its own
CALLS = dict(
    mxgemm_rmsnorm=dict(in_dtype=2, x=1 * MB, x_stride=256, residual=2 * MB, residual_stride=256, weight=3 * MB,
                        weight_dtype=1, eps=1e-5, rows=4, K=256, h=4 * MB, y=5 * MB, fmt=1, codes=6 * MB,
                        scales=7 * MB, rstd=8 * MB, flags=0, stream=None),
    mxgemm_rmsnorm_backward=dict(in_dtype=1, dy=1 * MB, dy_stride=256, h=2 * MB, h_stride=256, rstd=3 * MB,
                                 weight=4 * MB, weight_dtype=1, dh=5 * MB, dh_stride=256, rows=4, K=256, dx=6 * MB,
                                 dweight=7 * MB, workspace=None, ws_bytes=0, stream=None),
    mxgemm_glu=dict(act=1, in_dtype=2, gate=1 * MB, up=2 * MB, stride=256, rows=4, F=256, y=3 * MB, fmt=2,
                    codes=4 * MB, scales=5 * MB, flags=1, kept_codes=6 * MB, kept_scales=7 * MB, stream=None),
    mxgemm_glu_backward=dict(act=2, in_dtype=2, dy=1 * MB, dy_stride=256, gate=None, up=None, stride=0,
                             kept_codes=2 * MB, kept_scales=3 * MB, rows=4, F=256, dgu=4 * MB, fmt=1, codes=5 * MB,
                             scales=6 * MB, flags=1, a=7 * MB, stream=None),
    mxgemm_moe_sort=dict(expert_ids=1 * MB, id_bytes=8, slots=16, groups=4, offsets=2 * MB, row_of_slot=3 * MB,
                         slot_of_row=4 * MB, workspace=None, ws_bytes=0, stream=None),
    mxgemm_moe_dispatch=dict(in_dtype=2, x=1 * MB, x_stride=256, tokens=4, topk=2, K=256, row_of_slot=2 * MB, fmt=1,
                             rows=3 * MB, scales=4 * MB, stream=None),
    mxgemm_moe_combine=dict(in_dtype=2, y=1 * MB, y_stride=256, tokens=4, topk=2, N=256, row_of_slot=2 * MB,
                            weights=3 * MB, add=4 * MB, add_stride=256, out=5 * MB, stream=None),
    mxgemm_moe_combine_backward=dict(in_dtype=2, dout=1 * MB, dout_stride=256, y=2 * MB, y_stride=256, tokens=4,
                                     topk=2, N=256, row_of_slot=3 * MB, weights=4 * MB, dy=5 * MB, dweights=6 * MB,
                                     stream=None),
)
WITH_WORKSPACE = dict(
    mxgemm_rmsnorm_backward=dict(rows=1500, dy=16 * MB, h=32 * MB, dx=48 * MB, dh=None, workspace=64 * MB,
                                 ws_bytes=8 * MB),
    mxgemm_moe_sort=dict(slots=1 << 18, expert_ids=16 * MB, row_of_slot=32 * MB, slot_of_row=48 * MB,
                         workspace=64 * MB, ws_bytes=MB),
)
FROM_INPUTS = dict(kept_codes=None, kept_scales=None, gate=8 * MB, up=9 * MB, stride=256)

OVERLAPS = [  # (entry, output, the input or output it touches, offset from that one's start, other arguments)
    ("mxgemm_rmsnorm", "scales", "x", 2032, {}), ("mxgemm_rmsnorm", "scales", "residual", 0, {}),
    ("mxgemm_rmsnorm", "rstd", "x", 2044, {}), ("mxgemm_rmsnorm", "rstd", "weight", 1020, {}),
    ("mxgemm_rmsnorm", "h", "weight", 992, {}), ("mxgemm_rmsnorm", "y", "weight", 0, {}),
    ("mxgemm_rmsnorm", "codes", "weight", 1008, {}), ("mxgemm_rmsnorm", "scales", "weight", 0, {}),
    ("mxgemm_rmsnorm", "h", "y", 0, {}), ("mxgemm_rmsnorm", "rstd", "scales", 28, {}),
    ("mxgemm_rmsnorm", "codes", "y", 2032, {}), ("mxgemm_rmsnorm", "scales", "codes", 1008, {}),
    # the tile layout's scales run to row 128
    ("mxgemm_rmsnorm", "rstd", "scales", 1020, dict(flags=1)),
    ("mxgemm_rmsnorm_backward", "dx", "rstd", 0, {}), ("mxgemm_rmsnorm_backward", "dx", "weight", 992, {}),
    ("mxgemm_rmsnorm_backward", "dweight", "dy", 4064, {}), ("mxgemm_rmsnorm_backward", "dweight", "h", 0, {}),
    ("mxgemm_rmsnorm_backward", "dweight", "dh", 0, {}), ("mxgemm_rmsnorm_backward", "dweight", "weight", 0, {}),
    ("mxgemm_rmsnorm_backward", "dweight", "rstd", 0, {}), ("mxgemm_rmsnorm_backward", "dweight", "dx", 4064, {}),
    *(("mxgemm_rmsnorm_backward", "workspace", n, 0, WITH_WORKSPACE["mxgemm_rmsnorm_backward"])
      for n in ("dy", "h", "rstd", "weight", "dx", "dweight")),
    ("mxgemm_glu", "scales", "gate", 0, {}), ("mxgemm_glu", "scales", "up", 2032, {}),
    ("mxgemm_glu", "kept_scales", "gate", 2032, {}), ("mxgemm_glu", "kept_scales", "up", 0, {}),
    ("mxgemm_glu", "kept_codes", "codes", 496, {}), ("mxgemm_glu", "kept_scales", "scales", 1008, {}),
    ("mxgemm_glu", "y", "kept_codes", 2016, {}),
    ("mxgemm_glu_backward", "dgu", "kept_codes", 0, {}), ("mxgemm_glu_backward", "a", "kept_codes", 0, {}),
    ("mxgemm_glu_backward", "a", "kept_codes", 2016, {}), ("mxgemm_glu_backward", "codes", "kept_codes", 0, {}),
    ("mxgemm_glu_backward", "scales", "kept_codes", 2032, {}), ("mxgemm_glu_backward", "dgu", "kept_scales", 32, {}),
    ("mxgemm_glu_backward", "a", "kept_scales", 0, {}), ("mxgemm_glu_backward", "codes", "kept_scales", 48, {}),
    ("mxgemm_glu_backward", "scales", "kept_scales", 0, {}), ("mxgemm_glu_backward", "scales", "dy", 0, {}),
    ("mxgemm_glu_backward", "scales", "gate", 0, FROM_INPUTS), ("mxgemm_glu_backward", "scales", "up", 2032, FROM_INPUTS),
    ("mxgemm_glu_backward", "a", "dgu", 4064, {}), ("mxgemm_glu_backward", "codes", "a", 0, {}),
    # one row: a over gate, and dgu over both halves, each alone is fine
    ("mxgemm_glu_backward", "a", "gate", 0, dict(FROM_INPUTS, rows=1, up=8 * MB + 512, dgu=8 * MB)),
    ("mxgemm_moe_sort", "row_of_slot", "offsets", 36, {}), ("mxgemm_moe_sort", "slot_of_row", "row_of_slot", 60, {}),
    *(("mxgemm_moe_sort", "workspace", n, 0, WITH_WORKSPACE["mxgemm_moe_sort"])
      for n in ("expert_ids", "offsets", "row_of_slot", "slot_of_row")),
    ("mxgemm_moe_dispatch", "rows", "row_of_slot", 16, {}), ("mxgemm_moe_dispatch", "scales", "row_of_slot", 16, {}),
    ("mxgemm_moe_dispatch", "scales", "x", 0, {}), ("mxgemm_moe_dispatch", "scales", "rows", 2032, {}),
    ("mxgemm_moe_combine", "out", "row_of_slot", 0, {}), ("mxgemm_moe_combine", "out", "weights", 0, {}),
    ("mxgemm_moe_combine_backward", "dy", "row_of_slot", 0, {}), ("mxgemm_moe_combine_backward", "dy", "weights", 0, {}),
    ("mxgemm_moe_combine_backward", "dweights", "row_of_slot", 28, {}),
    ("mxgemm_moe_combine_backward", "dweights", "weights", 4, {}),
    ("mxgemm_moe_combine_backward", "dweights", "dout", 0, {}), ("mxgemm_moe_combine_backward", "dweights", "y", 4092, {}),
    ("mxgemm_moe_combine_backward", "dweights", "dy", 4092, {}),
]
SERVED = [(name, {}) for name in CALLS] + [
    *WITH_WORKSPACE.items(),
    ("mxgemm_rmsnorm", dict(h=2 * MB, y=1 * MB)), ("mxgemm_rmsnorm", dict(h=1 * MB, y=2 * MB)),
    ("mxgemm_rmsnorm", dict(residual=1 * MB, h=1 * MB)),
    ("mxgemm_rmsnorm", dict(codes=7 * MB - 1024, rstd=7 * MB + 32)),   # side by side, nothing shared
    ("mxgemm_rmsnorm_backward", dict(dx=5 * MB)),
    ("mxgemm_rmsnorm_backward", dict(workspace=7 * MB, ws_bytes=64)),  # few rows: it is not written
    ("mxgemm_glu", dict(y=1 * MB)), ("mxgemm_glu", dict(y=2 * MB)), ("mxgemm_glu", dict(up=1 * MB, y=1 * MB)),
    ("mxgemm_glu_backward", dict(a=1 * MB)), ("mxgemm_glu_backward", FROM_INPUTS),
    ("mxgemm_glu_backward", dict(FROM_INPUTS, a=8 * MB)), ("mxgemm_glu_backward", dict(FROM_INPUTS, a=9 * MB)),
    ("mxgemm_glu_backward", dict(FROM_INPUTS, up=8 * MB + 512, stride=512, dgu=8 * MB, a=1 * MB)),
    ("mxgemm_glu_backward", dict(FROM_INPUTS, rows=1, up=8 * MB + 512, a=8 * MB)),
    ("mxgemm_moe_combine", dict(out=4 * MB)),
    ("mxgemm_moe_combine_backward", dict(dy=2 * MB)), ("mxgemm_moe_combine_backward", dict(dweights=4 * MB)),
]

CHILD = """
import json, sys
from mx_block_scaled_gb300 import binding
print(json.dumps([getattr(binding._lib, name)(*args) for name, args in json.load(sys.stdin)]))
"""


def _args(name, change):
    args = dict(CALLS[name])
    assert set(change) <= set(args)
    args.update(change)
    return [name, list(args.values())]


@pytest.fixture(scope="module")
def status():
    """Statuses of the calls, in a process to which no device is visible."""
    from mx_block_scaled_gb300 import build
    build.build()
    calls = []
    for name, out, other, at, change in OVERLAPS:
        c = dict(CALLS[name], **change)
        calls.append(_args(name, dict(change, **{out: c[other] + at})))
    calls += [_args(name, change) for name, change in SERVED]
    r = subprocess.run([sys.executable, "-c", CHILD], input=json.dumps(calls), capture_output=True, text=True, cwd=ROOT,
                       env=dict(os.environ, CUDA_VISIBLE_DEVICES="", PYTHONPATH=ROOT), timeout=300)
    assert r.returncode == 0, r.stderr
    return json.loads(r.stdout.splitlines()[-1])


@pytest.mark.parametrize("i", range(len(OVERLAPS)), ids=lambda i: "{}-{}-over-{}+{}".format(*OVERLAPS[i]))
def test_overlap_is_refused(status, i):
    assert status[i] == ARG


@pytest.mark.parametrize("i", range(len(SERVED)), ids=lambda i: f"{SERVED[i][0]}-{i}")
def test_apart_and_named_in_place_forms_pass_the_checks(status, i):
    assert status[len(OVERLAPS) + i] == CUDA     # there is no device
