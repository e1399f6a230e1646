"""Arguments of the model's row operators at the ends of their ranges: refused, or served
in full.  The calls run in a process that sees no device (no GPU needed, none used)."""
import json
import os
import subprocess
import sys

import pytest

from test_model_ops_abi import ARG, CHILD, CUDA, ROOT, SHAPE, _args

HUGE = 3.0e38           # times log2(e) past FP32's largest value

CASES = [
    # heads whose token and head steps are alike, of so many tokens that their product passes 64 bits
    *(("mxgemm_qk_norm_rope", dict(tokens=1 << 24, q_heads=1, k_heads=1, **{f"{t}_token": s, f"{t}_head": s}), SHAPE)
      for t in "xy" for s in (1 << 40, 1 << 39)),
    ("mxgemm_qk_norm_rope_backward", dict(tokens=1 << 24, q_heads=1, k_heads=1, dy_token=1 << 40, dy_head=1 << 40), SHAPE),
    ("mxgemm_qk_norm_rope_backward", dict(tokens=1 << 24, q_heads=1, k_heads=1, dx_token=1 << 40, dx_head=1 << 40), SHAPE),
    ("mxgemm_qk_norm_rope", dict(tokens=1 << 20, x_token=1 << 20, x_head=(1 << 40) - (1 << 20)), SHAPE),      # a token too many
    # scales whose exponents FP32 cannot hold
    ("mxgemm_logprobs", dict(scale=HUGE), ARG), ("mxgemm_logprobs_backward", dict(scale=HUGE), ARG),
    ("mxgemm_logprobs", dict(scale=2.3e38), CUDA), ("mxgemm_logprobs_backward", dict(scale=2.3e38), CUDA),
    ("mxgemm_logprobs", dict(scale=1e-38), CUDA), ("mxgemm_logprobs_backward", dict(scale=1e-38), CUDA),
]


@pytest.fixture(scope="module")
def status():
    from mx_block_scaled_gb300 import build
    build.build()
    r = subprocess.run([sys.executable, "-c", CHILD], text=True, cwd=ROOT, timeout=300, capture_output=True,
                       input=json.dumps(dict(calls=[_args(n, c) for n, c, _ in CASES], grads=[])),
                       env=dict(os.environ, CUDA_VISIBLE_DEVICES="", PYTHONPATH=ROOT))
    assert r.returncode == 0, r.stderr
    return json.loads(r.stdout.splitlines()[-1])[0]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_limits(status, i):
    assert status[i] == CASES[i][2], CASES[i]
