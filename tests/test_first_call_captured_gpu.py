"""A process whose first call of an operator is captured into a graph: its kernels are
loaded and prepared there, and the replay gives what an ordinary call gives."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import sys, torch
from mx_block_scaled_gb300 import binding as mx
gen = torch.Generator(device="cuda"); gen.manual_seed(0)
r = lambda *s: torch.randn(s, generator=gen, device="cuda")
x, w, ids = r(1500, 256), r(256), torch.randint(0, 900, (1500,), generator=gen, device="cuda")
many = torch.randint(0, 900, (3000,), generator=gen, device="cuda")
h, hw, dm = r(700, 6, 64), r(64), r(3000, 256)
rstd, hr, st = r(1500).abs(), r(700, 6).abs(), torch.zeros(1500, 2, device="cuda")
a = torch.arange(1500, device="cuda") % 256
calls = dict(
    norm=lambda: mx.rmsnorm_backward(x, x, rstd, w),
    embed=lambda: (mx.embed_backward(x, ids, 900), mx.embed_backward(dm, many, 900)),
    heads=lambda: mx.qk_norm_rope(h, 4, hw, hw)[:2] + mx.qk_norm_rope_backward(h, h, hr, 4, hw, hw),
    logprobs=lambda: mx.logprobs(x, a, top=5, entropy=True) + (mx.logprobs_backward(x, a, st, rstd),),
    clip=lambda: (mx.grad_norm([x, w]), *mx.clip_grads([x, w], 0.5, out=[torch.empty_like(x), torch.empty_like(w)])[1]))
call = calls[sys.argv[1]]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = call()
g.replay()
want = call()
torch.cuda.synchronize()
assert len(got) == len(want) and all(torch.equal(i, j) for i, j in zip(got, want))
print("same")
"""


@pytest.mark.parametrize("name", ["norm", "embed", "heads", "logprobs", "clip"])
def test_first_call(name):
    from gpu_util import lib
    lib()
    p = subprocess.run([sys.executable, "-c", CHILD, name], capture_output=True, text=True, cwd=ROOT,
                       env=dict(os.environ, PYTHONPATH=ROOT), timeout=300)
    assert p.returncode == 0 and p.stdout.strip() == "same", p.stderr[-2000:]
