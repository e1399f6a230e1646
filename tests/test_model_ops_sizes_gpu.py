"""Both sides of the sizes at which the model's row operators take another table or
another block, against the 64-bit definitions."""
import numpy as np
import pytest

import test_clip_gpu as clip
import test_logprobs_gpu as logprobs
from gpu_util import lib

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    lib()


@pytest.mark.parametrize("form", ["in place", "f32", "bf16"])
@pytest.mark.parametrize("n", [31, 32, 33, 128, 129, 320, 321, 448, 640, 641, 1024, 1025, 2048, 2049])
def test_tables_of_gradients(n, form):
    """A launch's table holds up to 32, 128, 320, 640 or 1024 tensors."""
    rng = np.random.default_rng(n)
    shapes = [(int(s),) for s in rng.integers(0, 40, n)]
    shapes[0], shapes[n // 2], shapes[-1] = (4097,), (20000,), (4096,)     # more chunks than one, at both ends and inside
    dtypes = [["f32", "bf16"][int(i)] for i in rng.integers(0, 2, n)]
    grads, g64 = clip._grads(rng, shapes, dtypes)
    clip._check(grads, g64, 0.1, None if form == "in place" else [form] * n)


def test_norm_and_limit_infinite():
    """The formula as it stands: infinity over infinity."""
    g = [torch.ones(100, device="cuda"), torch.full((9,), float("inf"), device="cuda")]
    norm, out = lib().clip_grads(g, float("inf"), out=[torch.empty_like(x) for x in g])
    assert norm.item() == float("inf") and all(torch.isnan(o).all() for o in out)
    norm, out = lib().clip_grads(g[:1], float("inf"))
    assert norm.item() == 10.0 and (out[0] == 1).all()


@pytest.mark.parametrize("top", [0, 20, 32])
@pytest.mark.parametrize("rows,V,dtype", [(4870, 1200, "bf16"), (4870, 5000, "bf16"), (4870, 2501, "f32"),      # 32 threads
                                          (2440, 17000, "bf16"), (2500, 5000, "bf16"), (2440, 8201, "f32"),     # 64
                                          (1300, 20000, "bf16"), (1250, 33000, "bf16"), (1300, 9001, "f32")])   # 128
def test_blocks_of_many_short_rows(rows, V, dtype, top):
    """More rows than fit at once, of at most sixteen chunks a thread: blocks of 32, 64 and 128 threads."""
    rng = np.random.default_rng([rows, V, top])
    x, x64 = logprobs._logits(rng, rows, V, dtype, "steps" if top == 32 else "model")
    logprobs._check(x, x64, rng, top=top)
