"""Log probabilities at scales and logits whose products pass FP32's largest value: what
has a probability of zero adds nothing."""
import numpy as np
import pytest

import model_ops_ref as ref
from gpu_util import lib

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    lib()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scale,level", [(2.3e38, 4096.0), (1e30, 1e12), (1e8, 3e33), (1e6, 3e38), (1e4, 1.0)])
@pytest.mark.parametrize("V", [20, 1000, 40000])
def test_only_the_largest_count(V, scale, level, dtype):
    """k equal largest values, the others a 64th or more of the level below them: p is 1/k and 0."""
    b, rows, k = lib(), 3, 4
    rng = np.random.default_rng(V)
    x64 = level * (1 - rng.integers(1, 60, (rows, V)) / 64)
    best = np.sort(np.stack([rng.permutation(V)[:k] for _ in range(rows)]), 1)
    np.put_along_axis(x64, best, level, 1)
    x = torch.from_numpy(x64).cuda().to(dtype)
    other = np.array([next(v for v in range(V) if v not in best[r]) for r in range(rows)])
    for at, lp in ((best[:, 2], -np.log(k)), (other, -np.inf)):
        t = torch.from_numpy(at).cuda()
        got = b.logprobs(x, t, scale=scale, top=k, entropy=True)
        # ln of a sum of k exact ones: rounded by logf (one unit) and where it is stored
        for v, w in ((got.logprob, lp), (got.entropy, np.log(k)), (got.stats[:, 1], np.log(k))):
            v = v.double().cpu().numpy()
            if w == -np.inf and scale * level / 64 < 1e38:           # a number that FP32 has
                assert (v < -100).all()
            else:
                assert (v == w).all() or (np.abs(v - w) <= 4 * ref.U * abs(w)).all(), (v, w)
        assert np.array_equal(got.top_ids.cpu().numpy(), best)
        # the gradient's factor scale * g * (1 + entropy) has to be a number that FP32 has: 2.3e38 * (1 + ln 4) is 5.5e38
        one = 1.0 if scale * (1 + np.log(k)) < 3.4e38 else 2.0 ** -6
        g = torch.full((rows,), one, device="cuda")
        for dentropy in (None, g):
            d = b.logprobs_backward(x, t, got.stats, g, entropy=got.entropy, dentropy=dentropy, scale=scale)
            d = d.double().cpu().numpy()
            assert np.isfinite(d).all()
            rest = np.ones((rows, V), bool)
            np.put_along_axis(rest, best, False, 1)
            np.put_along_axis(rest, at[:, None], False, 1)
            assert (d[rest] == 0).all()
            if lp == -np.inf:
                s = np.float64(np.float32(scale)) * one              # its own term alone, rounded to the type
                assert (np.abs(np.take_along_axis(d, at[:, None], 1) - s) <= torch.finfo(dtype).eps / 2 * s).all()
