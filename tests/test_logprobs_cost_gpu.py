"""The most probable tokens are found beside one pass over the logits: they cost a part of
it, whatever the row's length and the block's size, not a pass each."""
import pytest

from gpu_util import lib

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    lib()


def _us(call):
    call()
    best = float("inf")
    for _ in range(3):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda.synchronize()
        a.record()
        for _ in range(3):
            call()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) / 3 * 1e3)
    return best


@pytest.mark.parametrize("rows,V,dtype,top", [(1300, 200_000, torch.float32, 20), (1300, 262_144, torch.float32, 32),
                                              (1300, 400_001, torch.bfloat16, 20), (320, 1_000_003, torch.float32, 32),
                                              (320, 2_000_000, torch.bfloat16, 20), (200, 3_000_017, torch.bfloat16, 32)])
def test_long_rows(rows, V, dtype, top):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(rows)
    x = torch.empty(rows, V, dtype=dtype, device="cuda").normal_(0, 2.5, generator=gen)
    got = lib().logprobs(x, top=top)
    want = torch.topk(x, top, sorted=True).values
    assert torch.equal(x.gather(1, got.top_ids), want)
    # equal ones by id, so that no id comes twice
    ids = got.top_ids
    assert ((want[:, 1:] < want[:, :-1]) | (ids[:, 1:] > ids[:, :-1])).all()
    plain, most = _us(lambda: lib().logprobs(x)), _us(lambda: lib().logprobs(x, top=top))
    # a pass a token is more than twenty of them; these are at the most one more
    assert most < 4 * plain, (plain, most)
