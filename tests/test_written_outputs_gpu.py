"""Outputs that share their memory copy-on-write with another tensor: a call writes into a
copy of its own, and the other tensor keeps its values."""
import pytest

from gpu_util import lib

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    lib()


def _rand(*shape, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda")


T, H, D, V = 5, 3, 32, 100


def _turn(x, y):
    return lib().qk_norm_rope(x, 2, torch.ones(D, device="cuda"), torch.ones(D, device="cuda"), y=y).y


def _turn_back(dy, dx):
    x, w = _rand(T, H, D, seed=1), torch.ones(D, device="cuda")
    return lib().qk_norm_rope_backward(dy, x, torch.ones(T, H, device="cuda"), 2, w, w, dx=dx)[0]


def _dlogits(x, d):
    stats = lib().logprobs(_rand(T, V)).stats
    t = torch.arange(T, device="cuda")
    return lib().logprobs_backward(x, t, stats, torch.ones(T, device="cuda"), dlogits=d)


def _clip(x, out):
    return lib().clip_grads([x], 0.5, out=None if out is x else [out])[1][0]


CALLS = dict(turn=(_turn, (T, H, D)), turn_back=(_turn_back, (T, H, D)), dlogits=(_dlogits, (T, V)), clip=(_clip, (T, V)),
             embed=(lambda x, out: lib().embed(torch.arange(T, device="cuda"), x, 2.0, out=out), (T, 64)))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("name", sorted(CALLS))
def test_shared_memory_keeps_its_values(name, in_place):
    call, shape = CALLS[name]
    if in_place and name == "embed":
        pytest.skip("no in-place form")
    x = _rand(*shape)
    want = call(x, torch.empty_like(x)).clone()
    other = x.clone() if in_place else torch.full_like(x, 7.0)
    before = other.clone()
    out = torch._lazy_clone(other)
    got = call(out if in_place else x, out)
    assert got is out and torch.equal(got, want)
    assert torch.equal(other, before)


def test_what_is_only_read_stays_shared():
    other = _rand(T, V)
    shared = torch._lazy_clone(other)
    b = lib()
    b.grad_norm([shared])
    b.logprobs(shared)
    b.clip_grads([shared], 0.5, out=[torch.empty_like(shared)])
    assert torch._C._is_cow_tensor(shared) and torch._C._is_cow_tensor(other)
