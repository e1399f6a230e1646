"""Preparing the device for one family of row operators says nothing about the others.
The host code of the entry points runs here beside a fake of the CUDA runtime and of the
kernels, in which a family's preparation fails (no GPU needed, none used)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, CUDA = 0, -6
FAMILIES = ("norm", "embed", "heads")

FAKE = """
#include "ops.h"
namespace { int g_fails, g_prepared[3]; cudaError_t prepare(int f)
{ ++g_prepared[f]; return g_fails >> f & 1 ? cudaErrorUnknown : cudaSuccess; } }
extern "C" {
void fake_fails(int mask) { g_fails = mask; }
int fake_prepared(int f) { return g_prepared[f]; }
cudaError_t cudaGetDevice(int *d) { *d = 0; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr a, int)
{ *v = a == cudaDevAttrComputeCapabilityMajor ? 10 : a == cudaDevAttrComputeCapabilityMinor ? 3 : 152; return cudaSuccess; }
void **__cudaRegisterFatBinary(void *) { return nullptr; }
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
}
namespace mxg {
cudaError_t prepare_norm() { return prepare(0); }
cudaError_t prepare_embed() { return prepare(1); }
cudaError_t prepare_heads() { return prepare(2); }
cudaError_t launch_rmsnorm(const NormParams &, int, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_rmsnorm_backward(const NormBackParams &, int, int, int, cudaStream_t) { return cudaSuccess; }
int64_t norm_back_blocks(int64_t, int64_t) { return 0; }
cudaError_t launch_glu(const GluParams &, int, int, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_glu_backward(const GluBackParams &, int, int, int, cudaStream_t) { return cudaSuccess; }
size_t sort_workspace(int64_t, int64_t) { return 0; }
cudaError_t launch_moe_sort(const void *, bool, int64_t, int, int64_t *, int32_t *, int32_t *, int32_t *, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_moe_dispatch(const DispatchParams &, int, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_moe_combine(const CombineParams &, int, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_moe_combine_backward(const CombineBackParams &, int, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_embed(const EmbedParams &, int, int, int, cudaStream_t) { return cudaSuccess; }
EmbedWorkspace embed_workspace(int64_t, int64_t) { return {}; }
cudaError_t launch_embed_backward(EmbedBackParams, const void *, bool, char *, int, int, cudaStream_t) { return cudaSuccess; }
int64_t heads_back_blocks(int64_t, int, int) { return 0; }
cudaError_t launch_heads(const HeadsParams &, int, int, bool, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_heads_backward(const HeadsBackParams &, int, int, bool, int, cudaStream_t) { return cudaSuccess; }
bool logprobs_fits(int64_t, int64_t) { return true; }
cudaError_t launch_logprobs(const LogprobsParams &, int, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_logprobs_backward(const LogprobsBackParams &, int, cudaStream_t) { return cudaSuccess; }
size_t grad_workspace(int64_t) { return 0; }
bool grads_fit(const GradTensor *, int64_t) { return true; }
cudaError_t launch_grad_norm(const GradTensor *, int64_t, double *, float *, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_clip_grads(const GradTensor *, int64_t, double *, float, float *, int, cudaStream_t) { return cudaSuccess; }
}
"""

# calls in a process of their own: a family's state is kept for the process
CHILD = """
import ctypes, sys
sys.path.insert(0, "tests")
from mx_block_scaled_gb300 import binding
import test_model_ops_abi as model, test_row_ops_overlap as rows
lib = ctypes.CDLL(sys.argv[1])
def call(name):
    table = model.CALLS if name in model.CALLS else rows.CALLS
    f = getattr(lib, name)
    f.restype, f.argtypes = next((r, a) for n, r, a in binding.SIGNATURES if n == name)
    return f(*table[name].values())
lib.fake_fails(int(sys.argv[2]))
first = [call(n) for n in sys.argv[3:]]
lib.fake_fails(0)
again = [call(n) for n in sys.argv[3:]]
print(*first, *again, *[lib.fake_prepared(f) for f in range(3)])
"""
CALLS = dict(norm=["mxgemm_rmsnorm_backward"], embed=["mxgemm_embed_backward"],
             heads=["mxgemm_qk_norm_rope", "mxgemm_qk_norm_rope_backward"],
             none=["mxgemm_rmsnorm", "mxgemm_glu", "mxgemm_glu_backward", "mxgemm_moe_sort", "mxgemm_moe_dispatch",
                   "mxgemm_moe_combine", "mxgemm_moe_combine_backward", "mxgemm_embed", "mxgemm_logprobs",
                   "mxgemm_logprobs_backward"])


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    from mx_block_scaled_gb300 import build
    build.build()
    d = tmp_path_factory.mktemp("fake")
    (d / "fake.cpp").write_text(FAKE)
    objects = []
    for name in ("ops", "ops_model"):
        objects.append(os.path.join(build.OBJ_DIR, name + ".o"))
        if not os.path.exists(objects[-1]):          # libraries without the objects that they were linked from
            objects[-1] = str(d / (name + ".o"))
            subprocess.run([build._nvcc(), *build.ARCH, *build.FLAGS, "-c", os.path.join(build.CSRC, name + ".cu"), "-o",
                            objects[-1]], check=True)
    cuda = os.path.dirname(os.path.dirname(build._nvcc()))
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-Wl,--no-undefined", "-o", str(d / "fake.so"),
                    str(d / "fake.cpp"), *objects, f"-I{build.CSRC}", f"-I{build.INCLUDE}",
                    f"-I{cuda}/include"], check=True)
    return str(d / "fake.so")


def _run(fake, fails, calls):
    r = subprocess.run([sys.executable, "-c", CHILD, fake, str(fails), *calls], capture_output=True, text=True, cwd=ROOT,
                       env=dict(os.environ, PYTHONPATH=ROOT))
    assert r.returncode == 0, r.stderr
    got = [int(v) for v in r.stdout.split()]
    return got[:len(calls)], got[len(calls):2 * len(calls)], got[2 * len(calls):]


@pytest.mark.parametrize("family", FAMILIES)
def test_a_failure_is_its_family_s(fake, family):
    """The family's calls fail, and are served once its preparation does not fail any more."""
    calls = [n for f in CALLS for n in CALLS[f]]
    first, again, prepared = _run(fake, 1 << FAMILIES.index(family), calls)
    assert first == [CUDA if n in CALLS[family] else OK for n in calls]
    assert again == [OK] * len(calls)
    # once, or once for every refused call and once more
    assert prepared == [len(CALLS[f]) + 1 if f == family else 1 for f in FAMILIES]


@pytest.mark.parametrize("family", (*FAMILIES, "none"))
def test_a_call_prepares_its_family_alone(fake, family):
    first, again, prepared = _run(fake, 0, CALLS[family])
    assert set(first + again) == {OK}
    assert prepared == [int(f == family) for f in FAMILIES]
