"""Build libmxgemm.so and libmxgemm_debug.so in-tree with nvcc for sm_103a.

Sixteen translation units (host API + relayout/reduce kernels, MXFP8 GEMM,
MXFP4 GEMM, BF16 GEMM, MX quantiser, scale-placement checker, tensor-pipe
probe, and the row operators: their host API, RMS norm, gated activation,
expert routing; the host API of those of a whole model, embedding, norm and
rotation of heads, log probabilities, gradient clipping) are compiled in
parallel and linked into ``mx_block_scaled_gb300/lib/libmxgemm.so``.  The four that hold the GEMM
kernels and their host code are compiled a second time with MXGEMM_DEBUG
(bounds-checked loads and stores, NaN-filled C, synchronous status) and linked
with the others into ``lib/libmxgemm_debug.so``.  The Python module that
marshals the row operators' tensors (rowops_py.cpp, host code against the
installed PyTorch's headers) becomes ``lib/_rowops.so``; without PyTorch it is
left out, and another PyTorch or Python rebuilds it.
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ_DIR = os.path.join(PKG, "_build")
LIB_DIR = os.path.join(PKG, "lib")
LIB_PATH = os.path.join(LIB_DIR, "libmxgemm.so")
DEBUG_LIB_PATH = os.path.join(LIB_DIR, "libmxgemm_debug.so")
ROWOPS_PATH = os.path.join(LIB_DIR, "_rowops.so")

SOURCES = ["mxgemm.cu", "gemm_fp8.cu", "gemm_fp4.cu", "gemm_bf16.cu", "quantize.cu", "placement.cu", "probe.cu",
           "ops.cu", "norm.cu", "glu.cu", "moe.cu", "ops_model.cu", "embed.cu", "heads.cu", "logprobs.cu", "clip.cu"]
MODULE_SOURCE = "rowops_py.cpp"
DEBUG_SOURCES = ["mxgemm.cu", "gemm_fp8.cu", "gemm_fp4.cu", "gemm_bf16.cu"]  # the rest is shared
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "-I" + INCLUDE, "-I" + CSRC]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmxgemm.so")


def _stale(made, sources) -> bool:
    sources = [*sources, os.path.join(INCLUDE, "mxgemm.h"), os.path.abspath(__file__)]
    return not all(os.path.exists(p) for p in made) or \
        max(os.path.getmtime(f) for f in sources) > min(os.path.getmtime(p) for p in made)


def _libraries_stale() -> bool:
    return _stale((LIB_PATH, DEBUG_LIB_PATH),
                  [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != MODULE_SOURCE])


def _torch_dir():
    """The installed PyTorch's folder (found, not imported), or None."""
    spec = importlib.util.find_spec("torch")
    return list(spec.submodule_search_locations)[0] if spec and spec.submodule_search_locations else None


def _rowops_key(torch_dir: str) -> str:
    """The Python and the PyTorch that _rowops.so is compiled against: their layouts are part of its code."""
    with open(os.path.join(torch_dir, "version.py")) as f:
        return f"{sysconfig.get_config_var('SOABI')}\n{torch_dir}\n{f.read()}"


def _key_path() -> str:
    return os.path.join(OBJ_DIR, "rowops.key")


def _rowops_stale() -> bool:
    torch_dir = _torch_dir()
    if torch_dir is None:
        return False
    key = _key_path()
    if _stale((ROWOPS_PATH, key), [os.path.join(CSRC, MODULE_SOURCE)]):
        return True
    with open(key) as f:
        return f.read() != _rowops_key(torch_dir)


def needs_build() -> bool:
    return _libraries_stale() or _rowops_stale()


def _link(nvcc: str, objs, path: str) -> None:
    tmp = path + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of {os.path.basename(path)} failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)


def _build_rowops(nvcc: str) -> None:
    """rowops_py.cpp -> _rowops.so, against the installed PyTorch; nothing where there is none."""
    torch_dir = _torch_dir()
    if torch_dir is None:
        return
    torch_lib = os.path.join(torch_dir, "lib")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    include = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(torch_dir, "include"),
               os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include")]
    tmp = ROWOPS_PATH + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", *(f"-I{d}" for d in include),
           os.path.join(CSRC, MODULE_SOURCE), "-o", tmp, "-L" + torch_lib, "-ltorch_python", "-ltorch_cpu", "-lc10",
           "-lc10_cuda", "-Wl,-rpath," + torch_lib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {MODULE_SOURCE}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, ROWOPS_PATH)
    with open(_key_path(), "w") as f:
        f.write(_rowops_key(torch_dir))


def _build_libraries(nvcc: str, verbose: bool) -> None:
    def compile_one(job):
        src, debug = job
        obj = os.path.join(OBJ_DIR, os.path.splitext(src)[0] + ("_debug.o" if debug else ".o"))
        cmd = [nvcc, *ARCH, *FLAGS, *(["-DMXGEMM_DEBUG"] if debug else []), "-c", os.path.join(CSRC, src),
               "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}{' (debug)' if debug else ''}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
        return obj

    jobs = [(src, False) for src in SOURCES] + [(src, True) for src in DEBUG_SOURCES]
    with ThreadPoolExecutor(max_workers=len(jobs)) as ex:
        objs = list(ex.map(compile_one, jobs))
    release = objs[:len(SOURCES)]
    debug = objs[len(SOURCES):] + [o for (src, _), o in zip(jobs, release) if src not in DEBUG_SOURCES]
    _link(nvcc, release, LIB_PATH)
    _link(nvcc, debug, DEBUG_LIB_PATH)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libmxgemm.so and libmxgemm_debug.so, and _rowops.so, where
    they are missing or stale; return the release library's path."""
    libraries, rowops = force or _libraries_stale(), force or _rowops_stale()
    if not libraries and not rowops:
        return LIB_PATH
    nvcc = _nvcc()
    os.makedirs(OBJ_DIR, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    with ThreadPoolExecutor(max_workers=1) as ex:
        module = ex.submit(_build_rowops, nvcc) if rowops else None
        if libraries:
            _build_libraries(nvcc, verbose)
        if module:
            module.result()
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
