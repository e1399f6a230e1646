"""What build() compiles and when, with the compilers replaced by a recorder (no compiler, no GPU)."""
import importlib.util
import os
import subprocess
import sysconfig
import types

import pytest

from mx_block_scaled_gb300 import build as b


@pytest.fixture
def tools(monkeypatch, tmp_path):
    """An empty output tree; compilers that write their -o file and note their command."""
    for name, path in dict(OBJ_DIR="obj", LIB_DIR="lib", LIB_PATH="lib/libmxgemm.so",
                           DEBUG_LIB_PATH="lib/libmxgemm_debug.so", ROWOPS_PATH="lib/_rowops.so").items():
        monkeypatch.setattr(b, name, str(tmp_path / path))
    nvcc = tmp_path / "nvcc"
    nvcc.write_text("")
    monkeypatch.setattr(b, "_nvcc", lambda: str(nvcc))

    class Tools:
        commands, failing = [], ()

        def ran(self, what):
            return [c for c in self.commands if any(a.endswith(what) for a in c)]

    t = Tools()
    t.commands = []

    def run(cmd, **kw):
        t.commands.append(cmd)
        if os.path.basename(cmd[0]) in t.failing:
            return subprocess.CompletedProcess(cmd, 1, "", "refused")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("made")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(subprocess, "run", run)
    return t


def _without_torch(monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))


def test_builds_all_once(tools):
    b.build()
    assert all(os.path.exists(p) for p in (b.LIB_PATH, b.DEBUG_LIB_PATH, b.ROWOPS_PATH))
    assert not b.needs_build()
    n = len(tools.commands)
    b.build()
    assert len(tools.commands) == n


def test_libraries_build_without_pytorch(tools, monkeypatch):
    _without_torch(monkeypatch)
    assert b.build() == b.LIB_PATH
    assert os.path.exists(b.LIB_PATH) and os.path.exists(b.DEBUG_LIB_PATH) and not os.path.exists(b.ROWOPS_PATH)
    assert not tools.ran("rowops_py.cpp") and not b.needs_build()


def test_module_is_added_when_pytorch_is(tools, monkeypatch):
    with monkeypatch.context() as m:
        _without_torch(m)
        b.build()
    tools.commands.clear()
    assert b.needs_build()
    b.build()
    assert os.path.exists(b.ROWOPS_PATH) and len(tools.commands) == 1


def test_libraries_are_linked_where_the_module_fails(tools):
    tools.failing = ("g++",)
    with pytest.raises(RuntimeError, match="rowops_py.cpp"):
        b.build()
    assert os.path.exists(b.LIB_PATH) and os.path.exists(b.DEBUG_LIB_PATH) and b.needs_build()


@pytest.mark.parametrize("what", ["torch", "python"])
def test_another_pytorch_or_python_rebuilds_the_module_alone(tools, monkeypatch, tmp_path, what):
    b.build()
    tools.commands.clear()
    if what == "torch":
        (tmp_path / "version.py").write_text("__version__ = '0.0.test'")
        spec = types.SimpleNamespace(submodule_search_locations=[str(tmp_path)])
        find = importlib.util.find_spec
        monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: spec if name == "torch" else find(name, *a))
    else:
        var = sysconfig.get_config_var
        monkeypatch.setattr(sysconfig, "get_config_var", lambda n: "cpython-0-test" if n == "SOABI" else var(n))
    assert b.needs_build()
    b.build()
    assert len(tools.commands) == 1 and tools.ran("rowops_py.cpp") and not b.needs_build()


@pytest.mark.parametrize("source,module_only", [("rowops_py.cpp", True), ("moe.cu", False)])
def test_a_newer_source_rebuilds_what_is_made_of_it(tools, monkeypatch, source, module_only):
    b.build()
    tools.commands.clear()
    real = os.path.getmtime
    later = max(real(p) for p in (b.LIB_PATH, b.DEBUG_LIB_PATH, b.ROWOPS_PATH)) + 10
    monkeypatch.setattr(os.path, "getmtime", lambda p: later if p == os.path.join(b.CSRC, source) else real(p))
    assert b.needs_build()
    b.build()
    assert bool(tools.ran("rowops_py.cpp")) == module_only and bool(tools.ran("moe.cu")) != module_only
