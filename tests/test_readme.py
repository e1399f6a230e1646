"""The calls that the usage text shows: names and arguments that the binding has, and every
`_backward` call with the settings of the forward call before it (no GPU)."""
import ast
import inspect
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SETTINGS = ("scale", "interleaved", "act", "q_heads")     # what a gradient has to be told again


def _blocks():
    with open(os.path.join(ROOT, "README.md")) as f:
        return re.findall(r"```python\n(.*?)```", f.read(), re.S)


def _calls(block):
    """(name, its arguments by parameter) of the calls mx.name(...), in the order of the text."""
    binding = pytest.importorskip("mx_block_scaled_gb300.binding")
    calls = [n for n in ast.walk(ast.parse(block)) if isinstance(n, ast.Call) and isinstance(n.func, ast.Attribute)
             and isinstance(n.func.value, ast.Name) and n.func.value.id == "mx"]
    for c in sorted(calls, key=lambda c: (c.lineno, c.col_offset)):
        bound = inspect.signature(getattr(binding, c.func.attr)).bind(*c.args, **{k.arg: k.value for k in c.keywords})
        yield c.func.attr, {k: ast.unparse(v) for k, v in bound.arguments.items() if isinstance(v, ast.AST)}


@pytest.mark.parametrize("i", range(len(_blocks())))
def test_calls_bind(i):
    list(_calls(_blocks()[i]))


@pytest.mark.parametrize("i", range(len(_blocks())))
def test_gradients_repeat_the_forward_settings(i):
    forward = {}
    for name, args in _calls(_blocks()[i]):
        if name.endswith("_backward"):
            before = forward[name[:-len("_backward")]]
            for s in SETTINGS:
                assert args.get(s) == before.get(s), (name, s)
        forward[name] = args
