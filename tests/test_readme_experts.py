"""The README's example of the mixture-of-experts operators and of the norm over
tensors: its calls fit the functions' parameters and name every entry point.  No GPU
work."""

import ast
import inspect
import os
import re

import gradient_reduce_zero_amd as grz

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_calls_of_the_example_fit():
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    (block,) = [b for b in blocks if "dp_expert_route" in b]
    seen = set()
    for c in ast.walk(ast.parse(block)):
        if isinstance(c, ast.Call) and isinstance(c.func, ast.Attribute) and \
                isinstance(c.func.value, ast.Name) and c.func.value.id == "grz":
            inspect.signature(getattr(grz, c.func.attr)).bind(
                *c.args, **{k.arg: k.value for k in c.keywords})
            seen.add(c.func.attr)
    assert {n for n in dir(grz) if n.startswith("dp_expert") or
            n.startswith("dp_grad") and "tensors" in n} <= seen
