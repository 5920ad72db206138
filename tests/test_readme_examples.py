"""The README's example of the token operators: its calls fit the functions'
parameters, and none reads what an earlier one has overwritten.  No GPU work."""

import ast
import inspect
import os
import re

import gradient_reduce_zero_amd as grz

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
WRITTEN = ("dlogits", "out", "logprob", "entropy", "top_ids", "top_logprobs", "loss")


def calls_of_the_example():
    """(line, function, its arguments by parameter) of each grz.dp_* call."""
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    (block,) = [b for b in blocks if "dp_embed_lookup" in b]
    calls = [c for c in ast.walk(ast.parse(block))
             if isinstance(c, ast.Call) and isinstance(c.func, ast.Attribute)
             and c.func.attr.startswith("dp_")]
    for c in sorted(calls, key=lambda c: c.lineno):
        bound = inspect.signature(getattr(grz, c.func.attr)).bind(
            *c.args, **{k.arg: k.value for k in c.keywords})
        yield c.lineno, c.func.attr, {k: ast.unparse(a) for k, a in bound.arguments.items()}


def test_token_operators_example_reads_nothing_overwritten():
    overwritten, seen = {}, set()
    for line, name, args in calls_of_the_example():
        seen.add(name)
        for param, value in args.items():
            if param not in WRITTEN:
                assert value not in overwritten, (
                    f"line {line}: {name} reads {value}, which line {overwritten[value]} overwrote")
        # An output in the place of an input, or of an earlier output.
        overwritten.update({args[p]: line for p in WRITTEN if p in args
                            and args[p] in [v for k, v in args.items() if k != p]})
    assert {"dp_embed_lookup", "dp_embed_grad", "dp_distill_grad", "dp_token_logprobs"} <= seen
