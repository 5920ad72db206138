"""The README's example of one clip factor over the arena and a rank's experts: the
factor exists before either is updated, and both updates take it."""

import ast
import os
import re
import types

import pytest
import torch

import gradient_reduce_zero_amd as grz

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U = 2.0 ** -24


def example():
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    (block,) = [b for b in blocks if "dp_grad_sqnorm_tensors(" in b]
    return block


def test_factor_comes_between_the_reduce_and_the_updates():
    calls = {}
    for c in ast.walk(ast.parse(example())):
        if isinstance(c, ast.Call) and isinstance(c.func, ast.Attribute):
            calls.setdefault(c.func.attr, []).append(c)
    line = {name: [c.lineno for c in cs] for name, cs in calls.items()}
    (norm,) = line["dp_grad_sqnorm_tensors"]
    assert max(line["dp_reduce_scatter_mean"]) < norm
    factor = ast.unparse(calls["dp_grad_sqnorm_tensors"][0].args[4])
    for update in ("zero1_adamw_gather", "zero1_adamw_step", "dp_grad_clip_tensors"):
        assert min(line[update]) > norm
        for c in calls[update]:
            assert factor in [ast.unparse(a) for a in c.args], update
    # The drivers' steps form a factor of their own and write it over the joint one.
    assert not {"step", "update", "enqueue", "finish"} & set(calls)


@pytest.mark.gpu
def test_example_updates_arena_and_experts_by_the_joint_factor():
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev).manual_seed(3)
    rand = lambda *s: torch.randn(*s, device=dev, generator=g)
    n, k, experts, d, numel, ranks = 50, 2, 6, 24, 10000, 2
    i32 = lambda *s: torch.empty(*s, device=dev, dtype=torch.int32)
    hyper = grz.Hyper(max_norm=0.5, weight_decay=0.0)
    pipe = grz.Zero1AllRanks([(0, 6000), (6000, 4000)], ranks, rand(numel), hyper, device=dev)
    masters = [w.clone() for w, _, _ in pipe.state]
    own = [types.SimpleNamespace(grad=rand(40, 30) * 0.1) for _ in range(3)]  # larger than
    arenas = [rand(numel) * 1e-3 for _ in range(ranks)]                         # the arena's
    state = [tuple(torch.zeros(1200, device=dev) for _ in range(3)) for _ in own]
    names = dict(
        grz=grz, torch=torch, dev=dev, n=n, k=k, experts=experts, pipe=pipe, arenas=arenas,
        args=grz.adamw_args(**grz.step_scalars(hyper, 1)),
        own_experts=own, experts_of_this_rank=own, expert_state=state, logits=rand(n, experts),
        ids=i32(n, k), w=rand(n, k), offsets=i32(experts + 1), places=i32(n, k), x=rand(n, d),
        rows=rand(n * k, d), y=rand(n * k, d), out=rand(n, d), dout=rand(n, d),
        dy=rand(n * k, d), dw=rand(n, k), drows=rand(n * k, d), dx=rand(n, d),
        dlogits=rand(n, experts))
    raw = [p.grad.clone() for p in own]
    exec(compile(example(), "README.md", "exec"), names)
    torch.cuda.synchronize()
    mean = (arenas[0].double() + arenas[1].double()) / ranks
    sq = float((mean ** 2).sum()) + sum(float((t.double() ** 2).sum()) for t in raw)
    factor = hyper.max_norm / sq ** 0.5
    assert factor < 0.5                                   # of the arena alone it is 1
    # The mean is off by two roundings, its square and the sum's root follow.
    assert abs(pipe.norm.sqnorm.item() - sq) <= 8 * U * sq
    assert abs(pipe.norm.scale.item() - factor) <= 8 * U * factor
    # After one step from zero m is (1 - beta1) times the clipped gradient: the factor's 8
    # roundings, two of the mean, of 1 - beta1 (a difference near 0.1: 16), two products.
    lim = (8 + 2 + 16 + 2) * U
    clipped = (1 - hyper.beta1) * factor
    for i, (c, (w, m, v)) in enumerate(zip(pipe.chunks, pipe.state)):
        at = torch.cat([torch.arange(o + first, o + first + count)
                        for o, length in pipe.buckets
                        for first, count in [grz.dp_chunk_range(length, ranks, c)]])
        want = clipped * mean[at.to(dev)]
        assert ((m.double() - want).abs() <= lim * want.abs() + 1e-12 * U).all()
        assert not torch.equal(w, masters[i])
    for p, r, (w, m, v) in zip(own, raw, state):
        want = clipped * r.double().reshape(-1)
        assert ((m.double() - want).abs() <= lim * want.abs()).all()
        assert (w != 0).all()
        assert torch.equal(p.grad, r * pipe.norm.scale)
