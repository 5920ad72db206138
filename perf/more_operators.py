"""Workloads of the mixture-of-experts operators and of the norm over many tensors:
the router and its gradient, tokens sorted by expert and laid out for the
experts, their outputs summed back with the router's weights, the gradient of
that sum, and the global gradient norm over many tensors with clipping.

``run`` computes a pass in elementary torch operations in 32 bits (the norm's
sums in 64), or with ``own`` through the package's entry points; ``exact`` is the
definition in 64 bits.  Widths are those of the repository's models (char GPT:
384; GPT-2: 768, 1600; the Llama shape: 4096), numbers of experts and slots are
generic, and ``draw`` takes ranges around them.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


def listed():
    return [
        # One decoded token's eight experts of 64, its weights summing to 1.
        dict(name="route_one", op="route", n=1, experts=64, k=8, stride=64, dtype="f32",
             normalize=True, allowed=64),
        # Four 4096-token contexts in training.
        dict(name="route_train", op="route", n=16384, experts=128, k=8, stride=128,
             dtype="bf16", normalize=True, allowed=128),
        # The char GPT with eight experts, two a token, weights of the whole softmax.
        dict(name="route_grad_char", op="route_grad", n=2048, experts=8, k=2, stride=8,
             dtype="f32", normalize=False, allowed=8),
        # Many experts, half of them closed to each token, rows padded in memory.
        dict(name="route_grad_wide", op="route_grad", n=16384, experts=256, k=8, stride=264,
             dtype="bf16", normalize=True, allowed=128),
        # The char GPT's batch of eight 256-token contexts to its experts: latency.
        dict(name="dispatch_char", op="dispatch", n=2048, dim=384, experts=8, k=2,
             dtype="bf16", out="bf16", weighted=False, ids=64),
        # Four 4096-token contexts of the Llama shape, six experts of 64 each.
        dict(name="dispatch_llama", op="dispatch", n=16384, dim=4096, experts=64, k=6,
             dtype="bf16", out="bf16", weighted=False, ids=32),
        # A decoding batch: 32 tokens back from eight experts of 128 each.
        dict(name="combine_decode", op="combine", n=32, dim=4096, experts=128, k=8,
             dtype="bf16", out="bf16", weighted=True, accumulate=False),
        # The dispatch's gradient in fp32, ragged packed contexts 1600 wide, added onto
        # what the residual path left.
        dict(name="combine_1p5b_added", op="combine", n=8011, dim=1600, experts=16, k=2,
             dtype="f32", out="f32", weighted=False, accumulate=True),
        # Eight 1024-token contexts 768 wide, two experts each, fp32 gradient coming in.
        dict(name="combine_grad_gpt2", op="combine_grad", n=8192, dim=768, experts=8, k=2,
             dtype="bf16", out="f32"),
        # The Llama-shaped layer's backward.
        dict(name="combine_grad_llama", op="combine_grad", n=16384, dim=4096, experts=64, k=6,
             dtype="bf16", out="bf16"),
        # The char GPT's gradients as its tensors: latency.
        dict(name="clip_char", op="clip", layers=6, dim=384, ffn=1536, experts=1, dtype="bf16"),
        # The experts a rank holds of a 1600-wide model, with the layers around them.
        dict(name="clip_experts", op="clip", layers=6, dim=1600, ffn=6400, experts=8,
             dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "dispatch", "dispatch", "combine", "combine_grad",
                     "clip"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "clip":
        dim = _log_int(rng, 96, 1600)
        return dict(op=op, layers=rng.randint(1, 6), dim=dim,
                    ffn=rng.choice([2 * dim, 4 * dim, 4 * dim + 3]),
                    experts=rng.choice([1, 2, 5, 8]), dtype=dtype)
    experts = _log_int(rng, 4, 256)
    k = rng.randint(1, min(8, experts))
    if op in ("route", "route_grad"):
        stride = experts + rng.choice([0, 0, 8, 3])
        return dict(op=op, n=_log_int(rng, 1, 16384), experts=experts, k=k, stride=stride,
                    dtype=dtype, normalize=rng.random() < 0.5,
                    allowed=rng.choice([experts, experts, max(1, experts // 2)]))
    dim = _log_int(rng, 96, 4096)
    if rng.random() < 0.6:
        dim = max(64, dim // 64 * 64)
    n = _log_int(rng, 1, max(1, min(16384, (180 << 20) // (dim * k))))
    case = dict(op=op, n=n, dim=dim, experts=experts, k=k, dtype=dtype,
                out=rng.choice(["bf16", "f32"]))
    if op == "dispatch":
        case.update(weighted=rng.random() < 0.3, ids=rng.choice([32, 64]))
    elif op == "combine":
        case.update(weighted=rng.random() < 0.7, accumulate=rng.random() < 0.3)
        if case["accumulate"]:
            case["out"] = "f32"
    return case


def _pads(n):
    """Positions of padding at a batch's end: tokens that go to no expert."""
    return n // 64


def _router_logits(g, n, experts, stride, dtype, allowed):
    # A trained router: some experts liked more than others, and a batch's last
    # positions padding, with every expert closed.
    full = torch.zeros(n, stride, device=DEV, dtype=dtype)
    x = torch.randn(n, experts, device=DEV, generator=g)
    x += 0.5 * torch.randn(experts, device=DEV, generator=g)
    if allowed < experts:
        order = torch.rand(n, experts, device=DEV, generator=g).argsort(1)
        x.scatter_(1, order[:, allowed:], float("-inf"))
    if _pads(n):
        x[n - _pads(n):] = float("-inf")
    full[:, :experts] = x
    return full[:, :experts]


def _top(x, k):
    """Ids of the k largest of each row, equal ones by lower id, -1 for -inf."""
    v, at = torch.sort(x, dim=1, descending=True, stable=True)
    return torch.where(v[:, :k] == float("-inf"), -1, at[:, :k]).int()


def _sorted_places(ids, experts):
    """(offsets, places) of the slots sorted by expert, slots of no expert at -1."""
    flat = ids.reshape(-1).long()
    ok = (flat >= 0) & (flat < experts)
    key = torch.where(ok, flat, experts)
    order = torch.sort(key, stable=True).indices
    places = torch.empty_like(flat)
    places[order] = torch.arange(flat.numel(), device=DEV)
    places = torch.where(ok, places, -1).reshape(ids.shape).int()
    counts = torch.zeros(experts + 1, device=DEV, dtype=torch.long)
    counts.index_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(experts + 1, device=DEV, dtype=torch.long)
    offsets[1:] = torch.cumsum(counts[:experts], 0)
    return offsets.int(), places


def _tensor_shapes(case):
    """(shape, type) of the gradients: two norms and a router in fp32, four attention
    matrices and each expert's two in the case's type, per layer."""
    d, f, out = case["dim"], case["ffn"], []
    for _ in range(case["layers"]):
        out += [((d,), "f32"), ((d,), "f32")]
        if case["experts"] > 1:
            out.append(((case["experts"], d), "f32"))
        out += [((d, d), case["dtype"])] * 4
        out += [((f, d), case["dtype"]), ((d, f), case["dtype"])] * case["experts"]
    return out


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    op = case["op"]
    s = dict(case)
    if op == "clip":
        s["grads"] = [torch.randn(shape, device=DEV, generator=g).mul_(0.02).to(TYPES[t])
                      for shape, t in _tensor_shapes(case)]
        # The clipped gradients go to flat arenas, one a type, tensor behind tensor.
        s["arenas"], s["clipped"] = {}, []
        for t in (torch.bfloat16, torch.float32):
            total = sum(x.numel() for x in s["grads"] if x.dtype == t)
            s["arenas"][t] = torch.empty(total, device=DEV, dtype=t)
        used = {t: 0 for t in s["arenas"]}
        for x in s["grads"]:
            at, used[x.dtype] = used[x.dtype], used[x.dtype] + x.numel()
            s["clipped"].append(s["arenas"][x.dtype][at:at + x.numel()].view(x.shape))
        s["max_norm"] = 1.0
        s["sqnorm"] = torch.empty(1, device=DEV, dtype=torch.float64)
        s["scale"] = torch.empty(1, device=DEV)
        if own:  # the program's lists and workspace
            import gradient_reduce_zero_amd as grz
            s["from"], s["to"] = grz.TensorList(s["grads"]), grz.TensorList(s["clipped"])
            s["ws"] = torch.empty(grz.dp_grad_sqnorm_tensors_workspace(s["from"]),
                                  device=DEV, dtype=torch.uint8)
        return s
    n, e, k = case["n"], case["experts"], case["k"]
    if op in ("route", "route_grad"):
        s["x"] = _router_logits(g, n, e, case["stride"], TYPES[case["dtype"]], case["allowed"])
        if op == "route":
            s["ids"] = torch.empty(n, k, device=DEV, dtype=torch.int32)
            s["weights"] = torch.empty(n, k, device=DEV)
        else:
            s["ids"] = _top(s["x"], k)
            s["dweights"] = torch.randn(n, k, device=DEV, generator=g)
            s["dx"] = torch.empty(n, case["stride"], device=DEV, dtype=s["x"].dtype)[:, :e]
        return s
    d, rows = case["dim"], n * k
    logits = _router_logits(g, n, e, e, torch.float32, e)
    ids = _top(logits, k)
    w = torch.softmax(logits, 1).gather(1, ids.clamp(min=0).long())
    s["weights"] = torch.where(ids >= 0, w / w.sum(1, keepdim=True), 0.0)
    # Activations, or their gradients, of unit size.
    if op == "dispatch":
        s["ids_in"] = ids if case["ids"] == 32 else ids.long()
        s["x"] = torch.randn(n, d, device=DEV, generator=g).to(TYPES[case["dtype"]])
        s["y"] = torch.zeros(rows, d, device=DEV, dtype=TYPES[case["out"]])
        s["offsets"] = torch.empty(e + 1, device=DEV, dtype=torch.int32)
        s["places"] = torch.empty(n, k, device=DEV, dtype=torch.int32)
        if own:  # the program's workspace
            import gradient_reduce_zero_amd as grz
            s["ws"] = torch.empty(max(1, grz.dp_expert_sort_workspace(n, k, e)), device=DEV,
                                  dtype=torch.uint8)
        return s
    s["places"] = _sorted_places(ids, e)[1]
    s["y"] = torch.randn(rows, d, device=DEV, generator=g).to(TYPES[case["dtype"]])
    if op == "combine":
        s["out_rows"] = torch.zeros(n, d, device=DEV, dtype=TYPES[case["out"]])
        if case["accumulate"]:
            s["out_rows"].normal_(generator=g)
    else:
        s["dout"] = torch.randn(n, d, device=DEV, generator=g).to(TYPES[case["out"]])
        s["dy"] = torch.zeros_like(s["y"])
        s["dweights"] = torch.empty(n, k, device=DEV)
    return s


def _run_own(s):
    import gradient_reduce_zero_amd as grz
    op = s["op"]
    if op == "route":
        grz.dp_expert_route(s["x"], s["ids"], s["weights"], normalize=s["normalize"])
        return {"ids": s["ids"], "weights": s["weights"]}
    if op == "route_grad":
        grz.dp_expert_route_grad(s["x"], s["ids"], s["dweights"], s["dx"],
                                 normalize=s["normalize"])
        return {"dlogits": s["dx"]}
    w = s.get("weights") if s.get("weighted", True) else None
    if op == "dispatch":
        grz.dp_expert_sort(s["ids_in"], s["experts"], s["offsets"], s["places"], s["ws"])
        grz.dp_expert_dispatch(s["x"], s["places"], s["y"], weights=w)
        return {"offsets": s["offsets"], "places": s["places"], "rows": s["y"]}
    if op == "combine":
        grz.dp_expert_combine(s["y"], s["places"], s["out_rows"], weights=w,
                              accumulate=s["accumulate"])
        return {"out": s["out_rows"]}
    if op == "combine_grad":
        grz.dp_expert_combine_grad(s["dout"], s["y"], s["places"], w, dy=s["dy"],
                                   dweights=s["dweights"])
        return {"dy": s["dy"], "dweights": s["dweights"]}
    grz.dp_grad_sqnorm_tensors(s["from"], s["max_norm"], s["ws"], s["sqnorm"], s["scale"])
    grz.dp_grad_clip_tensors(s["from"], s["scale"], out=s["to"])
    return {"sqnorm": s["sqnorm"], "scale": s["scale"],
            "bf16": s["arenas"][torch.bfloat16], "f32": s["arenas"][torch.float32]}


def _run_route(s):
    x, k = s["x"].float(), s["k"]
    open_row = (x > float("-inf")).any(1, keepdim=True)
    m = torch.where(open_row, x.max(1, keepdim=True).values, 0.0)
    e = torch.exp(x - m)
    ids = _top(x, k) if s["op"] == "route" else s["ids"]
    at, ok = ids.clamp(min=0).long(), ids >= 0
    chosen = torch.where(ok, e.gather(1, at), 0.0)
    total = (chosen if s["normalize"] else e).sum(1, keepdim=True)
    total = torch.where(open_row, total, 1.0)
    w = chosen / total
    if s["op"] == "route":
        return {"ids": ids, "weights": w}
    gw = torch.where(ok, s["dweights"], 0.0) * w
    both = gw.sum(1, keepdim=True)
    if s["normalize"]:
        dx = torch.zeros_like(x).scatter_add_(1, at, gw - w * both)
    else:
        dx = (-both * (e / total)).scatter_add_(1, at, gw)
    return {"dlogits": dx.to(s["x"].dtype)}


def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op in ("route", "route_grad"):
        return _run_route(s)
    if op == "clip":
        sq = torch.zeros(1, device=DEV, dtype=torch.float64)
        for t in s["grads"]:
            x = t.double()
            sq += (x * x).sum()
        norm = torch.sqrt(sq)
        scale = torch.where(norm > s["max_norm"], s["max_norm"] / norm, 1.0).float()
        out = {"sqnorm": sq, "scale": scale}
        for name, t in TYPES.items():
            parts = [(x.float() * scale).to(t).reshape(-1) for x in s["grads"] if x.dtype == t]
            out[name] = torch.cat(parts) if parts else torch.empty(0, device=DEV, dtype=t)
        return out
    n, k, rows = s["n"], s["k"], s["n"] * s["k"]
    out = TYPES[s["out"]]
    if op == "dispatch":
        offsets, places = _sorted_places(s["ids_in"], s["experts"])
        at = torch.where(places >= 0, places, rows).long()  # behind the rows: no place
        y = torch.zeros(rows + 1, s["dim"], device=DEV, dtype=out)
        for j in range(k):
            row = s["x"].float()
            if s["weighted"]:
                row = row * s["weights"][:, j:j + 1]
            y[at[:, j]] = row.to(out)
        return {"offsets": offsets, "places": places, "rows": y[:rows]}
    ok = s["places"] >= 0
    at = s["places"].clamp(min=0).long()
    if op == "combine":
        acc = s["out_rows"] if s["accumulate"] else torch.zeros(n, s["dim"], device=DEV)
        for j in range(k):
            row = torch.where(ok[:, j:j + 1], s["y"][at[:, j]].float(), 0.0)
            acc += row * s["weights"][:, j:j + 1] if s["weighted"] else row
        return {"out": acc.to(out)}
    dout = s["dout"].float()
    dy = torch.zeros(rows + 1, s["dim"], device=DEV, dtype=s["y"].dtype)
    dw = torch.empty(n, k, device=DEV)
    for j in range(k):
        dw[:, j] = torch.where(ok[:, j], (dout * s["y"][at[:, j]].float()).sum(1), 0.0)
        dy[torch.where(ok[:, j], at[:, j], rows)] = \
            (dout * s["weights"][:, j:j + 1]).to(dy.dtype)
    return {"dy": dy[:rows], "dweights": dw}


def work(case):
    op = case["op"]
    es = BYTES[case["dtype"]]
    if op == "clip":
        sizes = [(math.prod(shape), BYTES[t]) for shape, t in _tensor_shapes(case)]
        return {"bytes": sum(2 * c * b for c, b in sizes),
                "flops": 3 * sum(c for c, _ in sizes)}
    n, e, k = case["n"], case["experts"], case["k"]
    if op == "route":
        return {"bytes": n * e * es + 8 * n * k, "flops": 4 * n * e}
    if op == "route_grad":
        return {"bytes": 2 * n * e * es + 8 * n * k, "flops": 6 * n * e}
    d, eo, live = case["dim"], BYTES[case["out"]], n - _pads(n)
    if op == "dispatch":
        slots = n * k * (case["ids"] // 8 + 4 + (4 if case["weighted"] else 0))
        return {"bytes": slots + 4 * e + live * d * (es + k * eo), "flops": live * k * d}
    if op == "combine":
        slots = n * k * (4 + (4 if case["weighted"] else 0))
        sums = n * d * eo * (2 if case["accumulate"] else 1)
        return {"bytes": slots + live * k * d * es + sums, "flops": 2 * live * k * d}
    return {"bytes": 12 * n * k + live * d * (eo + 2 * k * es), "flops": 3 * live * k * d}


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "clip":
        sq = sum(torch.linalg.vector_norm(t, dtype=torch.float64) ** 2 for t in s["grads"])
        factor = torch.clamp(s["max_norm"] / torch.sqrt(sq), max=1.0)
        out = {"sqnorm": sq.reshape(1), "scale": factor.reshape(1)}
        for name, arena in s["arenas"].items():
            flat, at = torch.empty(arena.numel(), device=DEV, dtype=torch.float64), 0
            for x in (x for x in s["grads"] if x.dtype == name):
                flat[at:at + x.numel()] = torch.mul(x.double(), factor).flatten()
                at += x.numel()
            out["bf16" if name == torch.bfloat16 else "f32"] = flat
        return out
    n, k = s["n"], s["k"]
    if op in ("route", "route_grad"):
        # Over the open experts only: a closed one is left out, not multiplied by 0.
        x = s["x"].double()
        ids = (_top(s["x"], k) if op == "route" else s["ids"]).long()
        rest = torch.arange(n, device=DEV)[:, None]
        listed_ = x[rest, ids.clamp(min=0)].masked_fill(ids < 0, float("-inf"))
        pool = listed_ if s["normalize"] else x
        lse = torch.logsumexp(pool, 1, keepdim=True)
        w = torch.exp(listed_ - lse).masked_fill(ids < 0, 0.0)
        if op == "route":
            return {"ids": None, "weights": w}
        g = s["dweights"].double().masked_fill(ids < 0, 0.0)
        hot = torch.zeros(n, s["experts"], device=DEV, dtype=torch.float64)
        inner = (w * g).sum(1, keepdim=True)
        for j in range(k):
            share = w[:, j:j + 1] * (g[:, j:j + 1] - (inner if s["normalize"] else 0.0))
            hot.scatter_add_(1, ids[:, j:j + 1].clamp(min=0), share)
        if not s["normalize"]:
            p = torch.exp(x - lse)
            hot = hot - p.masked_fill(torch.isnan(p), 0.0) * inner
        return {"dlogits": hot}
    d = s["dim"]
    if op == "dispatch":
        # Expert by expert: its slots in the order of their tokens.
        flat = s["ids_in"].reshape(-1)
        slots = torch.cat([torch.nonzero(flat == e)[:, 0] for e in range(s["experts"])])
        rows = torch.zeros(n * k, d, device=DEV, dtype=torch.float64)
        rows[:slots.numel()] = s["x"].double()[slots // k]
        if s["weighted"]:
            rows[:slots.numel()] *= s["weights"].double().reshape(-1)[slots][:, None]
        return {"offsets": None, "places": None, "rows": rows}
    # The slot that lies at each row, from the slots' places.
    place = s["places"].reshape(-1)
    slots = torch.nonzero(place >= 0)[:, 0]
    at, token = place[slots].long(), slots // k
    w = s["weights"].double().reshape(-1)[slots][:, None]
    y = s["y"].double()
    if op == "combine":
        out = torch.zeros(n, d, device=DEV, dtype=torch.float64)
        for j in range(k):  # one slot of each token at a time
            some = slots % k == j
            out[token[some]] += y[at[some]] * (w[some] if s["weighted"] else 1.0)
        return {"out": out + s["out_rows"].double() if s["accumulate"] else out}
    dout = s["dout"].double()
    dy = torch.zeros_like(y)
    dw = torch.zeros(n * k, device=DEV, dtype=torch.float64)
    dy[at] = w * dout[token]
    dw[slots] = torch.linalg.vecdot(dout[token], y[at])
    return {"dy": dy, "dweights": dw.reshape(n, k)}
