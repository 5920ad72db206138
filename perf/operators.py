"""The token operators' workloads: embedding lookup and its gradient, token log
probabilities with entropy and top alternatives and their gradient, and
distillation from a teacher's top logits, forward and backward.

``run`` computes a pass in elementary torch operations in 32 bits, or with
``own`` through the package's entry points; ``exact`` is the definition in 64
bits.  Sizes are those of the repository's models (char GPT: vocabulary 65, 384
wide, context 256; GPT-2: 50257, 768 or 1600 wide, context 1024; the Llama
shape: 32000, 4096 wide) and ranges around them.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


def listed():
    return [
        # The char GPT's batch of eight 256-token contexts: a launch's latency.
        dict(name="lookup_char", op="lookup", n=2048, vocab=65, dim=384, dtype="bf16",
             out="bf16", scale=1.0, ids=64),
        # A Llama-shaped batch, scaled by sqrt(dim), into the bf16 residual stream.
        dict(name="lookup_llama", op="lookup", n=16384, vocab=32000, dim=4096, dtype="bf16",
             out="bf16", scale=64.0, ids=32),
        # The char GPT: 65 rows share 2048 tokens, so every row is a long sum.
        dict(name="embed_grad_char", op="embed_grad", n=2048, vocab=65, dim=384, dtype="bf16",
             out="bf16", scale=1.0, ids=64, accumulate=False),
        # GPT-2 124M, sixteen contexts of 1024, into the rank's bf16 gradient arena.
        dict(name="embed_grad_124m", op="embed_grad", n=16384, vocab=50257, dim=768,
             dtype="bf16", out="bf16", scale=1.0, ids=64, accumulate=False),
        # GPT-2 1.5B, tied head: ragged packed contexts added onto the head's gradient, fp32.
        dict(name="embed_grad_1p5b_tied", op="embed_grad", n=8011, vocab=50257, dim=1600,
             dtype="f32", out="f32", scale=1.0, ids=32, accumulate=True),
        # One answered token with its alternatives: serving, or one evaluated position.
        dict(name="logprobs_one", op="logprobs", n=1, vocab=32000, stride=32000, dtype="bf16",
             top=20, ids=64),
        # Evaluation of four GPT-2 contexts, or a teacher's top list for distillation.
        dict(name="logprobs_gpt2", op="logprobs", n=4096, vocab=50257, stride=50257,
             dtype="bf16", top=64, ids=64),
        # The char GPT's loss and entropy bonus, fp32 logits.
        dict(name="logprobs_grad_char", op="logprobs_grad", n=2048, vocab=65, stride=65,
             dtype="f32", ids=64),
        # Two 4096-token Llama contexts' cross entropy with an entropy term.
        dict(name="logprobs_grad_llama", op="logprobs_grad", n=8192, vocab=32000, stride=32000,
             dtype="bf16", ids=64),
        # Held-out loss against a teacher's stored list: fp32 logits, forward only.
        dict(name="distill_loss_llama", op="distill_loss", n=1027, vocab=32000, stride=32000,
             dtype="f32", k=64, temperature=1.0),
        # The char GPT's context distilled from its larger teacher's top eight.
        dict(name="distill_grad_char", op="distill_grad", n=256, vocab=65, stride=65,
             dtype="bf16", k=8, temperature=2.0),
        # Four GPT-2 contexts, the vocabulary padded to a multiple of 64 in memory.
        dict(name="distill_grad_gpt2", op="distill_grad", n=4096, vocab=50257, stride=50304,
             dtype="bf16", k=32, temperature=2.0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["lookup", "embed_grad", "logprobs", "logprobs_grad", "distill_loss",
                     "distill_grad"])
    vocab = _log_int(rng, 65, 50257)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    ids = rng.choice([32, 64])
    if op in ("lookup", "embed_grad"):
        dim = _log_int(rng, 96, 4096)
        if rng.random() < 0.6:
            dim = max(64, dim // 64 * 64)
        n = _log_int(rng, 1, max(1, min(16384, (32 << 20) // dim)))
        out = rng.choice(["bf16", "f32"])
        case = dict(op=op, n=n, vocab=vocab, dim=dim, dtype=dtype, out=out,
                    scale=rng.choice([1.0, math.sqrt(dim), 0.5]), ids=ids)
        if op == "embed_grad":
            case["accumulate"] = rng.random() < 0.3
            if case["accumulate"]:
                case["out"] = "f32"
        return case
    n = _log_int(rng, 1, max(1, min(16384, (64 << 20) // vocab)))
    stride = vocab if rng.random() < 0.5 else -(-vocab // 64) * 64 + rng.choice([0, 64])
    case = dict(op=op, n=n, vocab=vocab, stride=stride, dtype=dtype)
    if op == "logprobs":
        case.update(top=rng.choice([0, 1, 5, 20, 64]), ids=ids)
    elif op == "logprobs_grad":
        case.update(ids=ids)
    else:
        case.update(k=_log_int(rng, 1, 64), temperature=rng.choice([1.0, 2.0, 4.0]))
    return case


def _tokens(g, n, vocab, bits):
    # Text's ids: frequent ones small (probability falls as 1 / rank), and a few
    # positions of padding that name no row.
    u = torch.rand(n, device=DEV, generator=g, dtype=torch.float64)
    t = (torch.exp(u * math.log(vocab + 1.0)) - 1.0).long().clamp_(0, vocab - 1)
    pad = torch.rand(n, device=DEV, generator=g) < 0.02
    t = torch.where(pad & (torch.arange(n, device=DEV) > 0), torch.full_like(t, -100), t)
    return t if bits == 64 else t.int()


def _logits(g, case):
    # A trained model's rows: spread of a few units, some tokens well above it.
    n, v = case["n"], case["vocab"]
    full = torch.zeros(n, case["stride"], device=DEV, dtype=TYPES[case["dtype"]])
    x = torch.randn(n, v, device=DEV, generator=g).mul_(2.5)
    lift = torch.randint(0, v, (n, 4), device=DEV, generator=g)
    x.scatter_add_(1, lift, 3.0 + 4.0 * torch.rand(n, 4, device=DEV, generator=g))
    full[:, :v] = x
    return full[:, :v]


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    op, n, v = case["op"], case["n"], case["vocab"]
    s = dict(case)
    if op in ("lookup", "embed_grad"):
        d = case["dim"]
        s["tokens"] = _tokens(g, n, v, case["ids"])
        rows = v if op == "lookup" else n
        x = torch.randn(rows, d, device=DEV, generator=g).mul_(0.02)
        s["x"] = x.to(TYPES[case["dtype"]])
        shape = (n, d) if op == "lookup" else (v, d)
        s["y"] = torch.empty(shape, device=DEV, dtype=TYPES[case["out"]])
        if op == "embed_grad":
            if case["accumulate"]:
                s["y"].normal_(generator=g).mul_(0.02)
            if own:  # the program's workspace
                import gradient_reduce_zero_amd as grz
                s["ws"] = torch.empty(max(1, grz.dp_embed_grad_workspace(n, v, d)),
                                      device=DEV, dtype=torch.uint8)
        return s
    s["x"] = _logits(g, case)
    if op in ("logprobs", "logprobs_grad"):
        s["targets"] = _tokens(g, n, v, case["ids"])
        s["logprob"] = torch.empty(n, device=DEV)
        s["entropy"] = torch.empty(n, device=DEV)
        if op == "logprobs":
            k = case["top"]
            s["top_ids"] = torch.empty(n, k, device=DEV, dtype=torch.int32)
            s["top_logprobs"] = torch.empty(n, k, device=DEV)
        else:
            s["glogprob"] = torch.rand(n, device=DEV, generator=g).sub_(1.0)
            s["gentropy"] = torch.rand(n, device=DEV, generator=g).mul_(0.01)
    else:
        # The teacher agrees with the student on most of its list.
        k = min(case["k"], v)
        noisy = s["x"].float() + torch.randn(n, v, device=DEV, generator=g)
        s["teacher"], ids = torch.topk(noisy, k, dim=1)
        s["ids"] = ids.int()
        w = torch.rand(n, device=DEV, generator=g) + 0.5
        s["weights"] = torch.where(torch.rand(n, device=DEV, generator=g) < 0.02,
                                   torch.zeros_like(w), w)
        s["loss"] = torch.empty(n, device=DEV)
    if op in ("logprobs_grad", "distill_grad"):
        s["dx"] = torch.empty(n, case["stride"], device=DEV, dtype=s["x"].dtype)[:, :v]
    return s


def _run_own(s):
    import gradient_reduce_zero_amd as grz
    op = s["op"]
    if op == "lookup":
        grz.dp_embed_lookup(s["x"], s["tokens"], s["y"], scale=s["scale"])
        return {"out": s["y"]}
    if op == "embed_grad":
        grz.dp_embed_grad(s["x"], s["tokens"], s["y"], s["ws"], scale=s["scale"],
                          accumulate=s["accumulate"])
        return {"dtable": s["y"]}
    if op == "logprobs":
        grz.dp_token_logprobs(s["x"], s["targets"], s["logprob"], s["entropy"], s["top_ids"],
                              s["top_logprobs"])
        return {"logprob": s["logprob"], "entropy": s["entropy"], "top_ids": s["top_ids"],
                "top_logprobs": s["top_logprobs"]}
    if op == "logprobs_grad":
        grz.dp_token_logprobs_grad(s["x"], s["targets"], s["glogprob"], s["gentropy"], s["dx"],
                                   logprob=s["logprob"], entropy=s["entropy"])
        return {"logprob": s["logprob"], "entropy": s["entropy"], "dlogits": s["dx"]}
    if op == "distill_loss":
        grz.dp_distill_loss(s["x"], s["ids"], s["teacher"], s["loss"], weights=s["weights"],
                            temperature=s["temperature"])
        return {"loss": s["loss"]}
    grz.dp_distill_grad(s["x"], s["ids"], s["teacher"], s["dx"], weights=s["weights"],
                        temperature=s["temperature"], loss=s["loss"])
    return {"loss": s["loss"], "dlogits": s["dx"]}


def run(s):
    if own:
        return _run_own(s)
    op, x, v = s["op"], s["x"], s["vocab"]
    if op in ("lookup", "embed_grad"):
        t = s["tokens"].long()
        ok = (t >= 0) & (t < v)
        at = torch.where(ok, t, torch.zeros_like(t))
        if op == "lookup":
            rows = x[at].float() * s["scale"]
            return {"out": torch.where(ok[:, None], rows, 0.0).to(TYPES[s["out"]])}
        rows = torch.where(ok[:, None], x.float() * s["scale"], 0.0)
        acc = s["y"] if s["accumulate"] else torch.zeros(v, s["dim"], device=DEV)
        acc.index_add_(0, at, rows)
        return {"dtable": acc.to(TYPES[s["out"]])}
    x = x.float()
    if op in ("logprobs", "logprobs_grad"):
        t = s["targets"].long()
        ok = (t >= 0) & (t < v)
        at = torch.where(ok, t, torch.zeros_like(t))[:, None]
        m = x.max(1, keepdim=True).values
        e = torch.exp(x - m)
        total = e.sum(1, keepdim=True)
        lq = x - m - torch.log(total)
        q = e / total
        entropy = -(q * lq).sum(1)
        logprob = torch.where(ok, lq.gather(1, at)[:, 0], 0.0)
        if op == "logprobs":
            order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :s["top"]]
            return {"logprob": logprob, "entropy": entropy, "top_ids": order.int(),
                    "top_logprobs": lq.gather(1, order)}
        glp = torch.where(ok, s["glogprob"], 0.0)[:, None]
        dx = -q * (glp + s["gentropy"][:, None] * (lq + entropy[:, None]))
        dx.scatter_add_(1, at, glp)
        return {"logprob": logprob, "entropy": entropy, "dlogits": dx.to(s["x"].dtype)}
    tau, w, ids = s["temperature"], s["weights"], s["ids"].long()
    x = x / tau
    m = x.max(1, keepdim=True).values
    e = torch.exp(x - m)
    total = e.sum(1, keepdim=True)
    z = s["teacher"].float() / tau
    z = z - z.max(1, keepdim=True).values
    p = torch.exp(z)
    lp = z - torch.log(p.sum(1, keepdim=True))
    p = p / p.sum(1, keepdim=True)
    lq = x.gather(1, ids) - m - torch.log(total)
    loss = w * tau * tau * (p * (lp - lq)).sum(1)
    if op == "distill_loss":
        return {"loss": loss}
    dx = e / total
    dx.scatter_add_(1, ids, -p)
    dx = dx * (w * tau)[:, None]
    return {"loss": loss, "dlogits": dx.to(s["x"].dtype)}


def work(case):
    op, n, v = case["op"], case["n"], case["vocab"]
    es = BYTES[case["dtype"]]
    if op in ("lookup", "embed_grad"):
        d, rows, eo = case["dim"], min(n, v), BYTES[case["out"]]
        ids = n * case["ids"] // 8
        if op == "lookup":
            return {"bytes": ids + rows * d * es + n * d * eo, "flops": n * d}
        table = 2 * rows * d * eo if case["accumulate"] else v * d * eo
        return {"bytes": ids + n * d * es + table, "flops": 2 * n * d}
    b, f = n * v * es, 6 * n * v
    if op == "logprobs":
        b += n * (case["ids"] // 8 + 8 + 8 * case["top"])
    elif op == "logprobs_grad":
        b, f = 2 * b + n * (case["ids"] // 8 + 16), 12 * n * v
    else:
        b = b * (2 if op == "distill_grad" else 1) + n * (8 * case["k"] + 8)
        f = f * (2 if op == "distill_grad" else 1)
    return {"bytes": b, "flops": f}


def exact(case, seed):
    s = prepare(case, seed)
    op, v, x = s["op"], s["vocab"], s["x"].double()
    if op in ("lookup", "embed_grad"):
        t = s["tokens"].long()
        t = torch.where((t < 0) | (t >= v), torch.full_like(t, v), t)  # row v: no row
        if op == "lookup":
            ext = torch.cat([x, torch.zeros(1, s["dim"], device=DEV, dtype=x.dtype)])
            return {"out": torch.index_select(ext, 0, t) * s["scale"]}
        # Differences of running sums over the sorted tokens, column block by block.
        order = torch.sort(t, stable=True)
        ends = torch.searchsorted(order.values, torch.arange(v, device=DEV), right=True)
        run_sum = torch.zeros(s["n"] + 1, s["dim"], device=DEV, dtype=x.dtype)
        torch.cumsum(x[order.indices], 0, out=run_sum[1:])
        starts = torch.cat([ends.new_zeros(1), ends[:-1]])
        out = (run_sum[ends] - run_sum[starts]) * s["scale"]
        return {"dtable": out + s["y"].double() if s["accumulate"] else out}
    if op in ("logprobs", "logprobs_grad"):
        lq = x - torch.logsumexp(x, 1, keepdim=True)
        q = lq.exp()
        entropy = -torch.sum(q * lq, 1)
        t = s["targets"].long()
        ok = (t >= 0) & (t < v)
        rows = torch.arange(s["n"], device=DEV)
        logprob = lq[rows, t.clamp(0, v - 1)].masked_fill(~ok, 0.0)
        if op == "logprobs":
            order = torch.argsort(-x, dim=1, stable=True)[:, :s["top"]]
            return {"logprob": logprob, "entropy": entropy, "top_ids": None,
                    "top_logprobs": torch.take_along_dim(lq, order, 1)}
        glp = s["glogprob"].double().masked_fill(~ok, 0.0)
        ge = s["gentropy"].double()
        dx = glp[:, None] * -q - ge[:, None] * q * (lq + entropy[:, None])
        dx[rows, t.clamp(0, v - 1)] += glp
        return {"logprob": logprob, "entropy": entropy, "dlogits": dx}
    tau, w, ids = s["temperature"], s["weights"].double(), s["ids"].long()
    lq = torch.log_softmax(x / tau, 1)
    z = s["teacher"].double() / tau
    lp = z - torch.logsumexp(z, 1, keepdim=True)
    loss = w * tau ** 2 * torch.sum(lp.exp() * (lp - torch.take_along_dim(lq, ids, 1)), 1)
    if op == "distill_loss":
        return {"loss": loss}
    target = torch.zeros_like(x).scatter_add(1, ids, lp.exp())
    return {"loss": loss, "dlogits": (w * tau)[:, None] * (lq.exp() - target)}
