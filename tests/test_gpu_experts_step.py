"""The mixture-of-experts operators, the tensor lists and the data-parallel step
together: one layer's router, experts and residual trained by two simulated ranks,
the dense weights in an averaged arena, the experts' gradients as tensors of their own, one
clip factor over both.  Every gradient is compared with that of the whole batch's
loss in 64 bits."""

import pytest
import torch

import expert_ref as ref
import gradient_reduce_zero_amd as grz
from test_gpu_tokens import BF16, DEV, F32, gen
from token_ref import U

pytestmark = pytest.mark.gpu
I32 = torch.int32
N_TOKENS, DIM, HIDDEN, EXPERTS, K, PAD = 97, 24, 40, 6, 2, 5


class Layer:
    """A rank's forward and backward of sum(g * (x + moe(x))): x is given, the router
    is the dense weight, each expert two matrices with a square between them."""

    def __init__(self, router, w1, w2):
        self.router, self.w1, self.w2 = router, w1, w2

    def run(self, x, g, pad):
        n = x.shape[0]
        i32 = lambda *s: torch.empty(*s, device=DEV, dtype=I32)
        f32 = lambda *s: torch.empty(*s, device=DEV)
        logits = x @ self.router.t()
        if pad:
            logits[n - pad:] = -torch.inf           # padded positions go to no expert
        ids, w = i32(n, K), f32(n, K)
        grz.dp_expert_route(logits, ids, w, normalize=True)
        offsets, places = i32(EXPERTS + 1), i32(n, K)
        ws = torch.empty(max(4, grz.dp_expert_sort_workspace(n, K, EXPERTS)), device=DEV,
                         dtype=torch.uint8)
        grz.dp_expert_sort(ids, EXPERTS, offsets, places, ws)
        rows, y = torch.zeros(n * K, DIM, device=DEV), torch.zeros(n * K, DIM, device=DEV)
        grz.dp_expert_dispatch(x, places, rows)
        at = offsets.tolist()
        mids = {}
        for e in range(EXPERTS):
            r = rows[at[e]:at[e + 1]]
            h = r @ self.w1[e].t()
            mids[e] = (r, h)
            y[at[e]:at[e + 1]] = (h * h) @ self.w2[e].t()
        out = x.clone()                             # the residual, the sum added to it
        grz.dp_expert_combine(y, places, out, weights=w, accumulate=True)
        # Backward of sum(g * out).
        dy, dw = torch.zeros_like(y), f32(n, K)
        grz.dp_expert_combine_grad(g, y, places, w, dy=dy, dweights=dw)
        drows = torch.zeros_like(rows)
        d1, d2 = [], []
        for e in range(EXPERTS):
            d = dy[at[e]:at[e + 1]]
            r, h = mids[e]
            dh = 2 * h * (d @ self.w2[e])
            d2.append(d.t() @ (h * h))
            d1.append(dh.t() @ r)
            drows[at[e]:at[e + 1]] = dh @ self.w1[e]
        dx = g.clone()
        grz.dp_expert_combine(drows, places, dx, accumulate=True)
        grz.dp_expert_route_grad(logits, ids, dw, logits, normalize=True)  # over the logits
        drouter = logits.t() @ x
        dx += logits @ self.router
        return out, ids, drouter, d1, d2, dx


def exact(router, w1, w2, x, g, ids):
    """Loss gradients in 64 bits for the chosen experts."""
    p = [t.detach().double().cpu().requires_grad_(True) for t in (router, *w1, *w2, x)]
    router, w1, w2, x = p[0], p[1:1 + EXPERTS], p[1 + EXPERTS:1 + 2 * EXPERTS], p[-1]
    ids = ids.cpu().long()
    logits = x @ router.t()
    ok = ids >= 0
    at = ids.clamp(min=0)
    w = torch.softmax(logits.gather(1, at), 1) * ok
    out = x
    for e in range(EXPERTS):
        h = x @ w1[e].t()
        ye = (h * h) @ w2[e].t()
        out = out + ((at == e) * w).sum(1, keepdim=True) * ye
    (out * g.double().cpu()).sum().backward()
    return out.detach(), [t.grad for t in p]


def test_layer_to_the_next_weights():
    ranks = 2
    router = torch.randn(EXPERTS, DIM, device=DEV, generator=gen(1)) * 0.3
    w1 = [torch.randn(HIDDEN, DIM, device=DEV, generator=gen(10 + e)) * 0.2
          for e in range(EXPERTS)]
    w2 = [torch.randn(DIM, HIDDEN, device=DEV, generator=gen(20 + e)) * 0.2
          for e in range(EXPERTS)]
    numel = router.numel()
    buckets = [(0, numel)]
    hyper = grz.Hyper(max_norm=0.05, weight_decay=0.0)
    pipe = grz.Zero1AllRanks(buckets, ranks, router.reshape(-1), hyper, device=DEV)
    lead = pipe.norm.npieces
    results = []
    for r in range(ranks):
        n = N_TOKENS + 30 * r
        x = torch.randn(n, DIM, device=DEV, generator=gen(30 + r))
        g = torch.randn(n, DIM, device=DEV, generator=gen(40 + r)) / n
        res = Layer(router, w1, w2).run(x, g, PAD)
        want_out, want = exact(router, w1, w2, x, g, res[1])
        assert (res[1][n - PAD:] == -1).all() and (res[1][:n - PAD] >= 0).all()
        got = [res[2], *res[3], *res[4], res[5]]
        # Sums of at most n terms, and of at most 64 in each of the four products on the way
        # there; a square doubles what comes in, and a router's logit enters an
        # exponential and a difference: eight times (n + 256) roundings of the largest value.
        for a, b in zip([res[0], *got], [want_out, *want]):
            scale = b.abs().max()
            assert (a.double().cpu() - b).abs().max() <= (n + 256) * U * scale * 8
        results.append(res)
    # The router's gradient goes through the averaged arena, the experts' are summed over
    # the ranks' tokens by their owner and counted in the same norm.
    arenas = [res[2].reshape(-1).contiguous() for res in results]
    for c, mean in zip(pipe.chunks, pipe.means):
        grz.dp_reduce_scatter_mean(arenas, buckets, c, mean, pipe.norm.partials)
    experts = [a + b for a, b in zip(results[0][3] + results[0][4],
                                     results[1][3] + results[1][4])]
    grads = grz.TensorList(experts)
    ws = torch.empty(grz.dp_grad_sqnorm_tensors_workspace(grads, lead) // 8, device=DEV,
                     dtype=torch.float64)
    ws[:lead].copy_(pipe.norm.partials[:lead])
    grz.dp_grad_sqnorm_tensors(grads, hyper.max_norm, ws, pipe.norm.sqnorm, pipe.norm.scale,
                               lead=lead)
    mean = (arenas[0].double() + arenas[1].double()) / 2
    sq = float((mean ** 2).sum()) + sum(float((t.double() ** 2).sum()) for t in experts)
    # the mean's own roundings: two a value
    assert abs(pipe.norm.sqnorm.item() - sq) <= 8 * U * sq
    factor = pipe.norm.scale.item()
    assert factor < 1.0 and abs(factor - hyper.max_norm / sq ** 0.5) <= 8 * U * factor
    old = [t.clone() for t in experts]
    grz.dp_grad_clip_tensors(grads, pipe.norm.scale)
    for t, o in zip(experts, old):
        assert torch.equal(t, o * pipe.norm.scale)
    # One more norm, of what was clipped: the arena's pieces scaled by hand.
    ws[:lead].mul_(factor ** 2)
    sq2, sc2 = torch.empty_like(pipe.norm.sqnorm), torch.empty_like(pipe.norm.scale)
    grz.dp_grad_sqnorm_tensors(grads, 0.0, ws, sq2, sc2, lead=lead)
    assert abs(sq2.item() ** 0.5 - hyper.max_norm) <= 8 * U * hyper.max_norm
    assert sc2.item() == 1.0
    # AdamW takes the factor; the router moves on every rank alike.
    args = grz.adamw_args(**grz.step_scalars(hyper, 1))
    for c, (w, m, v), mu in zip(pipe.chunks, pipe.state, pipe.means):
        grz.zero1_adamw_gather(w, m, v, mu, buckets, ranks, c, pipe.norm.scale, args,
                               pipe.replicas)
    assert torch.equal(pipe.replicas[0], pipe.replicas[1])
    assert not torch.equal(pipe.replicas[0], router.reshape(-1).to(BF16))
    for t in experts:  # and so do the experts, unclipped gradients with the same factor
        w, m, v = (torch.zeros(t.numel(), device=DEV) for _ in range(3))
        grz.zero1_adamw_step(w, m, v, t.reshape(-1), None, args)
        assert torch.isfinite(w).all() and (w != 0).any()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_go_there_and_back(dtype):
    # Dispatch and combine with weights that sum to 1 give the tokens back: k products and
    # a sum, (k + 1) roundings and the weights' own.
    n, e, k, d = 3000, 40, 6, 300
    logits = torch.randn(n, e, device=DEV, generator=gen(50))
    x = torch.randn(n, d, device=DEV, generator=gen(51)).to(dtype)
    ids, w = torch.empty(n, k, device=DEV, dtype=I32), torch.empty(n, k, device=DEV)
    grz.dp_expert_route(logits, ids, w, normalize=True)
    offsets, places = torch.empty(e + 1, device=DEV, dtype=I32), torch.empty_like(ids)
    ws = torch.empty(grz.dp_expert_sort_workspace(n, k, e), device=DEV, dtype=torch.uint8)
    grz.dp_expert_sort(ids, e, offsets, places, ws)
    rows = torch.empty(n * k, d, device=DEV, dtype=dtype)
    grz.dp_expert_dispatch(x, places, rows)
    # each expert's rows are its tokens', in order
    at = offsets.tolist()
    for one in (0, e // 2, e - 1):
        mine = (ids == one).any(1)
        assert torch.equal(rows[at[one]:at[one + 1]], x[mine])
    back = torch.empty(n, d, device=DEV)
    grz.dp_expert_combine(rows, places, back, weights=w)
    r = ref.Route(logits, ids, True)
    lim = (3 * k + 4) * U + r.rel.max().item()
    assert ((back - x.float()).abs() <= lim * x.float().abs()).all()
    # and without weights k times the token
    grz.dp_expert_combine(rows, places, back)
    assert ((back - k * x.float()).abs() <= k * k * U * x.float().abs()).all()
