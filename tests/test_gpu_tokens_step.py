"""The token operators together, as a data-parallel step uses them: each rank
looks its tokens up in its weight replica, the loss over the vocabulary gives the
logits' gradients, the head's and the embedding's gradients land in the rank's
gradient arena, and the token-weighted ZeRO-1 step reduces, clips, updates and
writes the next replicas.  The reduced gradient is compared with that of the
whole batch's mean loss in 64 bits."""

import pytest
import torch

import gradient_reduce_zero_amd as grz
import token_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
VOCAB, DIM, NRANKS, PAD = 131, 48, 2, 7
OFFSET = 16                                     # the table's place in the arena
NUMEL = OFFSET + VOCAB * DIM + 16
BUCKETS = [(NUMEL // 2, NUMEL // 2), (0, NUMEL // 2)]
SCALE = DIM ** 0.5


def table_of(arena):
    return arena[OFFSET:OFFSET + VOCAB * DIM].view(VOCAB, DIM)


def rank_tokens(step, rank):
    """Ids and next ids of a padded batch of unequal length."""
    g = torch.Generator(device=DEV).manual_seed(100 * step + rank)
    n = 150 + 61 * rank
    ids = torch.randint(0, VOCAB, (n,), device=DEV, generator=g)
    ids[::3] = 5                                # a frequent token
    ids[-PAD:] = -1
    target = torch.roll(ids, -1)
    target[-PAD - 1:] = -1
    return ids, target


def rank_gradient(replica, ids, target, arena):
    """Sum over the rank's tokens of the loss's gradient, into ``arena``; the loss
    and the tokens' number."""
    n, w = ids.numel(), table_of(replica)
    arena.zero_()
    grad = table_of(arena)
    hidden = torch.empty(n, DIM, device=DEV)
    grz.dp_embed_lookup(w, ids, hidden, scale=SCALE)
    logits = hidden @ w.float().t()
    weight = (target >= 0).float()
    loss = torch.empty(n, device=DEV)
    grz.dp_distill_grad(logits, target[:, None].contiguous(), torch.zeros(n, 1, device=DEV),
                        logits, weights=weight, loss=loss)      # in place: d(logits)
    grad.copy_(logits.t() @ hidden)                             # the tied head
    dhidden = logits @ w.float()
    ws = torch.empty(grz.dp_embed_grad_workspace(n, VOCAB, DIM), device=DEV, dtype=torch.uint8)
    grz.dp_embed_grad(dhidden, ids, grad, ws, scale=SCALE, accumulate=True)
    return loss.double().sum().item(), int(weight.sum().item())


def whole_batch(replica, batches):
    """Mean loss of all ranks' tokens, its gradient, and a bound for an fp32 one."""
    w = table_of(replica).detach().double().cpu().requires_grad_(True)
    ids = torch.cat([b[0] for b in batches]).cpu()
    target = torch.cat([b[1] for b in batches]).cpu()
    ok, live = ids >= 0, target >= 0
    hidden = torch.where(ok[:, None], w[ids.clamp(min=0)] * SCALE, torch.zeros(1, dtype=w.dtype))
    logits = hidden @ w.t()
    lq = torch.log_softmax(logits, 1)
    count = int(live.sum())
    loss = -(lq.gather(1, target.clamp(min=0)[:, None])[:, 0] * live).sum() / count
    loss.backward()
    # Magnitudes: every product and sum below is one of the fp32 path's, so its
    # error is at most (terms of the sums + the softmax's) roundings of these.
    with torch.no_grad():
        a, h = w.abs(), hidden.abs()
        hot = torch.zeros_like(logits).scatter_(1, target.clamp(min=0)[:, None], 1.0)
        d = ((lq.exp() + hot) * live[:, None]) / count
        mag = d.t() @ h
        mag.index_add_(0, ids[ok], (d @ a)[ok] * SCALE)
        # logits: DIM products, so their absolute error enters the exponentials
        off = (DIM + 2) * ref.U * (h @ a.t()).max() * 2
        terms = len(ids) + VOCAB + DIM + ref.depth(VOCAB) + 40
        each = off + ref.Softmax(logits).tol.max()      # of one token's log q
        tol = mag * (terms * ref.U + 2 * each)
        loss_tol = each + len(ids) * ref.U * loss
    return loss.item(), float(loss_tol), w.grad, tol


def test_tokens_to_the_next_weights():
    g = torch.Generator(device=DEV).manual_seed(1)
    master = torch.randn(NUMEL, device=DEV, generator=g) * 0.05
    hyper = grz.Hyper(max_norm=0.0, weight_decay=0.0)
    pipe = grz.Zero1AllRanks(BUCKETS, NRANKS, master, hyper, device=DEV)
    arenas = [torch.zeros(NUMEL, device=DEV) for _ in range(NRANKS)]
    for step in (1, 2, 3):
        batches = [rank_tokens(step, r) for r in range(NRANKS)]
        before = pipe.replicas[0].clone()
        want_loss, loss_tol, want, tol = whole_batch(before, batches)
        sums = [rank_gradient(pipe.replicas[r], *batches[r], arenas[r]) for r in range(NRANKS)]
        counts = [c for _, c in sums]
        assert sum(counts) == sum(int((t >= 0).sum()) for _, t in batches)
        loss = sum(s for s, _ in sums) / sum(counts)
        assert abs(loss - want_loss) <= loss_tol
        pipe.step(arenas, step, token_counts=counts)
        # The ranks' shards of the mean back at their arena places.
        mean = torch.zeros(NUMEL, device=DEV)
        for r, part in enumerate(pipe.means):
            c, at = grz.owned_chunk(r, NRANKS), 0
            for off, length in BUCKETS:
                lo, cnt = grz.dp_chunk_range(length, NRANKS, c)
                mean[off + lo:off + lo + cnt] = part[at:at + cnt]
                at += cnt
        ref.assert_close(table_of(mean), want, tol, f"step {step}: mean gradient")
        assert (mean[:OFFSET] == 0).all() and (mean[OFFSET + VOCAB * DIM:] == 0).all()
        # The next lookup reads what the step wrote, on every rank.
        assert torch.equal(pipe.replicas[0], pipe.replicas[1])
        assert not torch.equal(pipe.replicas[0], before)
        ids = batches[0][0]
        out = torch.empty(ids.numel(), DIM, device=DEV, dtype=torch.bfloat16)
        grz.dp_embed_lookup(table_of(pipe.replicas[1]), ids, out)
        assert torch.equal(out[ids >= 0], table_of(pipe.replicas[0])[ids[ids >= 0]])
        assert (out[ids < 0] == 0).all()


def test_a_teachers_top_list_is_distilled():
    # The teacher's list is the student's input; with the list as long as the
    # vocabulary the loss is the whole divergence, and 0 for equal models.
    n, k = 37, VOCAB - 3
    g = torch.Generator(device=DEV).manual_seed(3)
    teacher = torch.randn(n, VOCAB, device=DEV, generator=g) * 2
    ids = torch.empty(n, k, device=DEV, dtype=torch.int32)
    logq = torch.empty(n, k, device=DEV)
    grz.dp_token_logprobs(teacher, top_ids=ids, top_logprobs=logq)
    student = teacher + 0.5 * torch.randn(n, VOCAB, device=DEV, generator=g)
    loss, dx = torch.empty(n, device=DEV), torch.empty_like(student)
    grz.dp_distill_grad(student, ids, logq, dx, temperature=2.0, loss=loss)
    # From the teacher's logits instead of their log probabilities: the same p, up
    # to the roundings of log q (half a step of |log q| and of the logits' own).
    z = teacher.gather(1, ids.long())
    d = ref.Distill(student, ids, z, 2.0)
    extra = ref.Softmax(teacher).tol.max() + 2 * ref.U * logq.abs().max().item()
    lq = torch.log_softmax(student.double().cpu() / 2, 1)
    ref.assert_close(loss, d.loss, d.loss_tol + 4 * 2 * extra * (lq.abs().max() + 10), "loss")
    ref.assert_close(dx, d.dx, d.dx_tol + 2 * 2 * extra, "dlogits")
