"""Token operators on the GPU: orders, layouts and uses at the edges of what their
entry points promise."""

import math

import pytest
import torch

import gradient_reduce_zero_amd as grz
import token_ref as ref
from test_gpu_tokens import (BF16, DEV, F32, grad_call, logits_of, logprob_call, matrix, order_of,
                             outside_untouched)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("v", [1, 2, 65, 100, 128, 129, 600, 3000, 33000, 70001])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_top_list_of_rows_with_a_nan_at_the_first_token(v, dtype):
    # NaN counts as largest, ties by lower id, up to the whole vocabulary.
    x = logits_of(6, v, dtype)
    x[0, 0] = math.nan
    x[1].fill_(math.nan)
    x[2, 0] = -math.nan                                # either sign
    x[2, v // 2] = math.nan
    x[3].fill_(-math.inf)
    x[3, 0] = math.nan
    x[4].fill_(math.inf)
    x[4, 0] = x[4, v - 1] = math.nan
    x[5, v - 1] = math.nan
    t = torch.zeros(6, device=DEV, dtype=torch.long)
    for top in {1, min(v, 3), min(v, 64), min(v, grz.GRZ_MAX_TOP)}:
        lp, h, ids, tl = logprob_call(x, t, top)
        assert torch.equal(ids.cpu().long(), order_of(x, top)), top
        assert torch.isnan(lp).all() and torch.isnan(h).all() and torch.isnan(tl).all()


@pytest.mark.parametrize("v", [65, 3000, 33000])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_values_written_over_the_ones_that_come_in(v, dtype):
    # One value a row: its row has read what came in before it writes.
    n, k = 2000 if v < 33000 else 600, 5
    g = torch.Generator(device=DEV).manual_seed(80)
    x = logits_of(n, v, dtype)
    t = torch.randint(-1, v, (n,), device=DEV, generator=g)
    a, b = (torch.randn(n, device=DEV, generator=g) for _ in range(2))
    a[::7] = 0.0
    b[::7] = 0.0
    dx, lp, h = torch.empty_like(x), torch.empty(n, device=DEV), torch.empty(n, device=DEV)
    grz.dp_token_logprobs_grad(x, t, a, b, dx, logprob=lp, entropy=h)
    for first in (False, True):  # each value over either one
        a2, b2, dx2 = a.clone(), b.clone(), torch.empty_like(x)
        lp2, h2 = (a2, b2) if first else (b2, a2)
        grz.dp_token_logprobs_grad(x, t, a2, b2, dx2, logprob=lp2, entropy=h2)
        assert torch.equal(dx2, dx) and torch.equal(lp2, lp) and torch.equal(h2, h)
    ids = torch.randint(-1, v, (n, k), device=DEV, generator=g)
    z = torch.randn(n, k, device=DEV, generator=g)
    loss, only = torch.empty(n, device=DEV), torch.empty(n, device=DEV)
    grz.dp_distill_grad(x, ids, z, dx, temperature=2.0, weights=a, loss=loss)
    grz.dp_distill_loss(x, ids, z, only, temperature=2.0, weights=a)
    w, dx2 = a.clone(), torch.empty_like(x)
    grz.dp_distill_grad(x, ids, z, dx2, temperature=2.0, weights=w, loss=w)
    assert torch.equal(dx2, dx) and torch.equal(w, loss)
    w = a.clone()
    grz.dp_distill_loss(x, ids, z, w, temperature=2.0, weights=w)
    assert torch.equal(w, only)


def test_arrays_between_the_rows_of_the_logits():
    # What lies between a matrix's rows is the caller's, its lists among it.
    n, v, stride, k = 3, 1000, 1064, 4
    buf = torch.zeros(n * stride, device=DEV)
    x = torch.as_strided(buf, (n, v), (stride, 1))
    x.copy_(logits_of(n, v, F32))

    def gap(row, at, *shape):
        return torch.as_strided(buf, shape, (shape[1], 1) if len(shape) == 2 else (1,),
                                row * stride + v + at)

    loss, w, z = gap(0, 0, n), gap(0, 60, n), gap(1, 50, n, k)
    lp, h, tl = gap(1, 0, n), gap(1, 4, n), gap(1, 10, n, k)
    w.fill_(1.5)
    z.normal_()
    ids = torch.arange(n * k, device=DEV).view(n, k)
    t = torch.arange(n, device=DEV)
    want = [torch.empty(n, device=DEV) for _ in range(3)]
    top, top2 = (torch.empty(n, k, device=DEV, dtype=torch.int32) for _ in range(2))
    wtl, dx = torch.empty(n, k, device=DEV), torch.empty(n, v, device=DEV)
    y = x.clone()
    grz.dp_token_logprobs(y, t, want[0], want[1], top, wtl)
    grz.dp_distill_grad(y, ids, z.clone(), dx, weights=w.clone(), loss=want[2])
    grz.dp_token_logprobs(x, t, lp, h, top2, tl)
    assert torch.equal(top, top2)
    grz.dp_distill_grad(x, ids, z, x, weights=w, loss=loss)
    for got, one in ((lp, want[0]), (h, want[1]), (tl, wtl), (loss, want[2]), (x, dx)):
        assert torch.equal(got, one)
    with pytest.raises(grz.GrzError):  # one place further it reaches the next row
        grz.dp_distill_grad(x, ids, z, x, weights=w, loss=gap(0, 62, n))


@pytest.mark.parametrize("n", [32769, 65536, 65537, 262145])
@pytest.mark.parametrize("vocab", [262143, 262144, 300000])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embed_grad_of_many_ids_into_large_tables(n, vocab, accumulate):
    # On both sides of where the ids' digits take a third pass of the sort, and of
    # where its tiles grow and their counts are summed by a launch of their own.
    dim = 4
    g = torch.Generator(device=DEV).manual_seed(90)
    ids = torch.randint(-1, vocab, (n,), device=DEV, generator=g)
    ids[torch.rand(n, device=DEV, generator=g) < 0.2] = vocab - 1
    ids[n // 2] = 0
    ids[n // 3] = vocab
    dout, _ = matrix(n, dim, F32, seed=91)
    table, buf = matrix(vocab, dim, F32, seed=92, pad=4, shift=4)
    before, old = buf.clone(), table.clone()
    grad_call(dout, ids, table, scale=0.5, accumulate=accumulate)
    want, tol = ref.embed_grad(dout, ids, vocab, 0.5, old if accumulate else None)
    ref.assert_close(table, want, tol, "dtable")
    assert outside_untouched(table, buf, before)
    again = old.clone()
    grad_call(dout, ids.int(), again, scale=0.5, accumulate=accumulate)
    ref.assert_close(again, want, tol, "int32 ids")


@pytest.mark.parametrize("n", [3, 4097, 40000])
def test_embed_grad_into_the_largest_table(n):
    # 2^26 rows, the most that are taken: keys of 27 bits.
    vocab = 2 ** 26
    g = torch.Generator(device=DEV).manual_seed(93)
    ids = torch.randint(0, vocab, (n,), device=DEV, generator=g)
    ids[0], ids[-1], ids[n // 2] = vocab - 1, 0, vocab
    dout, _ = matrix(n, 1, F32, seed=94)
    table = torch.full((vocab, 1), 7.0, device=DEV)
    grad_call(dout, ids, table)
    named, place = torch.unique(ids[ids < vocab], return_inverse=True)
    small = torch.full_like(ids, -1)
    small[ids < vocab] = place
    want, tol = ref.embed_grad(dout, small, len(named), 1.0)
    ref.assert_close(table[named], want, tol, "named rows")
    table[named] = 0.0
    assert (table == 0).all()
