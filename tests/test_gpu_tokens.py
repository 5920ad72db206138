"""Token operators on the GPU against their 64-bit forms (tests/token_ref.py)."""

import math

import pytest
import torch

import gradient_reduce_zero_amd as grz
import token_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, F32 = torch.bfloat16, torch.float32
LOWEST = {BF16: torch.finfo(BF16).min, F32: torch.finfo(F32).min}


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def matrix(rows, cols, dtype, seed=0, pad=0, shift=0, std=1.0, fill=None):
    """A rows x cols matrix whose rows lie ``cols + pad`` apart and whose first
    element lies ``shift`` elements into its buffer (filled with ``fill``)."""
    stride = cols + pad
    buf = torch.full((rows * stride + shift + 16,), float("nan") if fill is None else fill,
                     device=DEV, dtype=dtype)
    view = buf[shift:shift + rows * stride].view(rows, stride)[:, :cols]
    if std is not None:
        view.copy_(torch.randn(rows, cols, device=DEV, generator=gen(seed)) * std)
    return view, buf


def outside_untouched(view, buf, before):
    """The buffer around the view holds what it held."""
    inside = torch.zeros_like(buf, dtype=torch.bool)
    torch.as_strided(inside, view.shape, view.stride(), view.storage_offset()).fill_(True)
    a, b = buf[~inside], before[~inside]
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def token_ids(n, vocab, seed, bits=64, pads=True):
    u = torch.rand(n, device=DEV, generator=gen(seed), dtype=torch.float64)
    t = (torch.exp(u * math.log(vocab + 1.0)) - 1).long().clamp_(0, max(vocab - 1, 0))
    if pads and n > 3:
        t[n // 3] = -100
        t[n // 2] = vocab
    if vocab == 0:
        t.fill_(-1)
    return t if bits == 64 else t.int()


# -- lookup ------------------------------------------------------------------------

@pytest.mark.parametrize("n,vocab,dim", [(0, 5, 8), (1, 1, 1), (1, 65, 384), (7, 3, 5),
                                         (257, 65, 384), (33, 101, 385), (5, 50, 4100),
                                         (4, 9, 68)])
@pytest.mark.parametrize("ti,to", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 8), (3, 1)])
def test_lookup(n, vocab, dim, ti, to, pad, shift):
    table, _ = matrix(vocab, dim, ti, seed=1, pad=pad, shift=shift)
    out, buf = matrix(n, dim, to, pad=pad, shift=shift, std=None)
    before = buf.clone()
    for bits, scale in ((64, 1.0), (32, math.sqrt(dim))):
        ids = token_ids(n, vocab, 2, bits)
        grz.dp_embed_lookup(table, ids, out, scale=scale)
        ok = (ids >= 0) & (ids < vocab)
        s = torch.tensor(scale, dtype=F32, device=DEV)
        want = table[torch.where(ok, ids, torch.zeros_like(ids)).long()].float() * s
        want = torch.where(ok[:, None], want, torch.zeros_like(want)).to(to)
        assert torch.equal(out, want)  # one fp32 product, one rounding
        assert outside_untouched(out, buf, before)


def test_lookup_beyond_32_bit_offsets():
    # Rows 2^31 + 8 elements apart: the last row starts past 2^32 elements.
    stride = 2 ** 31 + 8
    buf = torch.empty(2 * stride + 64, device=DEV, dtype=BF16)
    table = torch.as_strided(buf, (3, 64), (stride, 1))
    table.copy_(torch.randn(3, 64, device=DEV, generator=gen(3)))
    out = torch.empty(4, 64, device=DEV, dtype=BF16)
    ids = torch.tensor([2, 0, 1, 2], device=DEV)
    grz.dp_embed_lookup(table, ids, out)
    assert torch.equal(out, table[ids])
    # The gradient reads rows and adds to rows that far apart.
    ws = torch.empty(grz.dp_embed_grad_workspace(3, 3, 64), device=DEV, dtype=torch.uint8)
    small = torch.zeros(3, 64, device=DEV, dtype=BF16)
    grz.dp_embed_grad(table, torch.tensor([1, 1, 0], device=DEV), small, ws)
    want, tol = ref.embed_grad(table, torch.tensor([1, 1, 0]), 3, 1.0)
    ref.assert_close(small, want, tol, "gradient of far rows")
    old = table.clone()
    grz.dp_embed_grad(out, ids, table, torch.empty(grz.dp_embed_grad_workspace(4, 3, 64),
                                                   device=DEV, dtype=torch.uint8),
                      accumulate=True)
    want, tol = ref.embed_grad(out, ids, 3, 1.0, old)
    ref.assert_close(table, want, tol, "gradient into far rows")


# -- gradient ------------------------------------------------------------------------

def grad_call(dout, ids, table, **kw):
    ws = torch.full((max(1, grz.dp_embed_grad_workspace(*dout.shape[:1], *table.shape)),), 0xA5,
                    device=DEV, dtype=torch.uint8)
    grz.dp_embed_grad(dout, ids, table, ws, **kw)


@pytest.mark.parametrize("n,vocab,dim", [(0, 5, 8), (1, 1, 1), (1, 65, 384), (2, 7, 5),
                                         (31, 3, 4), (32, 1, 8), (33, 1, 8), (65, 2, 260),
                                         (300, 65, 385), (4096, 600, 12), (4097, 65, 20),
                                         (9001, 50257, 16), (5000, 70000, 3),
                                         (4100, 300000, 4)])
@pytest.mark.parametrize("ti,to", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embed_grad(n, vocab, dim, ti, to, accumulate):
    for pad, shift, bits, scale in ((0, 0, 64, 1.0), (4, 4, 32, 0.5), (3, 1, 64, 27.7)):
        dout, _ = matrix(n, dim, ti, seed=4, pad=pad, shift=shift)
        ids = token_ids(n, vocab, 5, bits)
        table, buf = matrix(vocab, dim, to, seed=6, pad=pad, shift=shift)
        before, old = buf.clone(), table.clone()
        grad_call(dout, ids, table, scale=scale, accumulate=accumulate)
        want, tol = ref.embed_grad(dout, ids, vocab, float(torch.tensor(scale, dtype=F32)),
                                   old if accumulate else None)
        ref.assert_close(table, want, tol, f"pad {pad} scale {scale}")
        assert outside_untouched(table, buf, before)
        if accumulate:  # rows that no id names keep their bits
            named = torch.zeros(vocab, dtype=torch.bool, device=DEV)
            ok = (ids >= 0) & (ids < vocab)
            named[ids[ok].long()] = True
            assert torch.equal(table[~named], old[~named])


@pytest.mark.parametrize("n", [1, 31, 32, 63, 64, 65, 1000, 20000])
@pytest.mark.parametrize("which", ["one", "none", "all_but_one", "last"])
def test_embed_grad_of_repeated_and_absent_ids(n, which):
    vocab, dim = 40, 24
    ids = torch.full((n,), 7, device=DEV)
    if which == "none":
        ids.fill_(-1)
    elif which == "all_but_one":
        ids[n // 2] = 11
    elif which == "last":
        ids.fill_(vocab - 1)
        ids[: n // 2] = vocab
    dout, _ = matrix(n, dim, F32, seed=8)
    table, _ = matrix(vocab, dim, F32, seed=9)
    grad_call(dout, ids, table)
    want, tol = ref.embed_grad(dout, ids, vocab, 1.0)
    ref.assert_close(table, want, tol, which)


@pytest.mark.parametrize("n", [255, 257, 4095, 4097, 8191, 16385, 32768, 32769, 40003, 131073, 262145, 300007, 524289, 700001])
@pytest.mark.parametrize("vocab", [3, 700, 150000])
def test_embed_grad_of_many_ids(n, vocab):
    # Every way the digit counts are formed, every chunk length, runs over many
    # chunks: a third of the ids the same, a tenth of no row.
    dim = 4
    ids = token_ids(n, vocab, 5)
    u = torch.rand(n, device=DEV, generator=gen(7))
    ids[u < 0.33] = vocab // 2
    ids[u > 0.9] = -1
    dout, _ = matrix(n, dim, F32, seed=4)
    table, _ = matrix(vocab, dim, F32, seed=6)
    grad_call(dout, ids, table, scale=0.5)
    want, tol = ref.embed_grad(dout, ids, vocab, 0.5)
    ref.assert_close(table, want, tol, "dtable")


@pytest.mark.parametrize("n,vocab,dim", [(2080, 65, 384), (2081, 65, 384), (4096, 128, 1024),
                                         (4096, 128, 1028), (4097, 300, 8), (513, 17, 63),
                                         (64, 2, 5), (65, 2, 5), (4095, 512, 256)])
@pytest.mark.parametrize("ti,to", [(BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embed_grad_of_small_tables(n, vocab, dim, ti, to, accumulate):
    # On both sides of where a small table is summed without a sort; rows that no
    # id names, one that half of them name.
    ids = token_ids(n, vocab, 17)
    ids[: n // 2] = vocab - 1
    ids[ids == 1] = 0
    dout, _ = matrix(n, dim, ti, seed=18)
    table, buf = matrix(vocab, dim, to, seed=19, pad=3, shift=1)
    before, old = buf.clone(), table.clone()
    grad_call(dout, ids, table, scale=1.25, accumulate=accumulate)
    want, tol = ref.embed_grad(dout, ids, vocab, 1.25, old if accumulate else None)
    ref.assert_close(table, want, tol, "dtable")
    assert outside_untouched(table, buf, before)
    if accumulate:
        assert torch.equal(table[1].view(torch.uint8), old[1].view(torch.uint8))
    again = old.clone()
    grad_call(dout, ids, again, scale=1.25, accumulate=accumulate)
    ref.assert_close(again, want, tol, "another layout")


def test_embed_grad_bits_do_not_change_and_follow_the_rows():
    n, vocab, dim = 20011, 1000, 64
    dout, _ = matrix(n, dim, BF16, seed=10)
    ids = token_ids(n, vocab, 11)
    a, b = (torch.empty(vocab, dim, device=DEV) for _ in range(2))
    grad_call(dout, ids, a)
    grad_call(dout, ids, b)
    assert torch.equal(a.view(torch.int32), b.view(torch.int32))
    grad_call(dout.clone(), ids.int(), b)
    assert torch.equal(a.view(torch.int32), b.view(torch.int32))


def test_embed_grad_is_the_lookups_gradient_by_differences():
    # L = sum(c * lookup(T)): linear in T, so a difference quotient is exact up
    # to roundings; scale and ids as in the forward call.
    n, vocab, dim, scale = 50, 9, 6, 1.5
    table, _ = matrix(vocab, dim, F32, seed=12)
    c, _ = matrix(n, dim, F32, seed=13)
    ids = token_ids(n, vocab, 14)
    g = torch.empty(vocab, dim, device=DEV)
    grad_call(c, ids, g, scale=scale)

    def loss(t):
        out = torch.empty(n, dim, device=DEV)
        grz.dp_embed_lookup(t, ids, out, scale=scale)
        return (out.double() * c.double()).sum().item()

    base = loss(table)
    for v, d in ((0, 0), (1, 3), (8, 5), (4, 2)):
        t = table.clone()
        t[v, d] += 2.0 ** 10
        # each output is off by u (|T| + 2^10) scale, n outputs
        lim = 4 * ref.U * scale * (2 ** 10 + 8) * c.abs().double()[:, d].sum().item() / 2 ** 10
        lim += (n + 4) * ref.U * scale * c.abs().double()[:, d].sum().item()
        step = t[v, d].double().item() - table[v, d].double().item()
        assert abs((loss(t) - base) / step - g[v, d].item()) <= lim + 1e-9


# -- log probabilities -------------------------------------------------------------------

ROWS = [(1, 1), (3, 2), (2, 7), (5, 8), (4, 65), (3, 1000), (2, 2048), (3, 4097), (2, 16391),
        (2, 32000), (3, 50257), (2, 65537), (1, 131075), (1, 300001)]


def logits_of(n, v, dtype, seed=20, pad=0, shift=0, std=3.0):
    x, buf = matrix(n, v, dtype, seed=seed, pad=pad, shift=shift, std=std)
    return x


def order_of(x, k):
    """Top k by value, ties by lower index, NaN first, on the host."""
    key = x.detach().cpu().float()
    return torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]


def logprob_call(x, targets, top):
    n = x.shape[0]
    lp, h = torch.full((n,), 9.0, device=DEV), torch.full((n,), 9.0, device=DEV)
    ids = torch.full((n, top), -7, device=DEV, dtype=torch.int32)
    tl = torch.full((n, top), 9.0, device=DEV)
    grz.dp_token_logprobs(x, targets, lp, h, ids, tl)
    return lp, h, ids, tl


def check_logprobs(x, targets, top, what):
    lp, h, ids, tl = logprob_call(x, targets, top)
    sm = ref.Softmax(x)
    v = x.shape[1]
    t = targets.cpu().long()
    ok = (t >= 0) & (t < v)
    at = t.clamp(0, v - 1)[:, None]
    zero = torch.zeros(len(t), dtype=torch.float64)
    ref.assert_close(lp, torch.where(ok, sm.lq.gather(1, at)[:, 0], zero),
                     torch.where(ok, sm.tol.gather(1, at)[:, 0], zero), what + " logprob")
    want, tol = sm.entropy()
    ref.assert_close(h, want, tol, what + " entropy")
    order = order_of(x, top)
    assert torch.equal(ids.cpu().long(), order), what + " top ids"
    ref.assert_close(tl, sm.lq.gather(1, order), sm.tol.gather(1, order), what + " top logprobs")


@pytest.mark.parametrize("n,v", ROWS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pad,shift", [(0, 0), (5, 3)])
def test_logprobs(n, v, dtype, pad, shift):
    x = logits_of(n, v, dtype, pad=pad, shift=shift)
    for bits, top in ((64, min(v, 20)), (32, min(v, grz.GRZ_MAX_TOP)), (64, 0)):
        targets = token_ids(n, v, 21, bits)
        targets[-1] = v - 1
        check_logprobs(x, targets, top, f"top {top}")


@pytest.mark.parametrize("v", [65, 3000, 33000])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_logprobs_of_ties_and_masks(v, dtype):
    top = 33
    x = logits_of(10, v, dtype)
    x[0].fill_(1.5)                                    # every token alike
    x[1].fill_(-math.inf)
    x[1, v // 2] = 2.0                                 # one allowed token
    x[2, ::2] = -math.inf                              # half masked
    x[3].fill_(LOWEST[dtype])                          # all at the type's lowest
    x[4].fill_(LOWEST[dtype])
    x[4, 5] = 1.0
    x[5] = torch.round(x[5])                           # few distinct values
    x[6].fill_(0.0)
    x[6, ::3] = -0.0                                   # zeros of both signs tie
    x[7, 3] = 300.0                                    # all the probability on one token
    x[8] = x[8] + 1000.0                               # far from zero
    x[9] = x[9] * 1e-3
    targets = torch.full((10,), 5, device=DEV)
    targets[1] = v // 2
    check_logprobs(x, targets, top, "rows")
    targets[1] = 0                                     # a masked target: log 0
    assert logprob_call(x, targets, 0)[0][1].item() == -math.inf


@pytest.mark.parametrize("v", [65, 3000, 33000])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_logprobs_of_huge_logits(v, dtype):
    # Rows far from zero, whose differences are few steps of the type or none.
    x = logits_of(8, v, dtype)
    for i, at in enumerate((3e4, 6e5, 7e5, -8e5, 1e8, -1e10, 1e20, 3e37)):
        x[i] = at * (1 + torch.randint(0, 3, (v,), device=DEV, generator=gen(i)) *
                     torch.finfo(dtype).eps)
    targets = torch.arange(8, device=DEV)
    check_logprobs(x, targets, 5, "huge")
    glp = torch.linspace(-1, 1, 8, device=DEV)
    gent = torch.linspace(0.5, -0.5, 8, device=DEV)
    dx = torch.empty_like(x)
    grz.dp_token_logprobs_grad(x, targets, glp, gent, dx)
    want, tol = ref.logprob_grad(x, targets, glp, gent)
    ref.assert_close(dx, want, tol, "dlogits")


@pytest.mark.parametrize("v", [65, 3000, 33000])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_logprobs_of_rows_without_a_softmax(v, dtype):
    x = logits_of(4, v, dtype)
    x[0].fill_(-math.inf)
    x[1, 7] = math.nan
    x[2, 9] = math.inf
    x[2, 11] = math.inf
    lp, h, ids, tl = logprob_call(x, torch.zeros(4, device=DEV, dtype=torch.long), 6)
    assert torch.isnan(lp[:3]).all() and torch.isnan(h[:3]).all() and torch.isnan(tl[:3]).all()
    assert torch.isfinite(lp[3]) and torch.isfinite(h[3])
    assert torch.equal(ids.cpu().long(), order_of(x, 6))
    assert ids[0].tolist() == list(range(6)) and ids[1, 0] == 7 and ids[2, :2].tolist() == [9, 11]


@pytest.mark.parametrize("v,dtype", [(66003, BF16), (33003, F32), (140001, BF16), (70001, F32)])
def test_logprobs_of_long_rows_in_any_order(v, dtype):
    # Rows too long for the registers: their sums follow a maximum that moves.
    x = logits_of(12, v, dtype)
    x[0] = torch.linspace(-60, 60, v, device=DEV).to(dtype)      # it moves all the time
    x[1] = x[0].flip(0)
    x[2, : v - 9] = -math.inf                                    # most threads see masks only
    x[3, : v // 2] = -math.inf                                   # masks first
    x[4, ::2] = LOWEST[dtype]
    x[5].fill_(LOWEST[dtype])
    x[6] = 1e30 * x[6]
    x[7, : v // 2] = -3e38                                       # differences overflow
    x[7, v // 2:] = 3e38
    x[8] = 2.5
    x[9].fill_(-math.inf)
    x[10, v - 2] = math.nan
    x[11, v - 1] = math.inf
    targets = torch.arange(12, device=DEV)
    targets[2] = targets[3] = v - 4
    check_logprobs(x[:9], targets[:9], 25, "rows")
    lp, h, ids, tl = logprob_call(x, targets, 25)
    assert torch.isnan(lp[9:]).all() and torch.isnan(h[9:]).all() and torch.isnan(tl[9:]).all()
    assert torch.equal(ids.cpu().long(), order_of(x, 25))
    glp = torch.linspace(-1, 1, 9, device=DEV)
    gent = torch.linspace(0.5, -0.5, 9, device=DEV)
    dx = torch.empty_like(x[:9])
    grz.dp_token_logprobs_grad(x[:9], targets[:9], glp, gent, dx)
    want, tol = ref.logprob_grad(x[:9], targets[:9], glp, gent)
    ref.assert_close(dx, want, tol, "dlogits")
    k = torch.arange(0, v, v // 30, device=DEV)[:30].expand(9, 30).contiguous()
    keep = [0, 1, 4, 5, 6, 8]                # a listed masked token has no finite loss
    y, k = x[keep].contiguous(), k[keep].contiguous()
    z = torch.randn(len(keep), 30, device=DEV, generator=gen(26))
    loss, dy = torch.empty(len(keep), device=DEV), torch.empty_like(y)
    grz.dp_distill_grad(y, k, z, dy, temperature=2.0, loss=loss)
    d = ref.Distill(y, k, z, 2.0)
    ref.assert_close(loss, d.loss, d.loss_tol, "loss")
    ref.assert_close(dy, d.dx, d.dx_tol, "distillation's dlogits")


def test_logprobs_outputs_may_be_left_out():
    x = logits_of(5, 777, BF16)
    t = token_ids(5, 777, 22)
    lp, h, ids, tl = logprob_call(x, t, 4)
    only = torch.empty(5, device=DEV)
    grz.dp_token_logprobs(x, t, logprob=only)
    assert torch.equal(only, lp)
    grz.dp_token_logprobs(x, entropy=only)
    assert torch.equal(only, h)
    i2, l2 = torch.empty_like(ids), torch.empty_like(tl)
    grz.dp_token_logprobs(x, top_ids=i2, top_logprobs=l2)
    assert torch.equal(i2, ids) and torch.equal(l2, tl)
    grz.dp_token_logprobs(x[:0], t[:0], logprob=only[:0])


@pytest.mark.parametrize("n,v", ROWS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pad,shift,dpad,dshift", [(0, 0, 0, 0), (5, 3, 5, 3), (3, 0, 1, 1)])
def test_logprobs_grad(n, v, dtype, pad, shift, dpad, dshift):
    x = logits_of(n, v, dtype, pad=pad, shift=shift)
    targets = token_ids(n, v, 23)
    targets[0] = v - 1
    glp = torch.randn(n, device=DEV, generator=gen(24))
    gent = torch.randn(n, device=DEV, generator=gen(25)) * 0.3
    for a, b in ((glp, gent), (glp, None), (None, gent)):
        dx, buf = matrix(n, v, dtype, pad=dpad, shift=dshift, std=None)
        before = buf.clone()
        lp, h = torch.empty(n, device=DEV), torch.empty(n, device=DEV)
        grz.dp_token_logprobs_grad(x, targets, a, b, dx, logprob=lp, entropy=h)
        want, tol = ref.logprob_grad(x, targets, a, b)
        ref.assert_close(dx, want, tol, "dlogits")
        assert outside_untouched(dx, buf, before)
        l2, h2, _, _ = logprob_call(x, targets, 0)
        assert torch.equal(lp, l2) and torch.equal(h, h2)
        again = torch.empty(n, v, device=DEV, dtype=dtype)
        grz.dp_token_logprobs_grad(x, targets, a, b, again)
        assert torch.equal(again, dx)
    # In place: within the bound in another layout, the same bits in the same one
    # (the order of a row's sums follows its place on the 16-byte borders).
    inplace = x.clone()
    grz.dp_token_logprobs_grad(inplace, targets, None, gent, inplace)
    ref.assert_close(inplace, want, tol, "in place")
    same = logits_of(n, v, dtype, pad=pad, shift=shift)
    grz.dp_token_logprobs_grad(same, targets, None, gent, same)
    assert torch.equal(same, dx)


def test_logprobs_grad_by_differences():
    n, v, step = 3, 40, 1e-4
    x = logits_of(n, v, F32, std=1.5)
    t = torch.tensor([3, -1, 39], device=DEV)
    glp = torch.tensor([1.0, 2.0, -0.5], device=DEV)
    gent = torch.tensor([0.25, -1.0, 0.5], device=DEV)
    dx = torch.empty_like(x)
    grz.dp_token_logprobs_grad(x, t, glp, gent, dx)

    def value(y, i):
        lq = torch.log_softmax(y[i], 0)
        lp = lq[t[i]] if t[i] >= 0 else 0.0
        return (glp[i].double() * lp - gent[i].double() * (lq.exp() * lq).sum()).item()

    y = x.double()
    for i in range(n):
        for j in (0, 3, 17, 39):
            up, dn = y.clone(), y.clone()
            up[i, j] += step
            dn[i, j] -= step
            # third derivatives of log-sum-exp and of the entropy are below 20 here
            assert abs((value(up, i) - value(dn, i)) / (2 * step) - dx[i, j].item()) < 1e-6


@pytest.mark.parametrize("v", [65, 3000, 33000])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_logprobs_grad_of_masked_rows(v, dtype):
    x = logits_of(8, v, dtype)
    x[0, ::2] = -math.inf
    x[1].fill_(LOWEST[dtype])
    x[2].fill_(-math.inf)
    x[2, 1] = 0.0
    x[3].fill_(math.nan)                               # ignored row: nothing flows back
    x[4].fill_(-math.inf)                              # ignored too
    x[5].fill_(-math.inf)                              # no softmax
    t = torch.tensor([1, 5, 1, -100, v, 1, 3, -100], device=DEV)
    glp = torch.full((8,), -1.0, device=DEV)
    gent = torch.tensor([0.5, 0.5, 0.5, 0.0, 0.0, 0.5, 0.0, 0.0], device=DEV)
    dx = torch.empty_like(x)
    grz.dp_token_logprobs_grad(x, t, glp, gent, dx)
    good = torch.tensor([0, 1, 2, 6])
    want, tol = ref.logprob_grad(x[good], t[good], glp[good], gent[good])
    ref.assert_close(dx[good], want, tol, "masked rows")
    assert (dx[[3, 4, 7]] == 0).all()
    assert torch.isnan(dx[5]).all()
    # the same with the values asked for
    again, lp, h = torch.empty_like(x), torch.empty(8, device=DEV), torch.empty(8, device=DEV)
    grz.dp_token_logprobs_grad(x, t, glp, gent, again, logprob=lp, entropy=h)
    assert torch.equal(again[good], dx[good]) and (again[[3, 4, 7]] == 0).all()
    assert (lp[[3, 4, 7]] == 0).all()


# -- distillation ------------------------------------------------------------------------

def teacher_of(n, v, k, seed, bits, dtype):
    g = gen(seed)
    ids = torch.stack([torch.randperm(v, device=DEV, generator=g)[:k] for _ in range(n)]) \
        if k <= v else torch.randint(0, v, (n, k), device=DEV, generator=g)
    z = (torch.randn(n, k, device=DEV, generator=g) * 2).to(dtype)
    return (ids if bits == 64 else ids.int()), z


def distill_check(x, ids, z, tau, w, what, scale=1.0, dx=None):
    n = x.shape[0]
    d = ref.Distill(x, ids, z, tau, w, scale)
    loss = torch.full((n,), 9.0, device=DEV)
    grz.dp_distill_loss(x, ids, z, loss, temperature=tau, weights=w)
    ref.assert_close(loss, d.loss, d.loss_tol, what + " loss")
    both = torch.full((n,), 9.0, device=DEV)
    dx = torch.empty(n, x.shape[1], device=DEV, dtype=x.dtype) if dx is None else dx
    grz.dp_distill_grad(x, ids, z, dx, temperature=tau, weights=w, grad_scale=scale, loss=both)
    assert torch.equal(both, loss)
    ref.assert_close(dx, d.dx, d.dx_tol, what + " dlogits")
    alone = torch.empty(n, x.shape[1], device=DEV, dtype=x.dtype)
    grz.dp_distill_grad(x, ids, z, alone, temperature=tau, weights=w, grad_scale=scale)
    assert torch.equal(alone, dx)
    return dx, loss


@pytest.mark.parametrize("n,v", ROWS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pad,shift,dpad,dshift", [(0, 0, 0, 0), (5, 3, 5, 3), (3, 0, 1, 1)])
def test_distill(n, v, dtype, pad, shift, dpad, dshift):
    x = logits_of(n, v, dtype, pad=pad, shift=shift)
    w = torch.rand(n, device=DEV, generator=gen(30)) + 0.5
    for k, tau, bits, zt in ((1, 1.0, 64, F32), (min(v, 32), 2.0, 32, BF16),
                             (min(v, 128), 0.7, 64, F32)):
        ids, z = teacher_of(n, v, k, 31, bits, zt)
        dx, buf = matrix(n, v, dtype, pad=dpad, shift=dshift, std=None)
        before = buf.clone()
        distill_check(x, ids, z, tau, w, f"k {k} tau {tau}", scale=0.25, dx=dx)
        assert outside_untouched(dx, buf, before)
        d = ref.Distill(x, ids, z, tau, w, 0.25)
        inplace = x.clone()
        grz.dp_distill_grad(inplace, ids, z, inplace, temperature=tau, weights=w,
                            grad_scale=0.25)
        ref.assert_close(inplace, d.dx, d.dx_tol, "in place")
        same = logits_of(n, v, dtype, pad=pad, shift=shift)
        grz.dp_distill_grad(same, ids, z, same, temperature=tau, weights=w, grad_scale=0.25)
        assert torch.equal(same, dx)


@pytest.mark.parametrize("v", [65, 3000, 33000])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_distill_of_masked_lists_rows_and_weights(v, dtype):
    k = 6
    x = logits_of(9, v, dtype)
    ids, z = teacher_of(9, v, k, 33, 64, F32)
    w = torch.ones(9, device=DEV)
    ids[0, 2:] = -1                          # a short list
    z[0, 2:] = math.nan                      # what stands behind it does not matter
    ids[1, :] = ids[1, 0]                    # one token six times
    ids[2, 3] = ids[2, 0]                    # a token twice
    z[3, 1] = -math.inf                      # an entry of probability 0
    ids[4, :] = v                            # nothing listed
    x[4].fill_(math.nan)
    z[5, :] = -math.inf                      # nothing listed either
    w[6] = 0.0
    x[6].fill_(math.nan)
    x[7, ids[7, 0] - 1] = -math.inf          # a masked token that is not listed
    ids[7] = torch.where(ids[7] == (ids[7, 0] - 1) % v, ids[7, 0], ids[7])
    z[8, :] = LOWEST[F32]                    # a uniform teacher at the type's lowest
    zz = z.clone()
    zz[0, 2:] = 0.0                          # the reference masks by id
    d = ref.Distill(torch.nan_to_num(x, nan=0.0, neginf=-math.inf), ids, zz, 2.0, w)
    loss, dx = torch.full((9,), 9.0, device=DEV), torch.full_like(x, 9.0)
    grz.dp_distill_grad(x, ids, z, dx, temperature=2.0, weights=w, loss=loss)
    ref.assert_close(loss, d.loss, d.loss_tol, "loss")
    ref.assert_close(dx, d.dx, d.dx_tol, "dlogits")
    assert (dx[4:7] == 0).all() and (loss[4:7] == 0).all()
    # a listed token that the student rules out: infinite loss, finite gradient
    x2 = logits_of(1, v, dtype)
    x2[0, 5] = -math.inf
    i2 = torch.tensor([[5, 6]], device=DEV)
    l2, g2 = torch.empty(1, device=DEV), torch.empty_like(x2)
    grz.dp_distill_grad(x2, i2, torch.zeros(1, 2, device=DEV), g2, loss=l2)
    assert l2.item() == math.inf and g2[0, 5].item() == -0.5 and torch.isfinite(g2).all()


@pytest.mark.parametrize("tau", [1e-18, 1e-6, 1e6, 1e18])
def test_distill_at_extreme_temperatures(tau):
    # Cold: all of p and q on one token; hot: both uniform, p over the list.
    n, v, k = 3, 300, 4
    x = logits_of(n, v, F32)
    ids, _ = teacher_of(n, v, k, 38, 64, F32)
    z = x.gather(1, ids).contiguous()
    z[:, 0] += 100.0
    x[0, ids[0, 0]] = 200.0
    loss, dx = torch.empty(n, device=DEV), torch.empty_like(x)
    grz.dp_distill_grad(x, ids, z, dx, temperature=tau, loss=loss)
    t = torch.tensor(tau, dtype=F32).double().item()
    q = torch.softmax(x.double() / t, 1)
    p = torch.zeros_like(q).scatter_add_(1, ids, torch.softmax(z.double() / t, 1))
    assert torch.isfinite(dx).all() and not torch.isnan(loss).any()
    # a softmax's value is off by at most a few u (1 + |x| / T) of itself; here it is 0, 1 or
    # uniform up to 300 / T, so an absolute bound of 1e-4 T holds with room
    assert ((dx.double() - t * (q - p)).abs() <= 1e-4 * t).all()


def test_distill_with_one_token_is_the_cross_entropy():
    n, v = 6, 1000
    x = logits_of(n, v, F32)
    t = torch.arange(n, device=DEV) * 100
    w = torch.rand(n, device=DEV, generator=gen(35))
    loss, dx = torch.empty(n, device=DEV), torch.empty_like(x)
    grz.dp_distill_grad(x, t[:, None], torch.zeros(n, 1, device=DEV), dx, weights=w, loss=loss)
    lp, want = torch.empty(n, device=DEV), torch.empty_like(x)
    grz.dp_token_logprobs_grad(x, t, -w, None, want, logprob=lp)
    sm = ref.Softmax(x)
    tol = (sm.tol.max() * 2).item()
    assert (loss + w * lp).abs().max().item() <= tol
    assert (dx - want).abs().max().item() <= tol


def test_distill_grad_by_differences():
    n, v, k, tau, step = 2, 30, 5, 2.0, 1e-4
    x = logits_of(n, v, F32, std=1.5)
    ids, z = teacher_of(n, v, k, 36, 64, F32)
    w = torch.tensor([0.5, 2.0], device=DEV)
    dx = torch.empty_like(x)
    grz.dp_distill_grad(x, ids, z, dx, temperature=tau, weights=w)

    def value(y, i):
        p = torch.softmax(z[i].double() / tau, 0)
        lq = torch.log_softmax(y[i] / tau, 0)[ids[i]]
        return (w[i].double() * tau ** 2 * (p * (p.log() - lq)).sum()).item()

    y = x.double()
    for i in range(n):
        for j in (0, 1, int(ids[i, 0]), int(ids[i, 4])):
            up, dn = y.clone(), y.clone()
            up[i, j] += step
            dn[i, j] -= step
            assert abs((value(up, i) - value(dn, i)) / (2 * step) - dx[i, j].item()) < 1e-6


# -- streams, graphs, many rows --------------------------------------------------------------

def test_many_rows_of_a_small_vocabulary():
    n, v = 70001, 65
    x = logits_of(n, v, BF16)
    t = token_ids(n, v, 40)
    lp, h, ids, tl = logprob_call(x, t, 3)
    sm = ref.Softmax(x)
    tc = t.cpu()
    ok = (tc >= 0) & (tc < v)
    zero = torch.zeros(n, dtype=torch.float64)
    at = tc.clamp(0, v - 1)[:, None]
    ref.assert_close(lp, torch.where(ok, sm.lq.gather(1, at)[:, 0], zero),
                     torch.where(ok, sm.tol.gather(1, at)[:, 0], zero), "logprob")
    assert torch.equal(ids.cpu().long(), order_of(x, 3))


def _run_all(b):
    grz.dp_embed_lookup(b["table"], b["ids"], b["out"], scale=2.0)
    grz.dp_token_logprobs(b["x"], b["t"], b["lp"], b["h"], b["top"], b["tl"])
    grz.dp_token_logprobs_grad(b["x"], b["t"], b["g"], b["g"], b["dx"])
    grz.dp_distill_grad(b["x"], b["top"], b["tl"], b["dx2"], temperature=2.0, weights=b["g"],
                        loss=b["loss"])
    grz.dp_embed_grad(b["out"], b["ids"], b["dtable"], b["ws"])


def _buffers(seed):
    n, v, d = 700, 1111, 96
    b = {"table": matrix(v, d, BF16, seed=seed)[0], "ids": token_ids(n, v, seed),
         "out": torch.empty(n, d, device=DEV, dtype=BF16), "x": logits_of(n, v, BF16, seed=seed),
         "t": token_ids(n, v, seed + 1), "lp": torch.empty(n, device=DEV),
         "h": torch.empty(n, device=DEV), "top": torch.empty(n, 8, device=DEV, dtype=torch.int32),
         "tl": torch.empty(n, 8, device=DEV), "g": torch.rand(n, device=DEV, generator=gen(seed)),
         "dx": torch.empty(n, v, device=DEV, dtype=BF16),
         "dx2": torch.empty(n, v, device=DEV, dtype=BF16), "loss": torch.empty(n, device=DEV),
         "dtable": torch.empty(v, d, device=DEV),
         "ws": torch.empty(grz.dp_embed_grad_workspace(n, v, d), device=DEV, dtype=torch.uint8)}
    return b


OUTPUTS = ("out", "lp", "h", "top", "tl", "dx", "dx2", "loss", "dtable")


def test_captured_calls_replay_as_the_eager_ones():
    b = _buffers(50)
    _run_all(b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _run_all(b)
    for seed in (51, 52, 53):
        new = _buffers(seed)
        for k in ("table", "ids", "x", "t", "g"):
            b[k].copy_(new[k])
        for k in OUTPUTS:
            b[k].fill_(3)
        b["ws"].fill_(0xFF)
        graph.replay()
        _run_all(new)  # the program's own eager work between the replays
        torch.cuda.synchronize()
        for k in OUTPUTS:
            assert torch.equal(b[k], new[k]), k


def test_two_streams_at_once():
    one, two = _buffers(60), _buffers(61)
    want = []
    for b in (one, two):
        _run_all(b)
        want.append({k: b[k].clone() for k in OUTPUTS})
        for k in OUTPUTS:
            b[k].fill_(3)
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        for b, s in zip((one, two), streams):
            with torch.cuda.stream(s):
                _run_all(b)
    torch.cuda.synchronize()
    for b, w in zip((one, two), want):
        for k in OUTPUTS:
            assert torch.equal(b[k], w[k]), k
    one["out"].fill_(3)
    grz.dp_embed_lookup(one["table"], one["ids"], one["out"], scale=2.0, stream=streams[0])
    torch.cuda.synchronize()
    assert torch.equal(one["out"], want[0]["out"])


# -- large sizes ---------------------------------------------------------------------------

def test_rows_beyond_one_launch():
    # The row kernels take 2^21 rows a launch, the lookup 2^23.
    n, v = 2 ** 21 + 5, 8
    x = logits_of(n, v, BF16)
    t = token_ids(n, v, 70)
    lp, h, ids, _ = logprob_call(x, t, 2)
    tail = slice(n - 8, n)
    sm = ref.Softmax(x[tail])
    tc = t[tail].cpu()
    ok = (tc >= 0) & (tc < v)
    zero = torch.zeros(8, dtype=torch.float64)
    at = tc.clamp(0, v - 1)[:, None]
    ref.assert_close(lp[tail], torch.where(ok, sm.lq.gather(1, at)[:, 0], zero),
                     torch.where(ok, sm.tol.gather(1, at)[:, 0], zero), "logprob")
    assert torch.equal(ids[tail].cpu().long(), order_of(x[tail], 2))
    w = torch.zeros(n, device=DEV)
    w[0] = w[-1] = 2.0
    dx, loss = torch.full_like(x, 5.0), torch.empty(n, device=DEV)
    grz.dp_distill_grad(x, ids, torch.zeros(n, 2, device=DEV), dx, weights=w, loss=loss)
    ends = torch.tensor([0, n - 1], device=DEV)
    d = ref.Distill(x[ends], ids[ends], torch.zeros(2, 2), 1.0, w[ends])
    ref.assert_close(dx[ends], d.dx, d.dx_tol, "dlogits")
    ref.assert_close(loss[ends], d.loss, d.loss_tol, "loss")
    assert (dx[1:-1] == 0).all() and (loss[1:-1] == 0).all()
    n = 2 ** 23 + 3
    table, _ = matrix(5, 4, BF16, seed=71)
    ids = torch.arange(n, device=DEV, dtype=torch.int32) % 5
    out = torch.zeros(n, 4, device=DEV, dtype=BF16)
    grz.dp_embed_lookup(table, ids, out)
    assert torch.equal(out, table[ids.long()])


def test_logits_beyond_32_bit_offsets():
    # 86000 rows of 50304: the last ones begin past 2^32 elements.
    n, v, stride = 86000, 50257, 50304
    x = torch.empty(n * stride, device=DEV, dtype=BF16).view(n, stride)[:, :v]
    last = logits_of(3, v, BF16, seed=72)
    x[-3:] = last
    w = torch.zeros(n, device=DEV)
    w[-3:] = 1.5
    ids, z = teacher_of(3, v, 9, 73, 64, F32)
    all_ids, all_z = torch.zeros(n, 9, device=DEV, dtype=torch.long), torch.zeros(n, 9, device=DEV)
    all_ids[-3:], all_z[-3:] = ids, z
    loss = torch.empty(n, device=DEV)
    grz.dp_distill_grad(x, all_ids, all_z, x, temperature=2.0, weights=w, loss=loss)
    d = ref.Distill(last, ids, z, 2.0, w[-3:])
    ref.assert_close(x[-3:], d.dx, d.dx_tol, "dlogits")
    ref.assert_close(loss[-3:], d.loss, d.loss_tol, "loss")
    assert (x[:-3] == 0).all() and (loss[:-3] == 0).all()
    x[-3:] = last
    lp, h, top, tl = (torch.empty(n, device=DEV), torch.empty(n, device=DEV),
                      torch.empty(n, 4, device=DEV, dtype=torch.int32),
                      torch.empty(n, 4, device=DEV))
    grz.dp_token_logprobs(x, None, None, h, top, tl)
    sm = ref.Softmax(last)
    want, tol = sm.entropy()
    ref.assert_close(h[-3:], want, tol, "entropy")
    order = order_of(last, 4)
    assert torch.equal(top[-3:].cpu().long(), order)
    assert (top[:-3] == torch.arange(4, device=DEV, dtype=torch.int32)).all()


# -- refusals that need device tensors ---------------------------------------------------------

def test_binding_refuses_layouts_types_and_shapes():
    f = torch.zeros(6, 8, device=DEV)
    i = torch.zeros(6, device=DEV, dtype=torch.long)
    col = torch.zeros(6, device=DEV)
    ws = torch.zeros(1 << 16, device=DEV, dtype=torch.uint8)
    bad = [
        (ValueError, lambda: grz.dp_embed_lookup(f.t(), i, f)),              # columns not adjacent
        (ValueError, lambda: grz.dp_embed_lookup(f, i, f[:1].expand(6, 8))),  # rows overlap
        (ValueError, lambda: grz.dp_embed_lookup(f, i[:5], f.clone())),
        (ValueError, lambda: grz.dp_embed_lookup(f, i, torch.zeros(6, 7, device=DEV))),
        (TypeError, lambda: grz.dp_embed_lookup(f, i.float(), f.clone())),
        (TypeError, lambda: grz.dp_embed_lookup(f.half(), i, f)),
        (ValueError, lambda: grz.dp_embed_lookup(f.view(-1), i, f)),
        (ValueError, lambda: grz.dp_embed_lookup(f, torch.zeros(12, device=DEV,
                                                                dtype=torch.long)[::2],
                                                 f.clone())),
        (grz.GrzError, lambda: grz.dp_embed_lookup(f, i, f)),                 # over its table
        (ValueError, lambda: grz.dp_embed_grad(f, i, f.clone(), None)),
        (ValueError, lambda: grz.dp_embed_grad(f, i, f.clone(), ws[:8])),
        (grz.GrzError, lambda: grz.dp_embed_grad(f, i, f.clone(), ws[4:])),
        (grz.GrzError, lambda: grz.dp_embed_grad(f, i, f, ws)),
        (TypeError, lambda: grz.dp_token_logprobs(f, i, logprob=col.double())),
        (ValueError, lambda: grz.dp_token_logprobs(f, i, logprob=col[:5])),
        (ValueError, lambda: grz.dp_token_logprobs(f, i, top_ids=i.int())),
        (ValueError, lambda: grz.dp_token_logprobs(
            f, i, top_ids=torch.zeros(6, 2, device=DEV, dtype=torch.int32))),
        (grz.GrzError, lambda: grz.dp_token_logprobs(
            f, top_ids=torch.zeros(6, 9, device=DEV, dtype=torch.int32),
            top_logprobs=torch.zeros(6, 9, device=DEV))),
        (grz.GrzError, lambda: grz.dp_token_logprobs(f, i)),
        (grz.GrzError, lambda: grz.dp_token_logprobs(f, logprob=col)),
        (TypeError, lambda: grz.dp_token_logprobs_grad(f, i, col, None, f.bfloat16())),
        (ValueError, lambda: grz.dp_token_logprobs_grad(f, i, col, None, f[:5])),
        (grz.GrzError, lambda: grz.dp_token_logprobs_grad(f, i, None, None, f.clone())),
        (ValueError, lambda: grz.dp_distill_loss(f, i, f, col)),
        (ValueError, lambda: grz.dp_distill_loss(f, i[:, None], f, col)),
        (grz.GrzError, lambda: grz.dp_distill_loss(f, i[:, None], f[:, :1].contiguous(), col,
                                                   temperature=0.0)),
        (grz.GrzError, lambda: grz.dp_distill_grad(f[:, :4], i[:, None],
                                                   f[:, :1].contiguous(), f[:, 2:6])),
        (ValueError, lambda: grz.dp_distill_grad(f, i[:, None], f[:, :1].contiguous(),
                                                 torch.zeros(6, 8))),
    ]
    for k, (error, call) in enumerate(bad):
        with pytest.raises(error):
            call()
            raise AssertionError(f"call {k} was not refused")
    torch.cuda.synchronize()
    assert (f == 0).all()
