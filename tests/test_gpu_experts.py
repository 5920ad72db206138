"""Mixture-of-experts operators on the GPU against their 64-bit forms
(tests/expert_ref.py)."""

import math

import pytest
import torch

import expert_ref as ref
import gradient_reduce_zero_amd as grz
from test_gpu_tokens import BF16, DEV, F32, LOWEST, gen, matrix, outside_untouched
from token_ref import assert_close

pytestmark = pytest.mark.gpu
I32 = torch.int32
U_ROW = 2.0 ** -24  # half a step of fp32
LAYOUTS = [(0, 0), (8, 8), (3, 1)]  # elements between rows, and before the first


def logits_of(n, e, dtype, seed=0, pad=0, shift=0, std=2.0):
    return matrix(n, e, dtype, seed=seed, pad=pad, shift=shift, std=std)


def route_call(x, k, normalize):
    ids = torch.full((x.shape[0], k), -7, device=DEV, dtype=I32)
    w = torch.full((x.shape[0], k), math.nan, device=DEV)
    grz.dp_expert_route(x, ids, w, normalize=normalize)
    return ids, w


def check_route(x, k, what=""):
    want = ref.top_ids(x, k)
    for normalize in (False, True):
        ids, w = route_call(x, k, normalize)
        assert torch.equal(ids.cpu().long(), want), what
        r = ref.Route(x, ids, normalize)
        assert_close(w, r.w, r.tol, f"{what} weights, normalize {normalize}")


def check_route_grad(x, ids, dw, what="", out=None):
    for normalize in (False, True):
        want, tol = ref.Route(x, ids, normalize).grad(dw)
        dx, buf = out or matrix(*x.shape, x.dtype, pad=5, shift=3, std=None)
        before = buf.clone()
        grz.dp_expert_route_grad(x, ids, dw, dx, normalize=normalize)
        assert_close(dx, want, tol, f"{what} dlogits, normalize {normalize}")
        assert outside_untouched(dx, buf, before)


# -- router ------------------------------------------------------------------------

@pytest.mark.parametrize("n,e,k", [(0, 4, 2), (1, 1, 1), (1, 64, 8), (3, 2, 2), (17, 5, 3),
                                   (33, 16, 16), (100, 17, 4), (5, 60, 6), (64, 64, 1),
                                   (31, 65, 8), (200, 128, 8), (9, 130, 16), (40, 256, 8),
                                   (7, 256, 32), (11, 40, 17), (6, 257, 8), (13, 1000, 12),
                                   (4, 1024, 32), (2, 1021, 1)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pad,shift", LAYOUTS)
def test_route_and_its_gradient(n, e, k, dtype, pad, shift):
    x, _ = logits_of(n, e, dtype, seed=1, pad=pad, shift=shift)
    check_route(x, k, f"{n} x {e}")
    ids = torch.tensor(ref.top_ids(x, k).tolist(), device=DEV, dtype=I32).view(n, k)
    check_route_grad(x, ids, torch.randn(n, k, device=DEV, generator=gen(2)), f"{n} x {e}")


@pytest.mark.parametrize("e,k", [(6, 3), (64, 8), (128, 8), (256, 20), (700, 9)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_route_ties_masks_and_values_without_a_softmax(e, k, dtype):
    x, _ = logits_of(14, e, dtype, seed=3)
    x[0] = 1.5                                   # all equal
    x[1, 1::2] = x[1, 0]                         # half equal
    x[2] = -math.inf                             # nothing open
    x[3] = -math.inf
    x[3, e // 2] = 0.25                          # one open
    x[4] = LOWEST[dtype]                         # the type's lowest value everywhere
    x[5, : e // 2] = LOWEST[dtype]
    x[6, 0] = math.nan
    x[7, e - 1] = -math.nan
    x[8] = math.nan
    x[9, e // 3] = math.inf
    x[10, :2] = math.inf
    x[10, e - 1] = math.nan
    x[11] = 0.0
    x[11, 0] = -0.0                              # equal to the others
    x[12] = x[12] * 1e4                          # far apart
    x[13] = -math.inf
    x[13, : min(k, e)] = -3.0                    # exactly k open
    check_route(x, k, f"{e}")
    dw = torch.randn(14, k, device=DEV, generator=gen(4))
    ids, _ = route_call(x, k, False)
    check_route_grad(x, ids, dw, f"{e}")
    # Slots of no expert: what their dweights hold does not matter.
    dw[ids < 0] = math.nan
    check_route_grad(x, ids, dw, f"{e} NaN in unused dweights")
    # A row without an incoming gradient, or listed nowhere, gets zeros whatever it holds.
    for i, d in ((ids, torch.zeros_like(dw)), (torch.full_like(ids, -1), dw),
                 (torch.full_like(ids, e), dw)):
        dx = torch.full_like(x, 7.0)
        for normalize in (False, True):
            grz.dp_expert_route_grad(x, i, d, dx, normalize=normalize)
            assert (dx == 0).all()


@pytest.mark.parametrize("e,k", [(5, 4), (90, 8), (300, 32)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_route_grad_of_any_list(e, k, dtype):
    # Experts listed twice or often, closed ones, ids of none among them.
    n = 50
    x, _ = logits_of(n, e, dtype, seed=5)
    x[torch.rand(n, e, device=DEV, generator=gen(6)) < 0.3] = -math.inf
    x[:, 0] = 1.0
    ids = torch.randint(-1, min(e, 6) + 1, (n, k), device=DEV, generator=gen(7), dtype=I32)
    ids[0] = 0
    dw = torch.randn(n, k, device=DEV, generator=gen(8))
    check_route_grad(x, ids, dw)
    first = torch.empty_like(x)
    again = torch.empty_like(x)
    for normalize in (False, True):  # the same bits each time
        grz.dp_expert_route_grad(x, ids, dw, first, normalize=normalize)
        grz.dp_expert_route_grad(x, ids, dw, again, normalize=normalize)
        assert torch.equal(first, again)


@pytest.mark.parametrize("e,k", [(8, 2), (128, 8), (600, 20)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_route_grad_over_the_logits(e, k, dtype):
    x, buf = logits_of(333, e, dtype, seed=9, pad=3, shift=1)
    ids, _ = route_call(x, k, True)
    dw = torch.randn(333, k, device=DEV, generator=gen(10))
    for normalize in (False, True):
        want = torch.empty(333, e, device=DEV, dtype=dtype)
        grz.dp_expert_route_grad(x, ids, dw, want, normalize=normalize)
        before = buf.clone()
        keep = x.clone()
        grz.dp_expert_route_grad(x, ids, dw, x, normalize=normalize)
        assert torch.equal(x, want) and outside_untouched(x, buf, before)
        x.copy_(keep)


def test_route_gradient_against_differences():
    # d(sum of g w) along random directions, in 64 bits on the host, from the kernel's
    # gradient: central differences of step h are off by h^2 / 6 times a third
    # derivative that 6 |g| bounds, plus the gradient's own bound.
    n, e, k, h = 20, 12, 4, 1e-4
    x, _ = logits_of(n, e, F32, seed=11)
    ids, _ = route_call(x, k, False)
    dw = torch.randn(n, k, device=DEV, generator=gen(12))
    move = torch.randn(n, e, generator=torch.Generator().manual_seed(13), dtype=torch.float64)
    for normalize in (False, True):
        dx = torch.empty_like(x)
        grz.dp_expert_route_grad(x, ids, dw, dx, normalize=normalize)
        at = lambda t: (ref.Route(x.double().cpu() + t * move, ids, normalize).w
                        * dw.cpu().double()).sum(1)
        slope = (at(h) - at(-h)) / (2 * h)
        got = (dx.cpu().double() * move).sum(1)
        tol = ref.Route(x, ids, normalize).grad(dw)[1]
        lim = ((tol + 2 ** -24 * dx.cpu().double().abs()) * move.abs()).sum(1)
        # w's third derivative along v is at most 6 (2 max |v|)^3
        third = 6 * (2 * move.abs().max(1).values) ** 3 * dw.cpu().double().abs().sum(1)
        assert ((got - slope).abs() <= lim + h * h / 6 * third + 1e-10).all()


# -- sort ----------------------------------------------------------------------------

def sort_call(ids, experts):
    n, k = ids.shape
    ws = torch.full((max(4, grz.dp_expert_sort_workspace(n, k, experts)),), 0xA5, device=DEV,
                    dtype=torch.uint8)
    offsets = torch.full((experts + 1,), -9, device=DEV, dtype=I32)
    places = torch.full((n, k), -9, device=DEV, dtype=I32)
    grz.dp_expert_sort(ids, experts, offsets, places, ws)
    return offsets, places


@pytest.mark.parametrize("n,k", [(0, 3), (1, 1), (1, 32), (63, 1), (64, 2), (513, 2), (1024, 1),
                                 (1025, 1), (2048, 8), (2049, 8), (5461, 3), (30000, 1),
                                 (70001, 5)])
@pytest.mark.parametrize("experts", [1, 2, 8, 63, 64, 100, 128, 1000, 1024])
def test_sort(n, k, experts):
    ids = torch.randint(0, experts, (n, k), device=DEV, generator=gen(20))
    if n > 2:
        ids[n // 3] = -1
        ids[n // 2, 0] = experts
        ids[-1] = -5
        ids[: n // 4] = ids[0, 0]                 # a run of one expert
    if experts > 2:
        ids[ids == 1] = 2                         # an expert without tokens
    want = ref.sort(ids, experts)
    for one in (ids, ids.int()):
        got = sort_call(one, experts)
        assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[1].cpu(), want[1])


@pytest.mark.parametrize("n", [100, 20000])
def test_sort_of_extreme_ids(n):
    ids = torch.full((n, 2), 3, device=DEV)
    ids[5] = 2 ** 40 + 3                          # not 3 in 32 bits
    ids[6] = -2 ** 63
    ids[7] = 2 ** 63 - 1
    for one in (ids, torch.full_like(ids, -1)):
        got, want = sort_call(one, 4), ref.sort(one, 4)
        assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[1].cpu(), want[1])


# -- rows to their places and back -------------------------------------------------------

def slots_of(n, k, rows, seed):
    """Places in any order, some slots without one, some beyond the rows; weights."""
    total = n * k
    p = torch.randperm(max(total, rows), generator=torch.Generator().manual_seed(seed))[:total]
    p = torch.where(p < rows, p, torch.where(p % 2 == 0, -1, p + rows)).view(n, k)
    w = torch.randn(n, k, device=DEV, generator=gen(seed + 1))
    w[(p < 0).to(DEV)] = math.nan
    return p.int().to(DEV), w


SHAPES = [(0, 2, 8, 0), (1, 1, 1, 1), (1, 8, 384, 8), (3, 2, 7, 6), (5, 3, 129, 11),
          (17, 4, 260, 70), (9, 8, 513, 50), (6, 9, 1030, 54), (2, 32, 65, 40), (33, 6, 2056, 198),
          (4, 5, 4100, 0)]


@pytest.mark.parametrize("n,k,dim,rows", SHAPES)
@pytest.mark.parametrize("ti,to", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("pad,shift", LAYOUTS)
def test_dispatch_and_combine(n, k, dim, rows, ti, to, pad, shift):
    places, w = slots_of(n, k, rows, 30)
    x, _ = matrix(n, dim, ti, seed=31, pad=pad, shift=shift)
    y, _ = matrix(rows, dim, ti, seed=32, pad=pad, shift=shift)
    for weights in (None, w):
        out, buf = matrix(rows, dim, to, seed=33, pad=pad, shift=shift)
        before, want = buf.clone(), ref.dispatch(x, places, weights, out)
        grz.dp_expert_dispatch(x, places, out, weights=weights)
        assert torch.equal(out.cpu(), want)  # rows without a place among them
        assert outside_untouched(out, buf, before)
        for accumulate in (False, True):
            out, buf = matrix(n, dim, to, seed=34, pad=pad, shift=shift)
            before, old = buf.clone(), out.clone()
            want, tol = ref.combine(y, places, weights, old if accumulate else None)
            grz.dp_expert_combine(y, places, out, weights=weights, accumulate=accumulate)
            assert_close(out, want, tol, f"combine, accumulate {accumulate}")
            assert outside_untouched(out, buf, before)


@pytest.mark.parametrize("n,k,dim,rows", SHAPES)
@pytest.mark.parametrize("td,ty", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("pad,shift", LAYOUTS)
def test_combine_grad(n, k, dim, rows, td, ty, pad, shift):
    places, w = slots_of(n, k, rows, 40)
    dout, _ = matrix(n, dim, td, seed=41, pad=pad, shift=shift)
    y, ybuf = matrix(rows, dim, ty, seed=42, pad=pad, shift=shift)
    for weights in (None, w):
        dy, buf = matrix(rows, dim, ty, seed=43, pad=pad, shift=shift)
        before = buf.clone()
        want, dw, tol = ref.combine_grad(dout, y, places, weights, dy)
        got = torch.full((n, k), math.nan, device=DEV)
        grz.dp_expert_combine_grad(dout, y, places, weights, dy=dy, dweights=got)
        assert torch.equal(dy.cpu(), want) and outside_untouched(dy, buf, before)
        assert_close(got, dw, tol, "dweights")
        # One of the two; dy without y; dy over y.
        alone = torch.full((n, k), math.nan, device=DEV)
        grz.dp_expert_combine_grad(dout, y, places, weights, dweights=alone)
        assert torch.equal(alone, got)
        for given in (y, None):
            dy, buf = matrix(rows, dim, ty, seed=43, pad=pad, shift=shift)
            grz.dp_expert_combine_grad(dout, given, places, weights, dy=dy)
            assert torch.equal(dy.cpu(), want)
        keep, before = y.clone(), ybuf.clone()
        over = ref.combine_grad(dout, y, places, weights, y)[0]
        alone.fill_(math.nan)
        grz.dp_expert_combine_grad(dout, y, places, weights, dy=y, dweights=alone)
        assert torch.equal(y.cpu(), over) and torch.equal(alone, got)
        assert outside_untouched(y, ybuf, before)
        y.copy_(keep)


@pytest.mark.parametrize("n,k,dim", [(4099, 2, 130), (5000, 4, 70), (4500, 7, 68), (4100, 1, 1500),
                                     (17000, 2, 40)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_tokens(n, k, dim, dtype):
    # The shapes of launches that have enough tokens, back and forth: the weights'
    # sum times each row, and the gradients of that.
    rows = n * k
    places, w = slots_of(n, k, rows, 50)
    x, _ = matrix(n, dim, dtype, seed=51)
    out = torch.zeros(rows, dim, device=DEV, dtype=dtype)
    grz.dp_expert_dispatch(x, places, out)
    assert torch.equal(out[places.long()], x[:, None, :].expand(n, k, dim))
    back = torch.empty(n, dim, device=DEV)
    grz.dp_expert_combine(out, places, back, weights=w)
    want, tol = ref.combine(out, places, w)
    assert_close(back, want, tol, "combine")
    dw, dy = torch.empty(n, k, device=DEV), torch.zeros_like(out)
    grz.dp_expert_combine_grad(back, out, places, w, dy=dy, dweights=dw)
    d, o = back.double().cpu(), out.double().cpu()
    at = places.long().cpu()
    want = (d[:, None, :] * o[at]).sum(2)
    mag = (d[:, None, :] * o[at]).abs().sum(2)
    assert_close(dw, want, (dim / 64 + 25) * ref.U * mag, "dweights")
    assert torch.equal(dy[places.long()], (back[:, None, :] * w[:, :, None]).to(dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_named_twice_harm_no_others(dtype):
    n, k, d = 300, 3, 700
    places = torch.randperm(n * k, generator=torch.Generator().manual_seed(5)).int().view(n, k)
    twice = places[7, 1].item()
    places[200, 2] = twice
    places = places.to(DEV)
    x, _ = matrix(n, d, dtype, seed=55)
    out = torch.zeros(n * k, d, device=DEV, dtype=dtype)
    grz.dp_expert_dispatch(x, places, out)
    want = ref.dispatch(x, places, None, torch.zeros_like(out))
    others = torch.arange(n * k) != twice
    assert torch.equal(out.cpu()[others], want[others])
    both = torch.stack([x[7], x[200]]).cpu()
    assert ((out[twice].cpu() == both[0]) | (out[twice].cpu() == both[1])).all()
    dw = torch.empty(n, k, device=DEV)
    want, dwant, tol = ref.combine_grad(x, out, places, None, torch.zeros_like(out))
    dy = torch.zeros_like(out)
    grz.dp_expert_combine_grad(x, out, places, None, dy=dy, dweights=dw)
    assert torch.equal(dy.cpu()[others], want[others])
    assert_close(dw, dwant, tol, "dweights")


def test_weights_of_zero_infinity_and_nan():
    # A slot counts by its place: a weight of 0 times an infinity is a NaN, as written.
    places = torch.tensor([[0, 1], [2, -1]], device=DEV, dtype=I32)
    y = torch.ones(3, 40, device=DEV)
    y[0, 3], y[1, 5], y[2, 7] = math.inf, math.nan, -math.inf
    w = torch.tensor([[0.0, 2.0], [-1.0, math.nan]], device=DEV)
    out = torch.empty(2, 40, device=DEV)
    grz.dp_expert_combine(y, places, out, weights=w)
    want, tol = ref.combine(y, places, w)
    assert_close(out, want, tol, "combine")
    assert torch.isnan(out[0, 3]) and torch.isnan(out[0, 5]) and out[1, 7] == math.inf


@pytest.mark.parametrize("weighted", [False, True])
def test_gradients_against_differences(weighted):
    # The sum <g, combine(y, w)> is linear in y and in w, <G, dispatch(x)> in x: central
    # differences of the 64-bit forms along a direction are exact but for their own
    # roundings (1e-9 of the magnitudes here), so only the kernels' bounds remain.
    n, k, d, h = 30, 3, 45, 0.5
    places, w = slots_of(n, k, n * k - 7, 52)
    w = torch.nan_to_num(w) if weighted else None
    rows = n * k - 7
    y, _ = matrix(rows, d, F32, seed=53)
    g, _ = matrix(n, d, F32, seed=54)
    x, _ = matrix(n, d, F32, seed=55)
    dy, dw = torch.zeros_like(y), torch.empty(n, k, device=DEV)
    grz.dp_expert_combine_grad(g, y, places, w, dy=dy, dweights=dw)
    dx = torch.empty_like(x)
    grz.dp_expert_combine(y, places, dx, weights=w)       # y in the place of the rows' gradient
    gd, yd = g.double().cpu(), y.double().cpu()
    ones = torch.ones(n, k, dtype=torch.float64)
    wd = ones if w is None else w.double().cpu()
    rand = torch.Generator().manual_seed(56)
    ok, at = ref.live(places, rows)
    reached = torch.zeros(rows, dtype=torch.bool)
    reached[at[ok]] = True

    def slope(loss, point, move):
        return (loss(point + h * move) - loss(point - h * move)) / (2 * h)

    def loss_y(t):
        return (gd * ref.combine(t, places, wd)[0]).sum()

    def loss_w(t):
        return (gd * ref.combine(yd, places, t)[0]).sum()

    def loss_x(t):  # rows of a dispatch against y
        return sum(((wd[i, j] * t[i]) * yd[at[i, j]]).sum() for i, j in ok.nonzero().tolist())

    for loss, point, got, bound in (
            (loss_y, yd, dy, U_ROW * dy.abs()),
            (loss_w, wd, dw, ref.combine_grad(g, y, places, w, torch.zeros_like(y))[2]),
            (loss_x, x.double().cpu(), dx, ref.combine(y, places, w)[1])):
        move = torch.randn(point.shape, generator=rand, dtype=torch.float64)
        want = slope(loss, point, move)
        got = got.double().cpu()
        terms = (got * move).abs()
        lim = ((bound.double().cpu() + U_ROW * got.abs()) * move.abs()).sum() + 1e-9 * terms.sum()
        assert abs((got * move).sum() - want) <= lim
    assert (dy.cpu()[~reached] == 0).all()


# -- large offsets, batches of launches, streams, graphs ------------------------------------

def test_beyond_32_bit_offsets():
    # Rows 2^31 + 8 elements apart: the last starts past 2^32 elements.
    stride, d = 2 ** 31 + 8, 72
    buf = torch.zeros(2 * stride + 128, device=DEV, dtype=BF16)
    far = torch.as_strided(buf, (3, d), (stride, 1))
    x = torch.randn(2, d, device=DEV, generator=gen(60)).to(BF16)
    places = torch.tensor([[2, 0], [1, -1]], device=DEV, dtype=I32)
    w = torch.tensor([[0.5, 2.0], [3.0, 1.0]], device=DEV)
    grz.dp_expert_dispatch(x, places, far)
    assert torch.equal(far, x[[0, 1, 0]])
    out = torch.empty(2, d, device=DEV)
    grz.dp_expert_combine(far, places, out, weights=w)
    want, tol = ref.combine(far, places, w)
    assert_close(out, want, tol, "rows far apart")
    dw = torch.empty(2, 2, device=DEV)
    want, dwant, tol = ref.combine_grad(out, far, places, w, far)
    grz.dp_expert_combine_grad(out, far, places, w, dy=far, dweights=dw)
    assert torch.equal(far.cpu(), want)
    assert_close(dw, dwant, tol, "dweights")
    # tokens far apart
    grz.dp_expert_combine(x, torch.tensor([[1], [0], [1]], device=DEV, dtype=I32), far)
    assert torch.equal(far, x[[1, 0, 1]])
    ids = torch.empty(3, 4, device=DEV, dtype=I32)
    lw = torch.empty(3, 4, device=DEV)
    grz.dp_expert_route(far, ids, lw)
    assert torch.equal(ids.cpu().long(), ref.top_ids(far, 4))
    want, tol = ref.Route(far, ids, False).grad(lw)
    grz.dp_expert_route_grad(far, ids, lw, far)
    assert_close(far, want, tol, "logits far apart")


def test_more_tokens_than_one_launch_takes():
    n = 2 ** 21 + 5
    x = torch.arange(n, device=DEV, dtype=F32)[:, None].contiguous()
    places = torch.flip(torch.arange(n, device=DEV, dtype=I32), [0])[:, None].contiguous()
    out, back = torch.empty_like(x), torch.empty_like(x)
    grz.dp_expert_dispatch(x, places, out)
    assert torch.equal(out, torch.flip(x, [0]))
    grz.dp_expert_combine(out, places, back)
    assert torch.equal(back, x)
    dw, dy = torch.empty(n, 1, device=DEV), torch.empty_like(x)
    one = torch.ones_like(x)
    grz.dp_expert_combine_grad(one, out, places, None, dy=dy, dweights=dw)
    assert torch.equal(dw, x) and (dy == 1).all()
    logits = torch.stack([torch.zeros(n, device=DEV), x[:, 0] % 2 * 2 - 1], 1)
    ids, w = route_call(logits, 1, True)
    assert torch.equal(ids[:, 0], (torch.arange(n, device=DEV) % 2).int()) and (w == 1).all()
    dl = torch.empty_like(logits)
    grz.dp_expert_route_grad(logits, ids, w, dl, normalize=True)
    assert (dl == 0).all()
    offsets, sorted_places = sort_call(ids, 2)
    assert offsets.tolist() == [0, (n + 1) // 2, n]
    want = torch.where(ids[:, 0] == 0, torch.arange(n, device=DEV) // 2,
                       (n + 1) // 2 + torch.arange(n, device=DEV) // 2)
    assert torch.equal(sorted_places[:, 0].long(), want)


class Layer:
    """All operators in a row on buffers of their own; `run` is one pass."""

    def __init__(self, n, e, k, d, seed):
        g = gen(seed)
        self.e = e
        self.logits = torch.randn(n, e, device=DEV, generator=g)
        self.x = torch.randn(n, d, device=DEV, generator=g).to(BF16)
        self.dout = torch.randn(n, d, device=DEV, generator=g).to(BF16)
        i32 = lambda *s: torch.full(s, -3, device=DEV, dtype=I32)
        f32 = lambda *s: torch.full(s, math.nan, device=DEV)
        self.ids, self.places, self.offsets = i32(n, k), i32(n, k), i32(e + 1)
        self.w, self.dw, self.dlogits = f32(n, k), f32(n, k), f32(n, e)
        self.rows, self.dy = f32(n * k, d).to(BF16), f32(n * k, d).to(BF16)
        self.out, self.dx = f32(n, d), f32(n, d)
        self.ws = torch.empty(max(4, grz.dp_expert_sort_workspace(n, k, e)), device=DEV,
                              dtype=torch.uint8)

    def run(self, stream=None):
        s = dict(stream=stream)
        grz.dp_expert_route(self.logits, self.ids, self.w, normalize=True, **s)
        grz.dp_expert_sort(self.ids, self.e, self.offsets, self.places, self.ws, **s)
        grz.dp_expert_dispatch(self.x, self.places, self.rows, **s)
        grz.dp_expert_combine(self.rows, self.places, self.out, weights=self.w, **s)
        grz.dp_expert_combine_grad(self.dout, self.rows, self.places, self.w, dy=self.dy,
                                   dweights=self.dw, **s)
        grz.dp_expert_combine(self.dy, self.places, self.dx, **s)
        grz.dp_expert_route_grad(self.logits, self.ids, self.dw, self.dlogits, normalize=True,
                                 **s)

    def results(self):
        return [self.ids, self.w, self.offsets, self.places, self.rows, self.out, self.dy,
                self.dw, self.dx, self.dlogits]

    def change(self, seed):
        g = gen(seed)
        self.logits.copy_(torch.randn(self.logits.shape, device=DEV, generator=g))
        self.x.copy_(torch.randn(self.x.shape, device=DEV, generator=g))
        for t in self.results():
            t.fill_(-3)


@pytest.mark.parametrize("n", [40, 9000])
def test_captured_and_replayed(n):
    a, b = Layer(n, 24, 4, 200, 70), Layer(n, 24, 4, 200, 70)
    a.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run()
    for i in range(4):  # other inputs each time, eager work between the replays
        a.change(71 + i)
        b.change(71 + i)
        graph.replay()
        b.run()
        torch.cuda.synchronize()
        for got, want in zip(a.results(), b.results()):
            assert torch.equal(got, want), i


def test_two_streams_at_once():
    layers = [Layer(9000, 24, 4, 200, 80 + i) for i in range(2)]
    want = [Layer(9000, 24, 4, 200, 80 + i) for i in range(2)]
    for w in want:
        w.run()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        for layer, s in zip(layers, streams):
            layer.run(stream=s)
    torch.cuda.synchronize()
    for layer, w in zip(layers, want):
        for got, one in zip(layer.results(), w.results()):
            assert torch.equal(got, one)


def test_results_repeat_and_do_not_depend_on_the_layout():
    n, k, d = 700, 4, 333
    places, w = slots_of(n, k, n * k, 90)
    outs, dws = [], []
    for pad, shift in LAYOUTS + [(0, 0)]:
        y, _ = matrix(n * k, d, BF16, seed=91, pad=pad, shift=shift)
        out, _ = matrix(n, d, F32, pad=pad, shift=shift, std=None)
        grz.dp_expert_combine(y, places, out, weights=w)
        dw = torch.empty(n, k, device=DEV)
        grz.dp_expert_combine_grad(out, y, places, w, dweights=dw)
        outs.append(out.clone())
        dws.append(dw)
    assert all(torch.equal(o, outs[0]) for o in outs)
    assert all(torch.equal(o, dws[0]) for o in dws)


def test_refusals_with_device_tensors():
    f = torch.zeros(4, 8, device=DEV)
    ids = torch.zeros(4, 2, device=DEV, dtype=I32)
    w = torch.zeros(4, 2, device=DEV)
    rows = torch.zeros(8, 8, device=DEV)
    offsets = torch.zeros(9, device=DEV, dtype=I32)
    with pytest.raises(TypeError):
        grz.dp_expert_route(f, ids.long(), w)
    with pytest.raises(ValueError):
        grz.dp_expert_route(f, ids, w[:, :1])
    with pytest.raises(grz.GrzError):  # more slots than experts
        grz.dp_expert_route(f[:, :1], ids, w)
    with pytest.raises(ValueError):
        grz.dp_expert_route(f.t(), ids, w)
    with pytest.raises(ValueError):
        grz.dp_expert_sort(ids, 8, offsets[:3], ids.clone())
    with pytest.raises(TypeError):
        grz.dp_expert_sort(ids, 8, None, ids.clone())
    with pytest.raises(grz.GrzError):  # places over the ids
        grz.dp_expert_sort(ids, 8, offsets, ids)
    big = torch.zeros(20000, 2, device=DEV, dtype=I32)
    with pytest.raises(ValueError, match="workspace"):
        grz.dp_expert_sort(big, 8, offsets, big.clone())
    with pytest.raises(ValueError):
        grz.dp_expert_dispatch(f, ids[:3], rows)
    with pytest.raises(ValueError):
        grz.dp_expert_dispatch(f, ids, rows[:, :7])
    with pytest.raises(grz.GrzError):
        grz.dp_expert_dispatch(rows[:4], ids, rows)
    with pytest.raises(grz.GrzError):
        grz.dp_expert_combine(rows, ids, rows[:4])
    with pytest.raises(TypeError):
        grz.dp_expert_combine(rows, ids, f.half())
    with pytest.raises(ValueError):
        grz.dp_expert_combine_grad(f, None, ids, w, dweights=w.clone())
    with pytest.raises(ValueError):
        grz.dp_expert_combine_grad(f, None, ids, w)
    with pytest.raises(grz.GrzError):
        grz.dp_expert_combine_grad(f, rows, ids, w)
    with pytest.raises(grz.GrzError):  # dweights over the weights
        grz.dp_expert_combine_grad(f, rows, ids, w, dweights=w)
    with pytest.raises(TypeError):
        grz.dp_expert_combine_grad(f, rows, ids, w, dy=rows.to(BF16))
