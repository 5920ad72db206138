"""The kernels that dp_expert_combine and its gradient choose for many tokens: two or
four vectors a lane, two to eight rows at a time, rows read past the caches, sums added
to what is there, against 64-bit forms.  Widths leave a row's last run partly filled
and columns behind its last whole vector; some slots have no place."""

import math

import pytest
import torch

import gradient_reduce_zero_amd as grz
from test_gpu_experts import slots_of
from test_gpu_tokens import BF16, DEV, F32, matrix, outside_untouched
from token_ref import U, half_step

pytestmark = pytest.mark.gpu
MIB = 2 ** 20
PAIRS = [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)]


def columns(a, b):
    """Columns of a lane's vector."""
    return 8 if a == b == BF16 else 4


def tokens(k, dim, vec, size, streamed):
    """Tokens enough for more than 8192 waves of one vector a lane (2048 up to four
    slots), and with ``streamed`` for 64 MiB of rows."""
    runs = -(-dim // (64 * vec))
    n = (2048 if k <= 4 else 8192) // runs + 3
    return max(n, 64 * MIB // (k * dim * size) + 2) if streamed else n


def live(places, rows):
    return (places >= 0) & (places < rows), places.clamp(0, rows - 1).long()


def assert_near(got, want, tol, what):
    """|got - want| <= tol and the rounding to got's type of a value up to tol off."""
    lim = tol + half_step(got.dtype) * (want.abs() + tol) * (1 + U) + 2.0 ** -126
    off = (got.double() - want).abs()
    assert (off <= lim).all(), f"{what}: {(off - lim).max().item():.3g} over the bound"


def combine_exact(y, places, w, old):
    """(sum, sum of magnitudes) in 64 bits, slot by slot."""
    ok, at = live(places, y.shape[0])
    out = torch.zeros(places.shape[0], y.shape[1], device=DEV, dtype=torch.float64)
    if old is not None:
        out += old
    mag = out.abs()
    for j in range(places.shape[1]):
        rows = ok[:, j].nonzero()[:, 0]
        term = y[at[rows, j]].double()
        if w is not None:
            term *= w[rows, j, None]
        out[rows] += term
        mag[rows] += term.abs()
    return out, mag


# Narrow rows take two vectors a lane, those of eight vectors and more four.
@pytest.mark.parametrize("dim", [1603, 4101])
@pytest.mark.parametrize("k", [2, 3, 7, 11])
@pytest.mark.parametrize("ti,to", PAIRS)
@pytest.mark.parametrize("streamed", [False, True])
def test_combine_of_many_tokens(dim, k, ti, to, streamed):
    n = tokens(k, dim, columns(ti, to), ti.itemsize, streamed)
    rows = n * k - n // 3
    places, w = slots_of(n, k, rows, 100 + k)
    y, _ = matrix(rows, dim, ti, seed=101, pad=3, shift=1)
    for accumulate, weights in ((False, w), (True, w), (True, None)):
        out, buf = matrix(n, dim, to, seed=102, pad=5, shift=3)
        before, old = buf.clone(), out.double() if accumulate else None
        want, mag = combine_exact(y, places, weights, old)
        grz.dp_expert_combine(y, places, out, weights=weights, accumulate=accumulate)
        assert_near(out, want, (k + 1) * U * mag, f"accumulate {accumulate}")
        assert outside_untouched(out, buf, before)


@pytest.mark.parametrize("dim", [700, 1603, 2500, 4101])
@pytest.mark.parametrize("td,ty", PAIRS)
@pytest.mark.parametrize("streamed", [False, True])
def test_combine_gradient_of_many_tokens(dim, td, ty, streamed):
    k = 3
    n = tokens(k, dim, columns(td, ty), ty.itemsize, streamed)
    rows = n * k - n // 3
    places, w = slots_of(n, k, rows, 110)
    ok, at = live(places, rows)
    dout, _ = matrix(n, dim, td, seed=111, pad=3, shift=1)
    y, ybuf = matrix(rows, dim, ty, seed=112, pad=5, shift=3)
    dw = torch.zeros(n, k, device=DEV, dtype=torch.float64)
    mag = torch.zeros_like(dw)
    reached = []
    for j in range(k):
        some = ok[:, j].nonzero()[:, 0]
        term = dout[some].double() * y[at[some, j]].double()
        dw[some, j], mag[some, j] = term.sum(1), term.abs().sum(1)
        reached.append((at[some, j], (dout[some].float() * w[some, j, None]).to(ty)))
    # A lane's terms (the columns' 64th part, a run more of 16 at most), six steps in
    # its wave, the product.
    bound = (dim / 64 + 16 + 6 + 1) * U * mag
    dy, buf = matrix(rows, dim, ty, seed=113, pad=5, shift=3)
    want, before = dy.clone(), buf.clone()
    for r, v in reached:
        want[r] = v
    got = torch.full((n, k), math.nan, device=DEV)
    grz.dp_expert_combine_grad(dout, y, places, w, dy=dy, dweights=got)
    assert torch.equal(dy, want) and outside_untouched(dy, buf, before)
    assert_near(got, dw, bound, "dweights")
    # Over y, where rows without a place keep y's values.
    over, before = y.clone(), ybuf.clone()
    for r, v in reached:
        over[r] = v
    again = torch.full((n, k), math.nan, device=DEV)
    grz.dp_expert_combine_grad(dout, y, places, w, dy=y, dweights=again)
    assert torch.equal(y, over) and torch.equal(again, got)
    assert outside_untouched(y, ybuf, before)
