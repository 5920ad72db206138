"""Token operators over the vocabulary: an output that lies over an input or over
another output is refused before anything is launched.  No GPU work."""

import pytest

from gradient_reduce_zero_amd import _native as N
from test_tokens_host import distill, logprobs, logprobs_grad

# Never dereferenced.  4 rows of 10 bf16 logits at X are 80 bytes; a list of 4 fp32 values 16.
X, T, G, E, L, H, TI, TL, DX = (0x100000 * (i + 1) for i in range(9))
REFUSED = N.GRZ_EINVAL


@pytest.mark.parametrize("out", ["lp", "h", "ti", "tl"])
def test_logprobs_outputs(out):
    place = dict(lp=L, h=H, ti=TI, tl=TL)
    size = dict(lp=16, h=16, ti=32, tl=32)[out]

    def call(at):
        return logprobs(x=X, t=T, top=2, **{**place, out: at})

    for base, held in ((X, 80), (T, 32), *((p, dict(lp=16, h=16, ti=32, tl=32)[k])
                                           for k, p in place.items() if k != out)):
        for at in (base, base + held - 4, base + 4 - size):
            assert call(at) == REFUSED, (out, hex(at))
    # rows apart in memory: over the second row, from the gap before it
    assert logprobs(x=X, s=40, t=T, top=2, **{**place, out: X + 96 - size}) == REFUSED


@pytest.mark.parametrize("out", ["lp", "h", "dx"])
def test_logprobs_grad_outputs(out):
    place = dict(lp=L, h=H, dx=DX)
    held = dict(lp=16, h=16, dx=80)

    def call(at):
        return logprobs_grad(x=X, t=T, gl=G, ge=E, **{**place, out: at})

    inputs = [(T, 32)] + ([(G, 16), (E, 16)] if out == "dx" else [(X, 80)])
    for base, size in (*inputs, *((p, held[k]) for k, p in place.items() if k != out)):
        for at in (base, base + size - 4, base + 4 - held[out]):
            assert call(at) == REFUSED, (out, hex(at))
    if out != "dx":  # a value a row may replace one that comes in, row by row only
        for base in (G, E):
            assert call(base + 4) == REFUSED and call(base - 12) == REFUSED
    assert logprobs_grad(x=X, t=T, gl=DX + 40 * 2 * 3, ge=E, dx=DX, ds=40) == REFUSED


@pytest.mark.parametrize("which", ["loss", "grad"])
def test_distill_outputs(which):
    ids, z, w, loss = T, G, E, L

    def call(**kw):
        return distill(**{**dict(x=X, ids=ids, z=z, w=w, loss=loss, dx=DX, which=which), **kw})

    for base, size in ((X, 80), (ids, 96), (z, 48)):
        for at in (base, base + size - 4, base - 12):
            assert call(loss=at) == REFUSED, hex(at)
    assert call(loss=w + 4) == REFUSED and call(loss=w - 12) == REFUSED
    if which == "grad":
        for base, size in ((ids, 96), (z, 48), (w, 16), (loss, 16)):
            for at in (base, base + size - 4, base - 76):
                assert call(dx=at) == REFUSED, hex(at)
        assert call(dx=X, loss=X + 4) == REFUSED
