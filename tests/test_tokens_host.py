"""Token operators: arguments that are refused before anything is launched, and
workspace sizes.  No GPU work."""

import pytest
import torch

import gradient_reduce_zero_amd as grz
from gradient_reduce_zero_amd import _native as N

A, B, C, D, W = 0x100000, 0x900000, 0x1100000, 0x1900000, 0x2100000  # never dereferenced
F, H = N.GRZ_F32, N.GRZ_BF16


def lookup(table=A, tt=H, vocab=10, dim=8, ts=8, ids=B, bits=64, n=4, out=C, ot=H, os_=8):
    return grz.lib().dp_embed_lookup(table, tt, vocab, dim, ts, ids, bits, n, 1.0, out, ot, os_,
                                     None)


def grad(dout=A, dt=H, ds=8, ids=B, bits=64, n=4, vocab=10, dim=8, flags=0, ws=W, table=C, tt=H,
         ts=8):
    return grz.lib().dp_embed_grad(dout, dt, ds, ids, bits, n, vocab, dim, 1.0, flags, ws, table,
                                   tt, ts, None)


def logprobs(x=A, dt=H, n=4, v=10, s=10, t=B, bits=64, top=0, lp=C, h=None, ti=None, tl=None):
    return grz.lib().dp_token_logprobs(x, dt, n, v, s, t, bits, top, lp, h, ti, tl, None)


def logprobs_grad(x=A, dt=H, n=4, v=10, s=10, t=B, bits=64, gl=C, ge=None, lp=None, h=None,
                  dx=D, ds=10):
    return grz.lib().dp_token_logprobs_grad(x, dt, n, v, s, t, bits, gl, ge, lp, h, dx, ds, None)


def distill(x=A, dt=H, n=4, v=10, s=10, ids=B, bits=64, z=C, zt=F, k=3, tau=1.0, w=None, loss=W,
            dx=D, ds=10, which="both"):
    lib = grz.lib()
    a = lib.dp_distill_loss(x, dt, n, v, s, ids, bits, z, zt, k, tau, w, loss, None) \
        if which != "grad" else None
    b = lib.dp_distill_grad(x, dt, n, v, s, ids, bits, z, zt, k, tau, w, 1.0, loss, dx, ds, None) \
        if which != "loss" else None
    assert which != "both" or a == b
    return b if a is None else a


def test_matrices_and_ids_are_checked():
    for call, ptr, ld, size in ((lookup, "table", "ts", "vocab"), (lookup, "out", "os_", "n"),
                                (grad, "dout", "ds", "n"), (grad, "table", "ts", "vocab"),
                                (logprobs, "x", "s", "n"), (logprobs_grad, "x", "s", "n"),
                                (logprobs_grad, "dx", "ds", "n"), (distill, "x", "s", "n")):
        name = (call.__name__, ptr)
        assert call(**{ptr: None}) == N.GRZ_EINVAL, name
        assert call(**{ptr: A + 1}) == N.GRZ_EALIGN, name
        assert call(**{ld: 7}) == N.GRZ_EINVAL, name
        assert call(**{size: -1}) == N.GRZ_EINVAL, name
        assert call(**{size: 2 ** 31}) == N.GRZ_ERANGE, name
        assert call(**{ld: 2 ** 60}) == N.GRZ_ERANGE, name
    for call in (lookup, grad):
        assert call(dim=-1) == N.GRZ_EINVAL
        assert call(ids=None) == N.GRZ_EINVAL
        assert call(ids=B + 4) == N.GRZ_EALIGN
        assert call(ids=B + 2, bits=32) == N.GRZ_EALIGN
        assert call(bits=16) == N.GRZ_EINVAL
        assert call(tt=N.GRZ_F64) == N.GRZ_EINVAL and call(tt=7) == N.GRZ_EINVAL
    assert lookup(ot=N.GRZ_F64) == N.GRZ_EINVAL and grad(dt=N.GRZ_F64) == N.GRZ_EINVAL
    for call in (logprobs, logprobs_grad):
        assert call(t=B + 4) == N.GRZ_EALIGN and call(bits=0) == N.GRZ_EINVAL
    for call in (logprobs, logprobs_grad, distill):
        assert call(dt=N.GRZ_F64) == N.GRZ_EINVAL
        assert call(v=-1) == N.GRZ_EINVAL and call(v=0) == N.GRZ_EINVAL


def test_outputs_that_overlap_an_input_are_refused():
    assert lookup(out=A + 16) == N.GRZ_EINVAL
    assert grad(table=A + 16) == N.GRZ_EINVAL
    assert grad(ws=C + 16) == N.GRZ_EINVAL
    assert grad(ws=A + 16) == N.GRZ_EINVAL
    assert grad(ids=C + 16) == N.GRZ_EINVAL
    assert grad(ids=W + 16) == N.GRZ_EINVAL
    assert lookup(ids=C + 16) == N.GRZ_EINVAL
    assert logprobs_grad(dx=A + 2) == N.GRZ_EINVAL
    assert logprobs_grad(dx=A, ds=12) == N.GRZ_EINVAL
    assert distill(dx=A + 2, which="grad") == N.GRZ_EINVAL
    assert distill(dx=A, ds=12, which="grad") == N.GRZ_EINVAL


def test_embed_grad_flags_workspace_and_limits():
    assert grad(flags=N.GRZ_SUM) == N.GRZ_EINVAL
    assert grad(flags=N.GRZ_ACCUMULATE | 1) == N.GRZ_EINVAL
    assert grad(ws=None) == N.GRZ_EINVAL
    assert grad(ws=W + 8) == N.GRZ_EALIGN
    assert grad(n=2 ** 28 + 1) == N.GRZ_ERANGE
    assert grad(vocab=2 ** 26 + 1) == N.GRZ_ERANGE
    assert grad(dim=65535 * 64 + 1, ds=2 ** 23, ts=2 ** 23) == N.GRZ_ERANGE
    assert grz.dp_embed_grad_workspace(0, 5, 8) == 0
    assert grz.dp_embed_grad_workspace(2 ** 28 + 1, 5, 8) == 0
    sizes = [grz.dp_embed_grad_workspace(n, 50257, 768) for n in (1, 100, 4096, 4097, 10 ** 6)]
    assert sizes[0] > 0 and sizes == sorted(sizes)
    assert grz.dp_embed_grad_workspace(2 ** 28, 2 ** 26, 65535 * 64) > 2 ** 32


def test_logprobs_arguments():
    assert logprobs(lp=None) == N.GRZ_EINVAL                      # nothing asked for
    assert logprobs(t=None) == N.GRZ_EINVAL                       # logprob without targets
    assert logprobs(top=-1) == N.GRZ_EINVAL
    assert logprobs(top=11, ti=C, tl=D) == N.GRZ_EINVAL           # longer than the vocabulary
    assert logprobs(v=1000, s=1000, top=N.GRZ_MAX_TOP + 1, ti=C, tl=D) == N.GRZ_EINVAL
    assert logprobs(top=2, ti=C) == N.GRZ_EINVAL
    assert logprobs(top=2, tl=C) == N.GRZ_EINVAL
    assert logprobs(lp=C + 2) == N.GRZ_EALIGN
    assert logprobs(h=C + 2) == N.GRZ_EALIGN
    assert logprobs(top=2, ti=C + 2, tl=D) == N.GRZ_EALIGN
    assert logprobs_grad(gl=None) == N.GRZ_EINVAL                 # no incoming gradient
    assert logprobs_grad(t=None) == N.GRZ_EINVAL
    assert logprobs_grad(t=None, gl=None, ge=C, lp=W) == N.GRZ_EINVAL
    assert logprobs_grad(gl=C + 1) == N.GRZ_EALIGN and logprobs_grad(ge=C + 1) == N.GRZ_EALIGN


def test_distill_arguments():
    for tau in (0.0, -1.0, float("inf"), float("nan"), 1e-45, 0.9e-18, 1.1e18):
        assert distill(tau=tau) == N.GRZ_EINVAL
    assert distill(k=0) == N.GRZ_EINVAL and distill(k=N.GRZ_MAX_TOP + 1) == N.GRZ_EINVAL
    assert distill(ids=None) == N.GRZ_EINVAL and distill(z=None) == N.GRZ_EINVAL
    assert distill(ids=B + 4) == N.GRZ_EALIGN and distill(z=C + 2) == N.GRZ_EALIGN
    assert distill(z=C + 1, zt=H) == N.GRZ_EALIGN
    assert distill(zt=N.GRZ_F64) == N.GRZ_EINVAL
    assert distill(w=C + 1) == N.GRZ_EALIGN and distill(loss=C + 1) == N.GRZ_EALIGN
    assert distill(loss=None, which="loss") == N.GRZ_EINVAL
    assert distill(n=2 ** 31 - 1, k=2) == N.GRZ_ERANGE
    assert distill(dx=None, which="grad") == N.GRZ_EINVAL
    assert distill(dx=D + 1, which="grad") == N.GRZ_EALIGN


def test_empty_calls_do_nothing():
    assert lookup(n=0, ids=None, out=None) == N.GRZ_OK
    assert grad(n=0, vocab=0, ids=None, dout=None, table=None, ws=None) == N.GRZ_OK
    assert logprobs(n=0) == N.GRZ_OK and logprobs_grad(n=0) == N.GRZ_OK
    assert distill(n=0) == N.GRZ_OK


def test_binding_refuses_what_the_library_cannot_see():
    f = torch.zeros(4, 8)
    i = torch.zeros(4, dtype=torch.long)
    for call in (lambda: grz.dp_embed_lookup(f, i, f),
                 lambda: grz.dp_embed_grad(f, i, f, None),
                 lambda: grz.dp_token_logprobs(f, i, logprob=f[:, 0]),
                 lambda: grz.dp_token_logprobs_grad(f, i, f[:, 0], None, f),
                 lambda: grz.dp_distill_loss(f, i[:, None], f[:, :1], f[:, 0]),
                 lambda: grz.dp_distill_grad(f, i[:, None], f[:, :1], f)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(TypeError):
        grz.dp_embed_lookup(None, i, f)
