"""Mixture-of-experts operators and lists of tensors: arguments that are refused
before anything is launched, overlaps, sizes of workspaces.  No GPU work."""

import ctypes

import pytest
import torch

import gradient_reduce_zero_amd as grz
from gradient_reduce_zero_amd import _native as N

A, B, C, D, E, W = (0x1000000 * (i + 1) for i in range(6))  # never dereferenced
F, H = N.GRZ_F32, N.GRZ_BF16
INVALID, ALIGN, RANGE, OK = N.GRZ_EINVAL, N.GRZ_EALIGN, N.GRZ_ERANGE, N.GRZ_OK


def route(x=A, dt=H, n=4, e=10, s=10, k=2, flags=0, ids=B, w=C):
    return grz.lib().dp_expert_route(x, dt, n, e, s, k, flags, ids, w, None)


def route_grad(x=A, dt=H, n=4, e=10, s=10, k=2, flags=0, ids=B, dw=C, dx=D, ds=10):
    return grz.lib().dp_expert_route_grad(x, dt, n, e, s, k, flags, ids, dw, dx, ds, None)


def sort(ids=A, bits=64, n=4, k=2, e=10, ws=W, off=B, pl=C):
    return grz.lib().dp_expert_sort(ids, bits, n, k, e, ws, off, pl, None)


def dispatch(x=A, xt=H, xs=8, pl=B, w=None, n=4, k=2, dim=8, rows=8, out=C, ot=H, os_=8):
    return grz.lib().dp_expert_dispatch(x, xt, xs, pl, w, n, k, dim, rows, out, ot, os_, None)


def combine(y=A, yt=H, ys=8, rows=8, pl=B, w=None, n=4, k=2, dim=8, flags=0, out=C, ot=H,
            os_=8):
    return grz.lib().dp_expert_combine(y, yt, ys, rows, pl, w, n, k, dim, flags, out, ot, os_,
                                       None)


def combine_grad(d=A, dt=H, ds=8, y=B, yt=H, ys=8, rows=8, pl=C, w=None, n=4, k=2, dim=8, dy=D,
                 dys=8, dw=E):
    return grz.lib().dp_expert_combine_grad(d, dt, ds, y, yt, ys, rows, pl, w, n, k, dim, dy, dys,
                                            dw, None)


MATRICES = [(route, "x", "s", "n", "dt"), (route_grad, "x", "s", "n", "dt"),
            (route_grad, "dx", "ds", "n", "dt"), (dispatch, "x", "xs", "n", "xt"),
            (dispatch, "out", "os_", "rows", "ot"), (combine, "y", "ys", "rows", "yt"),
            (combine, "out", "os_", "n", "ot"), (combine_grad, "d", "ds", "n", "dt"),
            (combine_grad, "y", "ys", "rows", "yt"), (combine_grad, "dy", "dys", "rows", "yt")]


@pytest.mark.parametrize("call,ptr,ld,size,kind", MATRICES)
def test_matrices(call, ptr, ld, size, kind):
    if ptr != "dy":  # may be absent
        assert call(**{ptr: None}) == INVALID
    assert call(**{ptr: A + 1}) == ALIGN
    assert call(**{ptr: A + 2, kind: F}) == ALIGN
    assert call(**{ld: 7}) == INVALID
    assert call(**{size: -1}) == INVALID
    assert call(**{size: 2 ** 31}) == RANGE
    assert call(**{ld: 2 ** 60}) == RANGE
    assert call(**{kind: N.GRZ_F64}) == INVALID and call(**{kind: 7}) == INVALID


@pytest.mark.parametrize("call", [route, route_grad, sort, dispatch, combine, combine_grad])
def test_slots(call):
    for k in (0, -1, N.GRZ_MAX_SLOTS + 1):
        assert call(k=k) == INVALID, k
    assert call(n=2 ** 27 + 1) == RANGE and call(n=-1) == INVALID
    arrays = {route: "ids w", route_grad: "ids dw", sort: "pl off", dispatch: "pl", combine: "pl",
              combine_grad: "pl"}[call].split()
    for name in arrays:
        assert call(**{name: None}) == INVALID, name
        assert call(**{name: E + 0x800002}) == ALIGN, name
    if call in (dispatch, combine, combine_grad):
        assert call(w=E + 0x800001) == ALIGN
        assert call(dim=-1) == INVALID
        assert call(dim=65535 * 64 + 1, **{p: 2 ** 23 for p in (
            ("xs", "os_") if call is dispatch else ("ys", "os_") if call is combine
            else ("ds", "ys", "dys"))}) == RANGE


def test_experts_and_flags():
    for call in (route, route_grad, sort):
        assert call(e=0) == INVALID and call(e=-3) == INVALID
        assert call(e=N.GRZ_MAX_EXPERTS + 1, **({} if call is sort else dict(s=2000))) == RANGE
    for call in (route, route_grad):
        assert call(e=10, k=11) == INVALID
        assert call(flags=N.GRZ_ACCUMULATE) == INVALID
        assert call(flags=N.GRZ_NORMALIZE | 1) == INVALID
    assert combine(flags=N.GRZ_NORMALIZE) == INVALID
    assert combine(flags=N.GRZ_ACCUMULATE | 2) == INVALID
    assert sort(bits=16) == INVALID and sort(ids=None) == INVALID and sort(ids=A + 4) == ALIGN
    assert sort(ids=A + 2, bits=32) == ALIGN
    many = dict(n=20000, k=2)
    assert sort(ws=None, **many) == INVALID and sort(ws=W + 2, **many) == ALIGN
    assert combine_grad(dy=None, dw=None) == INVALID
    assert combine_grad(dw=E + 2) == ALIGN


def test_sort_workspace():
    size = grz.dp_expert_sort_workspace
    assert size(0, 1, 8) == 0 and size(64, 8, 128) == 0
    assert size(-1, 2, 8) == size(5, 0, 8) == size(5, 33, 8) == 0
    assert size(20000, 8, 0) == size(20000, 8, 1025) == size(2 ** 28 + 1, 1, 8) == 0
    # Counts of every expert in tiles of a thousand slots or more, bounded whatever the
    # slots.
    for n, k in ((20000, 8), (2 ** 20, 8), (2 ** 23 + 1, 8), (2 ** 28, 1), (8193, 1)):
        for experts in (1, 100, 1024):
            tiles, rest = divmod(size(n, k, experts), 4 * experts)
            assert rest == 0 and 0 < tiles <= -(-n * k // 1024) and tiles * experts <= 2 ** 18


def test_overlaps():
    # 4 bf16 rows of 10 at A are 80 bytes, a list of 4 x 2 values 32.
    for at in (A, A + 76, A - 28):
        assert route(ids=at) == INVALID and route(w=at) == INVALID
    assert route(w=B + 28) == INVALID and route(w=B - 28) == INVALID
    for base, held in ((B, 32), (C, 32)):
        for at in (base, base + held - 4, base - 76):
            assert route_grad(dx=at) == INVALID
    assert route_grad(dx=A + 4) == INVALID and route_grad(dx=A, ds=12) == INVALID
    for at in (A, A + 60):  # 8 ids of 8 bytes
        assert sort(pl=at) == INVALID and sort(off=at) == INVALID
    assert sort(off=C + 28) == INVALID and sort(pl=B + 40) == INVALID
    big = dict(n=20000, k=1)
    need = grz.dp_expert_sort_workspace(20000, 1, 10)
    for other in ("ids", "off", "pl"):
        assert sort(**{other: W + need - 8}, **big) == INVALID, other
    for out, held in ((A, 64), (B, 32)):  # x, places
        for at in (out, out + held - 4, out - 124):
            assert dispatch(out=at) == INVALID
    assert dispatch(out=D, w=D + 124) == INVALID
    for out, held in ((A, 128), (B, 32)):  # y, places
        for at in (out, out + held - 4, out - 60):
            assert combine(out=at) == INVALID
    assert combine(out=D, w=D + 60) == INVALID
    for base, held in ((A, 64), (C, 32), (E, 32)):  # dout, places, dweights
        for at in (base, base + held - 4, base - 124):
            assert combine_grad(dy=at) == INVALID, hex(at)
    assert combine_grad(dy=B + 4) == INVALID and combine_grad(dy=B, dys=16) == INVALID
    assert combine_grad(w=W, dy=W + 28) == INVALID
    for base, held in ((A, 64), (B, 128), (C, 32), (W, 32)):
        for at in (base, base + held - 4, base - 28):
            assert combine_grad(w=W, dw=at) == INVALID, hex(at)


def test_empty_calls_do_nothing():
    assert route(n=0, ids=None, w=None, x=None) == OK
    assert route_grad(n=0, ids=None, dw=None, x=None, dx=None) == OK
    assert dispatch(n=0, x=None, pl=None) == OK
    assert dispatch(dim=0, x=None, out=None, xs=0, os_=0) == OK
    assert dispatch(rows=0, out=None) == OK
    assert combine(n=0, pl=None, out=None) == OK and combine(dim=0, ys=0, os_=0) == OK
    assert combine_grad(n=0, d=None, pl=None) == OK
    assert combine_grad(rows=0, y=None, dy=None, dw=None) == OK


# -- lists of tensors -----------------------------------------------------------------

def table(*entries):
    """(address, numel[, type]) as the library takes them."""
    t = (N.Tensor * max(len(entries), 1))()
    for e, (at, numel, *kind) in zip(t, entries):
        e.data, e.numel, e.dtype = at, numel, kind[0] if kind else F
    return t, len(entries)


def norm(entries, max_norm=1.0, lead=0, ws=W, sq=D, sc=E):
    return grz.lib().dp_grad_sqnorm_tensors(*table(*entries), max_norm, lead, ws, sq, sc, None)


def clip(entries, out=None, scale=E):
    t, n = table(*entries)
    return grz.lib().dp_grad_clip_tensors(t, n, scale, None if out is None else table(*out)[0],
                                          None)


def test_pieces_and_workspace_of_a_list():
    pieces = grz.lib().dp_tensor_pieces
    assert pieces(*table()) == 0 and pieces(None, 0) == 0
    assert pieces(*table((A, 1), (0, 0), (B, 4096, H), (C, 4097))) == 4
    assert pieces(*table((A, -1))) == -INVALID and pieces(None, 1) == -INVALID
    assert pieces(*table((0, 1))) == -INVALID and pieces(*table((A, 1, N.GRZ_F64))) == -INVALID
    assert pieces(*table((A + 2, 1))) == -ALIGN and pieces(*table((A + 1, 1, H))) == -ALIGN
    assert pieces(*table((A, 2 ** 37))) == 2 ** 25
    assert pieces(*table((A, 2 ** 36), (B, 2 ** 36 + 1))) == -RANGE
    assert pieces(*table((A, 2 ** 63 - 1), (B, 2 ** 63 - 1))) == -RANGE
    size = grz.lib().dp_grad_sqnorm_tensors_workspace
    assert size(*table(), 0) == 0 and size(*table((A, 5)), 0) == 8
    assert size(*table((A, 5)), 4096) == 8 * (4097 + 2)
    assert size(*table((A, -5)), 0) == 0 and size(*table((A, 5)), -1) == 0
    assert size(*table((A, 5)), 4096 ** 3) == 0


def test_norm_of_a_list():
    one = [(A, 5000)]
    assert norm([(A, -1)]) == INVALID and norm([(A + 2, 4)]) == ALIGN
    assert norm(one, lead=-1) == INVALID and norm(one, lead=4096 ** 3) == RANGE
    assert norm(one, ws=None) == INVALID and norm(one, ws=W + 4) == ALIGN
    assert norm(one, sq=None, sc=None) == INVALID
    assert norm(one, sq=D + 4) == ALIGN and norm(one, sc=E + 2) == ALIGN
    assert norm(one, sq=A + 8) == INVALID and norm(one, sc=A + 19996) == INVALID
    assert norm(one, ws=A - 8) == INVALID and norm(one, sq=W + 8) == INVALID
    assert norm(one, sc=W + 12) == INVALID and norm(one, sq=D, sc=D + 4) == INVALID


def test_clip_of_lists():
    one = [(A, 100)]
    assert clip([(0, 4)]) == INVALID and clip(one, out=[(B, 99)]) == INVALID
    assert clip(one, out=[(B + 2, 100)]) == ALIGN and clip(one, scale=E + 2) == ALIGN
    assert clip(one, out=[(0, 100)]) == INVALID
    assert clip(one, scale=A + 8) == INVALID and clip(one, out=[(B, 100)], scale=B + 396) == INVALID
    assert clip([(A, 100), (A, 100)]) == INVALID                    # one twice
    assert clip([(A, 100), (A + 396, 100)]) == INVALID              # in part
    assert clip(one, out=[(A + 4, 100)]) == INVALID
    assert clip(one, out=[(A, 100, H)]) == INVALID                  # another type in place
    assert clip([(A, 10), (B, 10)], out=[(B, 10), (A, 10)]) == INVALID
    assert clip([(A, 10), (B, 10)], out=[(C, 10), (C + 36, 10)]) == INVALID
    assert clip([(A, 10), (B, 10)], out=[(A, 10), (A + 8, 10)]) == INVALID
    many = [(A + 400 * i, 100) for i in range(100)]
    assert clip(many + [(A + 400 * 50 + 396, 1)]) == INVALID
    assert clip(many[::-1] + [(A + 396, 2)]) == INVALID
    assert clip([]) == OK and clip([(A, 0), (A, 0)]) == OK and clip([], out=[]) == OK


def test_binding_refuses_what_the_library_cannot_see():
    f, w = torch.zeros(4, 8), torch.zeros(4, 2)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: grz.dp_expert_route(f, ids, w),
                 lambda: grz.dp_expert_route_grad(f, ids, w, f),
                 lambda: grz.dp_expert_sort(ids, 8, torch.zeros(9, dtype=torch.int32), ids),
                 lambda: grz.dp_expert_dispatch(f, ids, f),
                 lambda: grz.dp_expert_combine(f, ids, f),
                 lambda: grz.dp_expert_combine_grad(f, f, ids, w, dy=f),
                 lambda: grz.TensorList([f]),
                 lambda: grz.dp_grad_clip_tensors([f], None),
                 lambda: grz.dp_grad_sqnorm_tensors([], 1.0, f, None, None)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for call in (lambda: grz.dp_expert_route(None, ids, w), lambda: grz.TensorList([None]),
                 lambda: grz.dp_expert_sort([1], 8, None, None)):
        with pytest.raises(TypeError):
            call()


def test_layouts_of_a_list():
    from gradient_reduce_zero_amd.tensors import _one_run
    a = torch.zeros(6, 5, 4)
    for t in (a, a.permute(2, 0, 1), a.transpose(0, 1), a[2:3].transpose(0, 2),
              torch.zeros(3).expand(1, 3)):
        assert _one_run(t)
    for t in (a[:, :3], a[::2], a[:1].expand(6, 5, 4), a[..., 0], torch.zeros(1).expand(2)):
        assert not _one_run(t)


def test_structures_have_the_headers_layout():
    assert ctypes.sizeof(N.Tensor) == 24
    assert (N.Tensor.data.offset, N.Tensor.numel.offset, N.Tensor.dtype.offset) == (0, 8, 16)
