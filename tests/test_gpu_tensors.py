"""The norm and the clip over many tensors on the GPU."""

import math

import pytest
import torch

import gradient_reduce_zero_amd as grz
from test_gpu_tokens import BF16, DEV, F32, gen

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -53
# Additions a square takes part in: 16 in its lane, 8 in its piece, 24 a level of the
# tree (two at most here), and as many again in the reference's own sums.
TERMS = 2 * (16 + 8 + 2 * 24)

LENGTHS = [1, 0, 7, 4095, 4096, 4097, 12289, 64, 100003, 2, 8192, 3 * 4096 + 8]


def tensors_of(lengths, seed, types=(BF16, F32), odd=True, std=0.02):
    """Tensors inside larger buffers, at odd elements; the buffers around hold 7."""
    out, bufs = [], []
    for i, n in enumerate(lengths):
        t = types[i % len(types)]
        at = 1 + i % 9 if odd else 8
        buf = torch.full((n + at + 16,), 7.0, device=DEV, dtype=t)
        buf[at:at + n] = torch.randn(n, device=DEV, generator=gen(seed + i)) * std
        out.append(buf[at:at + n])
        bufs.append((buf, at, n))
    return out, bufs


def around(bufs):
    return all((b[:at] == 7).all() and (b[at + n:] == 7).all() for b, at, n in bufs)


def exact(tensors):
    return math.fsum(float((t.double() ** 2).sum()) for t in tensors)


def norm_call(tensors, max_norm, lead=None):
    k = 0 if lead is None else len(lead)
    ws = torch.full((grz.dp_grad_sqnorm_tensors_workspace(tensors, k) // 8,), math.nan,
                    device=DEV, dtype=torch.float64)
    if k:
        ws[:k] = lead
    sq = torch.empty(1, device=DEV, dtype=torch.float64)
    scale = torch.empty(1, device=DEV)
    grz.dp_grad_sqnorm_tensors(tensors, max_norm, ws, sq, scale, lead=k)
    return sq.item(), scale.item(), ws


def factor(sq, max_norm):
    """The clip factor of a squared norm, as fp32."""
    norm = math.sqrt(sq)
    return torch.tensor(max_norm / norm if max_norm > 0 and norm > max_norm else 1.0).item()


@pytest.mark.parametrize("types", [(BF16,), (F32,), (BF16, F32)])
@pytest.mark.parametrize("odd", [False, True])
def test_norm_of_many_tensors(types, odd):
    ts, _ = tensors_of(LENGTHS * 20, 1, types, odd)  # more than one launch holds
    want = exact(ts)
    sq, scale, ws = norm_call(ts, 0.5)
    assert abs(sq - want) <= TERMS * EPS * want
    assert scale == factor(sq, 0.5)
    # Each tensor's pieces, in order.
    at = 0
    for t in ts:
        for lo in range(0, t.numel(), 4096):
            w = float((t[lo:lo + 4096].double() ** 2).sum())
            assert abs(ws[at].item() - w) <= TERMS * EPS * w
            at += 1
    assert at == grz.dp_tensor_pieces(ts)
    assert norm_call(ts, 0.0)[1] == 1.0 and norm_call(ts, 1e9)[1] == 1.0


@pytest.mark.parametrize("n", [1, 255, 4096, 4097, 50000, 4096 * 4096 + 5])
@pytest.mark.parametrize("shift", [0, 1, 4])
def test_one_tensor_has_the_bits_of_the_flat_norm(n, shift):
    x = torch.randn(n + shift, device=DEV, generator=gen(2))[shift:]
    ws = torch.empty(grz.dp_grad_sqnorm_of_workspace(n) // 8, device=DEV, dtype=torch.float64)
    sq = torch.empty(1, device=DEV, dtype=torch.float64)
    scale = torch.empty(1, device=DEV)
    grz.dp_grad_sqnorm_of(x, 1.0, ws, sq, scale)
    got = norm_call([x], 1.0)
    assert got[:2] == (sq.item(), scale.item())
    pieces = -(-n // 4096)
    assert torch.equal(got[2][:pieces], ws[:pieces])
    # bf16 elements: the pieces of the same values in fp32.
    b = x.to(BF16)
    wide = norm_call([b.float()], 1.0)
    assert norm_call([b], 1.0)[:2] == wide[:2]
    # Cut at piece borders, the list's pieces are the array's.
    if n > 4096:
        parts = [x[:4096], x[4096:]]
        assert norm_call(parts, 1.0)[:2] == got[:2]


def test_lead_pieces_join_the_norm():
    ts, _ = tensors_of(LENGTHS, 3)
    arena = torch.randn(30000, device=DEV, generator=gen(4)) * 0.1
    n = -(-arena.numel() // 4096)
    lead = norm_call([arena], 1.0)[2][:n].clone()
    both = norm_call([arena, *ts], 0.25)
    sq, scale, ws = norm_call(ts, 0.25, lead)
    assert (sq, scale) == both[:2]
    assert torch.equal(ws[:n], lead)
    # No tensors: the norm of the pieces; nothing at all: 0 and 1.
    assert norm_call([], 0.25, lead)[:2] == norm_call([arena], 0.25)[:2]
    assert norm_call([], 0.25)[:2] == (0.0, 1.0)


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf, 3e38, 1e-30])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_of_extreme_values(value, dtype):
    t = torch.ones(5000, device=DEV, dtype=dtype)
    t[4500] = value
    sq, scale, _ = norm_call([t[:10], t], 2.0)
    if math.isnan(value):
        assert math.isnan(sq) and scale == 1.0
    elif math.isinf(value):
        assert sq == math.inf and scale == 0.0
    else:  # squares beyond fp32's range
        want = 10 + 4999 + float(t[4500]) ** 2
        assert abs(sq - want) <= TERMS * EPS * want and scale == factor(sq, 2.0)


def test_a_tensor_listed_twice_counts_twice():
    t = torch.randn(6000, device=DEV, generator=gen(5))
    assert abs(norm_call([t, t], 1.0)[0] - 2 * exact([t])) <= TERMS * EPS * 2 * exact([t])


@pytest.mark.parametrize("ti", [(BF16,), (F32,), (BF16, F32)])
@pytest.mark.parametrize("to", [None, (BF16,), (F32,), (F32, BF16)])
@pytest.mark.parametrize("odd", [False, True])
def test_clip(ti, to, odd):
    lengths = LENGTHS * 14  # more than one launch holds
    ts, bufs = tensors_of(lengths, 6, ti, odd)
    outs, obufs = (None, None) if to is None else tensors_of(lengths, 7, to, not odd)
    scale = torch.tensor([0.37], device=DEV)
    kinds = [t.dtype for t in (ts if to is None else outs)]
    want = [(t.float() * scale).to(k) for t, k in zip(ts, kinds)]
    old = [t.clone() for t in ts]
    grz.dp_grad_clip_tensors(ts, scale, out=outs)
    for t, w in zip(ts if to is None else outs, want):
        assert torch.equal(t, w)
    assert around(bufs)
    if to is not None:
        assert around(obufs) and all(torch.equal(a, b) for a, b in zip(ts, old))


@pytest.mark.parametrize("in_place", [False, True])
def test_clip_by_one_and_without_a_factor(in_place):
    ts, bufs = tensors_of(LENGTHS, 8)
    ts[3][5] = math.nan
    old = [t.clone() for t in ts]
    for scale in (torch.ones(1, device=DEV), None):
        outs = None if in_place else [torch.zeros_like(t) for t in ts]
        grz.dp_grad_clip_tensors(ts, scale, out=outs)
        for t, o in zip(ts if in_place else outs, old):
            assert torch.equal(torch.nan_to_num(t.float(), 99.0),
                               torch.nan_to_num(o.float(), 99.0))
    assert around(bufs)


@pytest.mark.parametrize("value", [0.0, math.nan, math.inf])
def test_clip_by_extreme_factors(value):
    ts = [torch.tensor([1.0, -2.0, 0.0, math.inf], device=DEV).to(t) for t in (F32, BF16)]
    s = torch.tensor([value], device=DEV)
    want = [(t.float() * s).to(t.dtype) for t in ts]
    grz.dp_grad_clip_tensors(ts, s)
    for t, w in zip(ts, want):
        assert torch.equal(torch.nan_to_num(t.float(), 99.0, 1e30, -1e30),
                           torch.nan_to_num(w.float(), 99.0, 1e30, -1e30))


def test_clip_of_large_tensors_past_the_caches():
    # Enough bytes to be streamed; and the norm after it is the wanted one.
    ts = [torch.randn(n, device=DEV, generator=gen(9)).to(t)
          for n, t in ((60_000_001, BF16), (40_000_003, F32))]
    sq, scale, _ = norm_call(ts, 1.0)
    want = exact(ts)
    assert abs(sq - want) <= 1e-12 * want
    s = torch.tensor([scale], device=DEV)
    expected = [(t.float() * s).to(t.dtype) for t in ts]
    outs = [torch.empty_like(t) for t in ts]
    grz.dp_grad_clip_tensors(ts, s, out=outs)
    grz.dp_grad_clip_tensors(ts, s)
    for t, o, e in zip(ts, outs, expected):
        assert torch.equal(t, e) and torch.equal(o, e)


def test_a_tensor_beyond_32_bit_offsets():
    n = 2 ** 32 + 4099
    t = torch.zeros(n, device=DEV, dtype=BF16)
    t[-1], t[2 ** 31 + 5], t[0] = 3.0, 4.0, 12.0
    sq, scale, _ = norm_call([t], 6.5)
    assert (sq, scale) == (169.0, 0.5)
    grz.dp_grad_clip_tensors([t], torch.tensor([scale], device=DEV))
    assert (t[-1].item(), t[2 ** 31 + 5].item(), t[0].item()) == (1.5, 2.0, 6.0)
    assert norm_call([t], 0.0)[0] == 42.25


def test_more_pieces_than_one_launch_takes():
    # A launch ends inside the second tensor, at a piece's border (2^22 pieces).
    n = 4096 * (2 ** 22 - 1) + 9000
    a = torch.ones(10, device=DEV, dtype=BF16)
    t = torch.zeros(n, device=DEV, dtype=BF16)
    edge = 4096 * (2 ** 22 - 1)
    t[edge - 1], t[edge], t[-1], t[0] = 3.0, 4.0, 12.0, 1.0
    b = torch.full((5,), 2.0, device=DEV)
    sq, scale, ws = norm_call([a, t, b], 7.0)
    assert (sq, scale) == (200.0, torch.tensor(7.0 / math.sqrt(200.0)).item())
    assert grz.dp_tensor_pieces([a, t, b]) == 2 ** 22 + 2 + 2
    assert ws[2 ** 22 - 1].item() == 9.0 and ws[2 ** 22].item() == 16.0
    assert ws[2 ** 22 + 2].item() == 144.0 and ws[2 ** 22 + 3].item() == 20.0
    grz.dp_grad_clip_tensors([a, t, b], torch.tensor([0.5], device=DEV))
    assert [t[i].item() for i in (edge - 1, edge, -1, 0)] == [1.5, 2.0, 6.0, 0.5]
    assert (a == 0.5).all() and (b == 1.0).all()
    assert norm_call([a, t, b], 0.0)[0] == 50.0


def test_orders_of_dimensions_and_refused_layouts():
    a = torch.randn(30, 40, 5, device=DEV, generator=gen(10))
    ts = [a.permute(2, 0, 1), a.transpose(0, 1).contiguous().transpose(0, 1)[:, :, :]]
    want = exact(ts)
    assert abs(norm_call(ts, 1.0)[0] - want) <= TERMS * EPS * want
    expected = ts[0] * 0.5
    grz.dp_grad_clip_tensors([ts[0]], torch.tensor([0.5], device=DEV))
    assert torch.equal(ts[0], expected)
    for bad in (a[:, :39], a[::2], a[:1].expand(30, 40, 5)):
        with pytest.raises(ValueError, match="apart"):
            grz.TensorList([bad])
    with pytest.raises(ValueError, match="strides"):
        grz.dp_grad_clip_tensors([a], None,
                                 out=[torch.empty(5, 40, 30, device=DEV).permute(2, 1, 0)])
    with pytest.raises(ValueError, match="shape"):
        grz.dp_grad_clip_tensors([a], None, out=[torch.empty(30, 200, device=DEV)])
    with pytest.raises(ValueError):
        grz.dp_grad_clip_tensors([a], None, out=[a, a])
    with pytest.raises(TypeError):
        grz.TensorList([a.double()])
    with pytest.raises(ValueError, match="GPU"):
        grz.TensorList([a, torch.zeros(3)])


def test_overlaps_are_refused():
    a = torch.zeros(10000, device=DEV)
    s = torch.ones(1, device=DEV)
    for ts, outs in (([a, a], None), ([a[:100], a[99:200]], None),
                     ([a[:100]], [a[1:101]]), ([a[:50], a[50:100]], [a[50:100], a[:50]]),
                     ([a[:50], a[60:70]], [a[:50], a[40:50]])):
        with pytest.raises(grz.GrzError):
            grz.dp_grad_clip_tensors(ts, s, out=outs)
    with pytest.raises(grz.GrzError):  # the factor inside an output
        grz.dp_grad_clip_tensors([a], a[5:6])
    many = list(a.split(100))
    with pytest.raises(grz.GrzError):
        grz.dp_grad_clip_tensors(many + [a[350:351]], s)
    grz.dp_grad_clip_tensors(many, s)
    grz.dp_grad_clip_tensors([a[:50], a[50:100]], s, out=[a[:50], a[200:250]])
    ws = torch.empty(16, device=DEV, dtype=torch.float64)
    sq, sc = torch.empty(1, device=DEV, dtype=torch.float64), torch.empty(1, device=DEV)
    with pytest.raises(grz.GrzError):
        grz.dp_grad_sqnorm_tensors([a], 1.0, ws, ws[1:2], sc)
    with pytest.raises(grz.GrzError):
        grz.dp_grad_sqnorm_tensors([a], 1.0, ws, sq, a[3:4])
    with pytest.raises(ValueError, match="workspace"):
        grz.dp_grad_sqnorm_tensors([a], 1.0, ws[:2], sq, sc)
    with pytest.raises(TypeError):
        grz.dp_grad_sqnorm_tensors([a], 1.0, ws, sc, sc)


def test_captured_with_its_list_and_replayed():
    ts, _ = tensors_of(LENGTHS * 20, 11)
    ws = torch.empty(grz.dp_grad_sqnorm_tensors_workspace(ts) // 8, device=DEV,
                     dtype=torch.float64)
    sq, sc = torch.empty(1, device=DEV, dtype=torch.float64), torch.empty(1, device=DEV)

    def step():
        grz.dp_grad_sqnorm_tensors(ts, 1.0, ws, sq, sc)
        grz.dp_grad_clip_tensors(ts, sc)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        for j, t in enumerate(ts):
            t.copy_(torch.randn(t.numel(), device=DEV, generator=gen(100 * i + j)))
        old = [t.clone() for t in ts]
        want = norm_call(old, 1.0)
        graph.replay()
        torch.cuda.synchronize()
        assert (sq.item(), sc.item()) == want[:2]
        for t, o in zip(ts, old):
            assert torch.equal(t, (o.float() * sc).to(t.dtype))


def test_lists_on_two_streams():
    sets = [tensors_of([500_000 + i, 70_000, 3], 20 + i)[0] for i in range(2)]
    want = [norm_call(ts, 1.0)[:2] for ts in sets]
    ws = [torch.empty(grz.dp_grad_sqnorm_tensors_workspace(ts) // 8, device=DEV,
                      dtype=torch.float64) for ts in sets]
    out = [(torch.empty(1, device=DEV, dtype=torch.float64), torch.empty(1, device=DEV))
           for _ in sets]
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        for ts, w, (sq, sc), s in zip(sets, ws, out, streams):
            grz.dp_grad_sqnorm_tensors(grz.TensorList(ts), 1.0, w, sq, sc, stream=s)
    torch.cuda.synchronize()
    assert [(sq.item(), sc.item()) for sq, sc in out] == want
