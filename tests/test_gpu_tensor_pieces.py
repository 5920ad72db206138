"""Piece sums of tensor lists past the few pieces that take a workgroup each: the bits of
the flat norm's pieces, whatever the type, the place in memory and the call."""

import pytest
import torch

import gradient_reduce_zero_amd as grz
from test_gpu_tensors import norm_call
from test_gpu_tokens import BF16, DEV, F32, gen

pytestmark = pytest.mark.gpu
PIECE = 4096
FEW = 6144  # pieces of a launch that take a workgroup each


def flat(x):
    """(squared norm, factor, piece sums) of dp_grad_sqnorm_of."""
    ws = torch.empty(grz.dp_grad_sqnorm_of_workspace(x.numel()) // 8, device=DEV,
                     dtype=torch.float64)
    sq, scale = torch.empty(1, device=DEV, dtype=torch.float64), torch.empty(1, device=DEV)
    grz.dp_grad_sqnorm_of(x, 1.0, ws, sq, scale)
    return sq.item(), scale.item(), ws[:-(-x.numel() // PIECE)].clone()


def pieces(tensors):
    out = norm_call(tensors, 1.0)
    return out[0], out[1], out[2][:grz.dp_tensor_pieces(tensors)].clone()


# fp32: 96 MiB and more, read past the caches.  bf16: half of that, through them; and
# twice as many elements, past them.
@pytest.mark.parametrize("dtype,times", [(F32, 1), (BF16, 1), (BF16, 2)])
@pytest.mark.parametrize("shift", [0, 1, 5])
@pytest.mark.parametrize("rest", [777, 4095, 1])
def test_a_wave_a_piece_has_the_flat_norms_bits(dtype, times, shift, rest):
    n = times * FEW * PIECE + 2 * PIECE + rest
    x = torch.randn(n + shift, device=DEV, generator=gen(1)).to(dtype)[shift:]
    want = flat(x.float())
    got = pieces([x])
    assert torch.equal(got[2], want[2]) and got[:2] == want[:2]
    # The same pieces from two calls below the limit each, and from one list.
    half = (FEW // 2) * PIECE
    parts = [x[i:i + half] for i in range(0, n, half)]
    assert all(-(-p.numel() // PIECE) <= FEW for p in parts)
    assert torch.equal(torch.cat([pieces([p])[2] for p in parts]), want[2])
    assert torch.equal(pieces(parts)[2], want[2])


@pytest.mark.parametrize("types", [(F32,), (BF16, F32)])
def test_tensors_with_short_last_pieces(types):
    # 184 tensors in one launch of more than 6144 pieces, below 96 MiB: read through the
    # caches, each one's last piece a single element or a few.
    lengths = [33 * PIECE + 1 + i % 7 for i in range(184)]
    ts = [(torch.randn(n + 3, device=DEV, generator=gen(i)).to(types[i % len(types)]))[i % 4:][:n]
          for i, n in enumerate(lengths)]
    assert grz.dp_tensor_pieces(ts) == 184 * 34 > FEW
    assert sum(t.numel() * t.element_size() for t in ts) < 96 * 2 ** 20
    assert torch.equal(pieces(ts)[2], torch.cat([flat(t.float().contiguous())[2] for t in ts]))
