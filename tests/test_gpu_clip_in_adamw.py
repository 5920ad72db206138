"""Tensors of their own in AdamW: handed the unclipped gradient and the factor, it gives
the bits it gives for the clipped gradient, and the oracle's."""

import numpy as np
import pytest
import torch

import gradient_reduce_zero_amd as grz
from oracle.step import Hyper as OracleHyper, adamw
from test_gpu_tokens import DEV, gen

pytestmark = pytest.mark.gpu


def test_factor_in_adamw_is_the_clip():
    grads = [torch.randn(n, device=DEV, generator=gen(n)) for n in (1, 4096, 70001)]
    sq, scale = torch.empty(1, device=DEV, dtype=torch.float64), torch.empty(1, device=DEV)
    ws = torch.empty(grz.dp_grad_sqnorm_tensors_workspace(grads) // 8, device=DEV,
                     dtype=torch.float64)
    grz.dp_grad_sqnorm_tensors(grads, 0.25, ws, sq, scale)
    assert 0 < scale.item() < 0.01
    clipped = [torch.empty_like(t) for t in grads]
    grz.dp_grad_clip_tensors(grads, scale, out=clipped)
    hyper = grz.Hyper(max_norm=0.25)
    for raw, small in zip(grads, clipped):
        start = [torch.randn(raw.numel(), device=DEV, generator=gen(9 + i)) for i in range(3)]
        start[1] *= 1e-4                              # moments of the clipped size
        start[2] = start[2] ** 2 * 1e-8
        results = []
        for g, factor in ((raw, scale), (small, None)):
            w, m, v = (t.clone() for t in start)
            for t in (1, 2):
                args = grz.adamw_args(**grz.step_scalars(hyper, t))
                grz.zero1_adamw_step(w, m, v, g, factor, args)
            results.append((w, m, v))
        for a, b in zip(*results):
            assert torch.equal(a, b)
        # The oracle's, of the product in fp32.
        host = [t.cpu().numpy() for t in start]
        g = raw.cpu().numpy() * np.float32(scale.item())
        for t in (1, 2):
            host = adamw(*host, g, **OracleHyper(max_norm=0.25).scalars(t))
        for a, b in zip(results[0], host):
            assert np.array_equal(a.cpu().numpy(), b)
        # An unclipped gradient without the factor leads elsewhere.
        w, m, v = (t.clone() for t in start)
        grz.zero1_adamw_step(w, m, v, raw, None, grz.adamw_args(**grz.step_scalars(hyper, 1)))
        assert not torch.equal(m, results[0][1]) and not torch.equal(v, results[0][2])
