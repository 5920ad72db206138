"""Token operators on the GPU: orders, layouts and uses at the edges of what their
entry points promise."""

import math

import pytest
import torch

import gradient_reduce_zero_amd as grz
from test_gpu_tokens import BF16, DEV, F32, logits_of, logprob_call, order_of

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
