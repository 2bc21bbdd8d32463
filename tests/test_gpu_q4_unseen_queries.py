"""Queries that are not finite, of tokens whose mask leaves nothing: zeros, as for any query
and any number of rows, over caches of 4 and of 16 bits."""

import math

import numpy as np
import pytest
import torch

from cache_helpers import mask_words
from test_gpu_attention_q4 import Setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("four", [True, False])
@pytest.mark.parametrize("N,Hq,D", [(2, 4, 64), (2, 8, 128), (8, 8, 128), (20, 8, 64), (70, 4, 128)])
def test_rows_that_see_nothing(N, Hq, D, four):
    s = Setup(71, [0, 40, 0], N, Hq, 2, D, 16, "bf16")
    if not four:
        s.k, s.v = (torch.randn(*x.shape[:3], D, device="cuda").to(torch.bfloat16) for x in (s.k, s.v))
    sees = np.tril(np.ones((3, N, N), bool))
    sees[0, 1] = False  # of a sequence without a context
    sees[2] = False
    kw = dict(tree_mask=s.dev(mask_words(sees)))
    clean = s.call(**kw)
    assert not clean.out[0, 1].any() and not clean.out[2].any()
    s.q[0, 1, 0] = math.nan
    s.q[0, 1, 1, 3] = math.inf
    s.q[2, 0, :, 5] = -math.inf
    s.q[1, 0, 1, 0] = math.nan  # sees its context
    res = s.call(**kw)
    assert torch.isnan(res.out[1, 0, 1]).all() and torch.isnan(res.lse[1, 0, 1])
    res.out[1, 0, 1], res.lse[1, 0, 1] = clean.out[1, 0, 1], clean.lse[1, 0, 1]
    assert torch.equal(res.out, clean.out) and torch.equal(res.lse, clean.lse)
