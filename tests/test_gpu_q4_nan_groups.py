"""A group of NaNs beside groups of large scales in a row of values that every token sees."""

import math

import pytest
import torch

from test_gpu_attention_q4 import Setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [1000.0, 8000.0])
@pytest.mark.parametrize("N,Hq,D", [(1, 4, 64), (1, 4, 128), (2, 4, 64), (2, 4, 128), (1, 8, 128), (16, 4, 128)])
def test_other_groups_of_the_row(N, Hq, D, scale):
    s = Setup(41, [300], N, Hq, 1, D, 16, "bf16")
    s.q.fill_(1.0)
    for g in range(4):
        s.put(s.k, 0, 7, 0, g, 0.0, 12 / math.sqrt(D))  # 12 nats: the largest weight
        if g != 2:
            s.put(s.v, 0, 7, 0, g, scale / 2 ** g, -2.0 * scale / 2 ** g)
    s.put(s.v, 0, 7, 0, 2, math.nan, math.nan)
    res = s.call()
    each = D // 4
    assert torch.isnan(res.out[..., 2 * each:3 * each]).all()
    s.put(s.v, 0, 7, 0, 2, 0.0, 0.0)
    clean = s.call()
    out = res.out.clone()
    out[..., 2 * each:3 * each] = clean.out[..., 2 * each:3 * each]
    s.check(type(res)(out, res.lse, res.flags))
