"""Small scales beside large ones in the same keys: the larger do not cost the smaller their bits."""

import pytest
import torch

from test_gpu_attention_q4 import Setup
from test_gpu_q4_precision import check, put_groups

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,Hq,Hkv,D", [(16, 4, 1, 128), (9, 1, 1, 64), (40, 4, 1, 64)])
def test_a_small_scale_beside_a_large_one(N, Hq, Hkv, D):
    s = Setup(61, [50, 0, 400], N, Hq, Hkv, D, 16, "f16")
    scale = torch.tensor([64.5 * 2.0 ** -20, 0.3, 1.0, 4.5])  # a sixteenth of the first lies between float16's steps
    put_groups(s.v, scale, -7.0 * scale)
    s.q /= 64  # scores near zero: what is left are the values' errors
    check(s, s.call(), only=sorted({0, N - 1}))
