"""Values over the whole range of 4-bit rows, where a tile is not seen whole: the last
keys of a context, new tokens, trees and windows."""

import numpy as np
import pytest
import torch

import speculative_decoding_verification_temp_gb300 as sv

from cache_helpers import random_trees
from test_gpu_attention_q4 import Setup

pytestmark = pytest.mark.gpu

# (scale, minimum) of the four groups: values between -61440 and 61440, -30000 and 30000,
# -22000 and 22000, -32992 and 8
SPANS = [(8192.0, -61440.0), (4000.0, -30000.0), (2934.0, -22000.0), (2200.0, -32992.0)]


def put_groups(cache, spans):
    """The groups' scales and minima in every row that is not one of NaN."""
    D = (cache.shape[-1] - 16) * 2
    pair = cache[..., D // 2:].contiguous().view(torch.float16).unflatten(-1, (4, 2))
    new = torch.tensor(spans, device="cuda").half().expand_as(pair)
    pair = torch.where(torch.isnan(pair), pair, new)
    cache[..., D // 2:] = pair.flatten(-2).contiguous().view(torch.uint8)


SIZES = [(1, 4, 2, 64), (1, 8, 2, 128), (1, 8, 1, 64), (2, 8, 2, 128), (6, 4, 2, 64), (8, 8, 2, 128), (16, 8, 2, 128),
         (16, 8, 2, 64), (40, 8, 2, 64), (40, 8, 2, 128)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("N,Hq,Hkv,D", SIZES)
def test_groups_that_span_zero(N, Hq, Hkv, D, dtype):
    s = Setup(31, [50, 0, 700, 31], N, Hq, Hkv, D, 16, dtype)
    put_groups(s.v, SPANS)
    s.check(s.call())
    s.check(s.call(window=20, sinks=3), window=20, sinks=3)


@pytest.mark.parametrize("N,Hq,Hkv,D", [(6, 2, 1, 128), (12, 4, 2, 64), (40, 4, 2, 128)])
def test_over_trees(N, Hq, Hkv, D):
    s = Setup(32, [50, 0, 200], N, Hq, Hkv, D, 16, "bf16")
    put_groups(s.v, SPANS)
    mk = sv.tree_mask(s.dev(random_trees(s.rng, 3, N)), N)
    sees = np.unpackbits(mk.mask.cpu().numpy().view(np.uint8), axis=-1, bitorder="little").reshape(3, N, -1)
    s.check(s.call(tree_mask=mk.mask), sees=sees[:, :, :N].astype(bool))


@pytest.mark.parametrize("N,Hq,Hkv,D", [(1, 4, 2, 64), (1, 8, 1, 128), (9, 8, 2, 128), (40, 8, 2, 64)])
def test_groups_whose_unused_codes_lie_beyond_float16(N, Hq, Hkv, D):
    """Codes up to 11 of a scale of 5000: values up to 55000, code 15 would be 75000."""
    s = Setup(33, [50, 0, 300], N, Hq, Hkv, D, 16, "bf16")
    s.v[..., :D // 2] &= 0xBB
    put_groups(s.v, [(5000.0, 0.0), (0.3, -2.0), (5200.0, -100.0), (1.0, 0.0)])
    s.check(s.call())


@pytest.mark.parametrize("N,Hq,Hkv,D", [(1, 4, 2, 64), (1, 8, 1, 128), (9, 8, 2, 128), (40, 8, 2, 64)])
def test_appended(N, Hq, Hkv, D):
    """The same through the writer: rows of -30000 .. 30000 appended and read by attention."""
    s = Setup(34, [50, 0, 300], N, Hq, Hkv, D, 16, "bf16")
    gen = torch.Generator("cuda")
    gen.manual_seed(34)
    new = [torch.randn(3, N, Hkv, D, generator=gen, device="cuda") for _ in "kv"]
    values = ((torch.rand(3, N, Hkv, D, generator=gen, device="cuda") * 2 - 1) * 30000).to(torch.bfloat16)
    sv.cache_append(new[0].to(torch.bfloat16), values, s.k, s.v, s.dev(s.table), s.dev(s.ctx))
    s.check(s.call())
