"""Integer tensors wider than 32 bits: what does not fit is flagged, not wrapped
into a page, a length or a node that exists."""

import numpy as np
import pytest
import torch

import speculative_decoding_verification_temp_gb300 as sv

from test_gpu_paged_attention import Setup

pytestmark = pytest.mark.gpu

FAR = 2 ** 32


def wide(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int64).cuda()


@pytest.mark.parametrize("dtype,N", [("bf16", 1), ("f32", 3), ("f16", 40)])
def test_attention(dtype, N):
    s = Setup(51, [40, 40, 40], N, 4, 2, 64, 16, dtype)
    table, ctx = wide(s.table), wide(s.ctx)
    want = s.call()
    got = sv.paged_attention(s.q, s.k, s.v, table, ctx, return_lse=True, return_flags=True)
    assert torch.equal(got.out, want.out) and not got.flags.any()
    table[1, 1] += FAR
    ctx[2] += FAR
    got = sv.paged_attention(s.q, s.k, s.v, table, ctx, num_new=wide([N, N, N]), return_lse=True,
                             return_flags=True)
    assert got.flags.tolist() == [0, sv.FLAG_BAD_PAGE, sv.FLAG_BAD_LENGTH]
    assert torch.equal(got.out[0], want.out[0]) and not torch.equal(got.out[1], want.out[1])
    assert (got.out[2] == 0).all() and (got.lse[2] == -torch.inf).all()
    got = sv.paged_attention(s.q, s.k, s.v, s.dev(s.table), s.dev(s.ctx),
                             num_new=wide([N + FAR, N, -FAR + N]), return_flags=True)
    assert got.flags.tolist() == [sv.FLAG_BAD_LENGTH, 0, sv.FLAG_BAD_LENGTH]
    assert torch.equal(got.out[:2], want.out[:2])


def test_pages_and_paths():
    pool = sv.page_pool(4, 8, 32)
    assert not sv.cache_resize(pool, wide([40, 40, 40, 0]), 16).any()
    flags = sv.cache_resize(pool, wide([40, 40 + FAR, 40 - FAR, 0]), 16)
    assert flags.tolist() == [0, sv.FLAG_BAD_LENGTH, sv.FLAG_BAD_LENGTH, 0]
    assert pool.page_count.tolist() == [3, 3, 3, 0]
    k, v = (torch.randn(32, 16, 2, 64, device="cuda") for _ in "kv")
    before = k.clone(), v.clone()
    new = torch.randn(4, 2, 2, 64, device="cuda")
    flags = sv.cache_append(new, new, k, v, pool.page_table, wide([20 + FAR, -FAR, 8 + FAR, FAR]),
                            return_flags=True)
    assert flags.tolist() == [sv.FLAG_BAD_LENGTH] * 4
    path, taken = wide([[0, 3], [0, 3 + FAR], [FAR, 3], [0, 3]]), wide([1 + FAR, 1, 1, -1 - FAR])
    res = sv.cache_compact(k, v, pool.page_table, wide([8, 8, 8, 8]), path, taken)
    assert res.flags[[0, 2, 3]].tolist() == [sv.FLAG_BAD_TREE] * 3 and res.flags[1] != 0
    assert res.context_len.tolist() == [8] * 4
    ctx = torch.tensor([40, 40, 40, 0], dtype=torch.int32, device="cuda")
    flags = sv.cache_fork(pool, k, v, ctx, wide([FAR, 0]), wide([3, 3 + FAR]))
    assert flags.tolist() == [sv.FLAG_BAD_SEQUENCE] * 2
    assert torch.equal(k, before[0]) and torch.equal(v, before[1])
