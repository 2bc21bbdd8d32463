"""A score that is NaN reaches the rows that see its key and no others, however
their keys are dealt out to warps, lane quarters and pieces of cut units."""

import math

import numpy as np
import pytest
import torch

from test_gpu_paged_attention import KERNELS, WHOLE, Setup

pytestmark = pytest.mark.gpu


def check_rows(s, res, clean, rows):
    """rows [B, N, Hq]: out and lse are NaN there, the bits of `clean` elsewhere."""
    rows = torch.from_numpy(rows).cuda()
    assert torch.isnan(res.out[rows]).all() and torch.isnan(res.lse[rows]).all()
    assert torch.equal(res.out[~rows], clean.out[~rows])
    assert torch.equal(res.lse[~rows], clean.lse[~rows])
    assert torch.isfinite(clean.out).all() and torch.isfinite(clean.lse).all()


# contexts, and whether the page table is so wide that units are cut: into one,
# more than 16, up to 16 and (most of them) two or three pieces
BATCHES = {"whole": ([3, 0, 20, 9], False), "many": ([9000], True), "some": ([1500, 1100, 30], True),
           "few": ([700] * 90, True)}


@pytest.mark.parametrize("batch", list(BATCHES))
@pytest.mark.parametrize("kernel", list(zip(KERNELS, WHOLE)), ids=str)
def test_a_query_with_a_nan(kernel, batch):
    (dtype, N, Hq, Hkv, D, page), tokens = kernel
    ctx, wide = BATCHES[batch]
    if not wide:
        ctx = [min(c, tokens // page * page - N) for c in ctx]
    s = Setup(41, ctx, N, Hq, Hkv, D, page, dtype,
              max_pages=-(-(max(ctx) + N + 4096) // page) if wide else tokens // page)
    clean = s.call()
    rows = np.zeros(s.q.shape[:3], bool)
    for b in range(len(ctx)):
        n, h = b % N, 3 * b % Hq
        s.q[b, n, h, (7 * b) % D] = math.nan
        rows[b, n, h] = True
    check_rows(s, s.call(), clean, rows)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("kernel", list(zip(KERNELS, WHOLE)), ids=str)
def test_a_key_with_a_nan_alone_in_its_share(kernel, wide):
    """The last new token's key, which that token alone sees, at places that are the
    first of a warp's, a quarter's, a tile's and a piece's keys, and at others."""
    (dtype, N, Hq, Hkv, D, page), tokens = kernel
    places = [0, 1, 4, 8, 12, 16, 31, 32, 33, 48, 64, 96, 100, 128, 192, 256, 384, 640, 2048, 4097]
    ctx = [p - N + 1 for p in places if p >= N - 1 and (wide or p < tokens // page * page)]
    assert ctx
    s = Setup(42, ctx, N, Hq, Hkv, D, page, dtype,
              max_pages=-(-(max(ctx) + N + 4096) // page) if wide else tokens // page)
    clean = s.call()
    rows = np.zeros(s.q.shape[:3], bool)
    rows[:, N - 1, :Hq // Hkv] = True  # the query heads of key head 0
    for b, c in enumerate(ctx):
        p, i = s.slot(b, c + N - 1)
        s.k[p, i, 0, (5 * b) % D] = math.nan
    check_rows(s, s.call(), clean, rows)


@pytest.mark.parametrize("dtype,N,Hq,Hkv,D,page", KERNELS)
def test_a_context_of_nan_keys(dtype, N, Hq, Hkv, D, page):
    """Every key of one head: no finite score stands beside a NaN anywhere."""
    s = Setup(43, [40, 700, 2600], N, Hq, Hkv, D, page, dtype)
    clean = s.call()
    for b, c in enumerate(s.ctx):
        for t in range(0, int(c) + N, page):
            p = int(s.table[b, t // page])
            s.k[p, :, 0] = math.nan
    rows = np.zeros(s.q.shape[:3], bool)
    rows[:, :, :Hq // Hkv] = True
    check_rows(s, s.call(), clean, rows)


@pytest.mark.parametrize("dtype,N,Hq,Hkv,D,page", KERNELS)
def test_a_score_of_plus_infinity(dtype, N, Hq, Hkv, D, page):
    """exp(inf - inf): NaN, as in the definition's quotient."""
    s = Setup(44, [31, 640, 2047], N, Hq, Hkv, D, page, dtype)
    s.q[:] = s.q.abs() + 0.5
    clean = s.call()
    rows = np.zeros(s.q.shape[:3], bool)
    for b, c in enumerate(s.ctx):
        p, i = s.slot(b, int(c) + N - 1)
        s.k[p, i, 0, b] = math.inf
    rows[:, N - 1, :Hq // Hkv] = True
    check_rows(s, s.call(), clean, rows)
