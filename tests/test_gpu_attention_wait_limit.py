"""Bounded waits of the attention kernels on tensor memory that run out, on
purpose and without a fault: set_wait_limit(0) makes a thread block's first wait
for keys one test, which fails while they are on their way.  The block lets
its copies and products finish, frees its tensor memory and ends; the call
returns, and the next one is as the one before."""

import numpy as np
import pytest
import torch

import speculative_decoding_verification_temp_gb300 as sv

from test_gpu_paged_attention import KERNELS, WHOLE, Setup

pytestmark = pytest.mark.gpu

WIDE = [(k, t) for k, t in zip(KERNELS, WHOLE) if k[0] != "f32" and k[4] in (64, 128) and k[5] % 8 == 0]


def short_wait(call):
    try:
        sv.set_wait_limit(0)
        res = call()
        torch.cuda.synchronize()
    finally:
        sv.set_wait_limit(None)
    return res


# one sequence of one tile; whole units; cut ones; more units than thread blocks
BATCHES = {"one": [5], "whole": [100, 0, 300], "cut": [5000, 40, 0, 2000], "many": [200] * 200}


@pytest.mark.parametrize("batch", list(BATCHES))
@pytest.mark.parametrize("kernel", WIDE, ids=str)
def test_wait_runs_out_then_recovers(kernel, batch):
    (dtype, N, Hq, Hkv, D, page), tokens = kernel
    ctx = BATCHES[batch]
    n_new = np.full(len(ctx), N)
    n_new[1::3] = 0
    s = Setup(71, ctx, N, Hq, Hkv, D, page, dtype, n_new=n_new,
              max_pages=tokens // page if batch in ("one", "whole") else None)
    before = s.call(out=torch.zeros_like(s.q))
    assert not before.flags.any()
    given_up = short_wait(lambda: s.call())
    assert given_up.flags.tolist() == [sv.FLAG_TIMEOUT if n else 0 for n in n_new]
    after = s.call(out=torch.zeros_like(s.q))
    assert not after.flags.any() and torch.equal(after.out, before.out)
    for b, n in enumerate(n_new):
        assert torch.equal(after.lse[b, :n], before.lse[b, :n])


@pytest.mark.parametrize("batch", list(BATCHES))
@pytest.mark.parametrize("kernel", WIDE, ids=str)
def test_no_answer_without_flags(kernel, batch):
    """Without flags the outputs themselves say that a wait gave up."""
    (dtype, N, Hq, Hkv, D, page), tokens = kernel
    ctx = BATCHES[batch]
    n_new = np.full(len(ctx), N)
    n_new[1::3] = N // 2
    s = Setup(73, ctx, N, Hq, Hkv, D, page, dtype, n_new=n_new,
              max_pages=tokens // page if batch in ("one", "whole") else None)
    out = torch.full_like(s.q, 3.0)
    res = short_wait(lambda: sv.paged_attention(s.q, s.k, s.v, s.dev(s.table), s.dev(s.ctx),
                                                num_new=s.dev(s.n_new), return_lse=True, out=out))
    for b, n in enumerate(n_new):
        assert torch.isnan(res.out[b, :n]).all() and torch.isnan(res.lse[b, :n]).all()
        assert (res.out[b, n:] == 3.0).all()


def test_other_kernels_make_no_such_wait():
    for dtype, N, Hq, Hkv, D, page in (k for k in KERNELS if k not in [x for x, _ in WIDE]):
        s = Setup(72, [100, 0], N, Hq, Hkv, D, page, dtype)
        want = s.call()
        got = short_wait(s.call)
        assert not got.flags.any() and torch.equal(got.out, want.out)
