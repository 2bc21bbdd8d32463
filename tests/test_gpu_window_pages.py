"""Pages between the sinks and the window: no call needs them or flags them."""

import numpy as np
import pytest
import torch

import speculative_decoding_verification_temp_gb300 as sv

from cache_helpers import mask_words, visible
from test_gpu_paged_attention import KERNELS, Setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,N,Hq,Hkv,D,page", KERNELS)
def test_hidden_pages_are_not_looked_at(dtype, N, Hq, Hkv, D, page):
    ctx = [0, 50, 64, 65, 300, 1111]
    s = Setup(61, ctx, N, Hq, Hkv, D, page, dtype)
    whole = s.table.copy()
    tree = np.tril(np.ones((6, N, N), bool))
    some = False
    for window, sinks, masked in ((17, 0, False), (64, 4, False), (65, 40, True), (1, 1, False)):
        kw = dict(window=window, sinks=sinks)
        if masked:
            kw |= dict(tree_mask=s.dev(mask_words(tree)), position=s.dev(np.tile(np.arange(N), (6, 1))))
        want = s.call(**kw)
        assert not want.flags.any()
        seen = [np.array([visible(c, N, N, window=window, sinks=sinks).any(0)[t:t + page].any()
                          for t in range(0, c + N, page)]) for c in ctx]
        for away in (-1, s.k.shape[0], None):
            for b, shown in enumerate(seen):
                # given back, or another sequence's page by now
                s.table[b, :len(shown)][~shown] = s.table[0, 0] if away is None else away
                some |= not shown.all()
            res = s.call(**kw)
            assert not res.flags.any()
            assert torch.equal(res.out, want.out) and torch.equal(res.lse, want.lse)
            s.table[:] = whole
        # every page that a token sees is looked at
        for b, shown in enumerate(seen):
            for i in np.unique(np.flatnonzero(shown)[[0, -1, len(np.flatnonzero(shown)) // 2]]):
                s.table[b, i] = -1
                assert s.call(**kw).flags.tolist() == [sv.FLAG_BAD_PAGE if x == b else 0 for x in range(6)]
                s.table[:] = whole
    assert some
