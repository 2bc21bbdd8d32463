"""Attention over a paged cache of 4-bit rows against a plain 64-bit computation on
what the rows stand for: types, head layouts, page sizes, lengths from none to many
splits, chains, trees, windows with sinks, ragged batches, and what must not be read."""

import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_temp_gb300 as sv

from cache_helpers import DTYPES, attention_reference, make_pages, mask_words, random_trees, visible
from rows_helpers import half_step, stands_for

pytestmark = pytest.mark.gpu


def tolerance(out, lse, mean, reach, vmax, T, D, dtype, wide):
    """Bounds on |out| and |lse| errors.

    As attention_tolerance() for float16 weights of up to 2^15, those below 2^-24 times
    that lost (2^-32 of the largest, of a sum of at least 1: T 2^-32 vmax, and half of
    float16's smallest step for each), and two things more.  Values enter as float16:
    half a step of a value, (|m| + 15 s) 2^-11 at most, which is 2^-11 vmax' for the
    largest magnitude vmax' <= 3 vmax of a group's ends (a value that is seen and the
    group's whole span, of which each end is within a step of some value: vmax is taken
    over the row's seen values of all dimensions).  Scores: on the exact codes the
    queries' float16 (2^-24 of a row's largest), two terms of their sums (2^-22), the
    sums' float32; in the kernels on tensor memory keys are float16 as the values are (both
    a sixteenth, so that magnitudes below 2^-10 are off by 2^-21, which the 1 % that reach
    is taken larger covers for keys of 2^-4 on average), each product
    off by 2^-11 of |q| times a key's magnitude: reach 2^-11.
    """
    d = (D + 16) * 2.0 ** -22 * reach + 2.0 ** -20 + T * 2.0 ** -23
    if wide:
        d = d + reach * 2.0 ** -11 * 1.01
    tol = (mean + out.abs()) * (d[..., None] + 2.0 ** -22) + out.abs() * half_step(dtype) * (1 + 2.0 ** -6)
    tol = tol + mean * 2.0 ** -11 * (1 + 2.0 ** -6) + 3 * 2.0 ** -12 * vmax[..., None]
    tol = tol + (T * 2.0 ** -31 * vmax + 2.0 ** -25)[..., None]
    return tol, d + 2.0 ** -22 * (1 + lse.abs())


class Setup:
    """Inputs of a call; every slot behind a sequence's tokens holds rows of NaN."""

    def __init__(self, seed, ctx, N, Hq, Hkv, D, page, dtype, n_new=None, layout="hnd", max_pages=None):
        rng = np.random.default_rng(seed)
        gen = torch.Generator("cuda")
        gen.manual_seed(seed)
        self.rng, self.page, self.dtype, self.N = rng, page, dtype, N
        self.ctx = np.asarray(ctx, np.int32)
        B = len(self.ctx)
        self.n_new = None if n_new is None else np.asarray(n_new, np.int32)
        lens = self.ctx + (N if n_new is None else self.n_new)
        self.table, pages = make_pages(rng, lens, page, max_pages)
        row = D // 2 + 16

        def cache():
            codes = torch.randint(0, 256, (pages, page, Hkv, D // 2), generator=gen, device="cuda", dtype=torch.uint8)
            scale = torch.rand((pages, page, Hkv, 4), generator=gen, device="cuda") * 0.4 + 0.05
            low = torch.randn((pages, page, Hkv, 4), generator=gen, device="cuda") * 0.7 - 7.5 * scale
            pair = torch.stack([scale, low], -1).half()
            used = torch.zeros(pages, page, dtype=torch.bool)
            for b, n in enumerate(lens):
                for t in range(0, int(n), page):
                    used[self.table[b, t // page], :min(page, int(n) - t)] = True
            pair[~used.cuda()] = math.nan
            rows = torch.cat([codes, pair.flatten(-2).view(torch.uint8)], -1)
            if layout == "hnd":
                x = torch.empty(pages, Hkv, page, row, dtype=torch.uint8, device="cuda").transpose(1, 2)
            elif layout == "nhd":
                x = torch.empty(pages, page, Hkv, row, dtype=torch.uint8, device="cuda")
            else:  # more heads than the call has, and rows apart
                x = torch.empty(pages, page, Hkv + 1, row + 16, dtype=torch.uint8, device="cuda")[:, :, :Hkv, :row]
            x.copy_(rows)
            return x

        self.k, self.v = cache(), cache()
        self.q = (torch.randn((B, N, Hq, D), generator=gen, device="cuda") * 1.5).to(DTYPES[dtype])

    def dev(self, x):
        return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()

    def slot(self, b, t):
        return int(self.table[b, t // self.page]), t % self.page

    def put(self, cache, b, t, h, group, scale, low):
        """The scale and minimum of a group of a row."""
        p, i = self.slot(b, t)
        D = (cache.shape[-1] - 16) * 2
        pair = torch.tensor([scale, low], device="cuda").half().view(torch.uint8)
        cache[p, i, h, D // 2 + 4 * group:D // 2 + 4 * group + 4] = pair

    def call(self, **kw):
        res = sv.paged_attention(self.q, self.k, self.v, self.dev(self.table), self.dev(self.ctx),
                                 num_new=self.dev(self.n_new), return_lse=True, return_flags=True, **kw)
        torch.cuda.synchronize()
        return res

    def gather(self, cache, row, T):
        out = torch.full((T, cache.shape[2], (cache.shape[3] - 16) * 2), math.nan, dtype=torch.float64)
        for t in range(0, T, self.page):
            p = int(row[t // self.page])
            if 0 <= p < cache.shape[0]:
                n = min(self.page, T - t)
                out[t:t + n] = stands_for(cache[p, :n])
        return out

    def check(self, res, sees=None, position=None, window=0, sinks=0, scale=None, only=None):
        q, k_cache, v_cache = self.q.cpu(), self.k.cpu(), self.v.cpu()
        out, lse = res.out.cpu().double(), res.lse.cpu().double()
        B, N, Hq, D = q.shape
        wide = N * (Hq // k_cache.shape[2]) > 8  # rows on tensor memory
        for b in range(B):
            n = N if self.n_new is None else int(self.n_new[b])
            if n == 0:
                continue
            c = int(self.ctx[b])
            T = c + n
            pos = None if position is None else (position[b] if position.ndim == 2 else position)
            m = None if sees is None else (sees[b] if sees.ndim == 3 else sees)
            vis = visible(c, n, N, m, pos, window, sinks)
            vis &= np.array([0 <= int(self.table[b, t // self.page]) < k_cache.shape[0] for t in range(T)], bool)
            k, v = (self.gather(x, self.table[b], T) for x in (k_cache, v_cache))
            rows = range(n) if only is None else only
            want, want_lse, mean, reach, vmax = attention_reference(
                q[b, list(rows)], k, v, vis[list(rows)], D ** -0.5 if scale is None else scale)
            tol, lse_tol = tolerance(want, want_lse, mean, reach, vmax, T, D, self.dtype, wide)
            where = f"sequence {b} ctx {c} new {n}"
            got, got_lse = out[b, list(rows)], lse[b, list(rows)]
            empty = want_lse == -math.inf
            assert (got_lse[empty] == -math.inf).all() and (got[empty] == 0).all(), where
            assert torch.isfinite(got).all(), where
            err = (got - want).abs()
            assert (err <= tol).all(), f"{where}: {(err / tol).max().item():.3g} of the tolerance"
            e = (got_lse - want_lse).abs()[~empty]
            assert (e <= lse_tol[~empty]).all(), f"{where}: lse off by {e.max().item():.3g}"


LENS = [0, 1, 15, 16, 17, 63, 64, 65, 127, 129, 300, 1000]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("Hq,Hkv,D,page,layout", [
    (4, 4, 64, 16, "hnd"), (8, 2, 128, 16, "hnd"), (7, 1, 128, 64, "nhd"), (32, 2, 64, 5, "hnd"),
    (40, 2, 128, 1, "nhd"), (9, 1, 128, 24, "hnd"), (5, 5, 64, 128, "apart"), (16, 1, 64, 7, "apart"),
    (3, 3, 128, 200, "hnd"), (24, 1, 128, 16, "hnd")])
def test_one_token(dtype, Hq, Hkv, D, page, layout):
    s = Setup(1, LENS, 1, Hq, Hkv, D, page, dtype, layout=layout)
    res = s.call()
    assert not res.flags.any()
    s.check(res)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("N,Hq,Hkv,D", [(2, 4, 2, 64), (5, 8, 8, 64), (8, 8, 2, 128), (33, 4, 1, 128),
                                        (130, 4, 4, 64), (70, 10, 2, 128), (16, 2, 2, 128)])
def test_chain(dtype, N, Hq, Hkv, D):
    s = Setup(2, [0, 1, 16, 77, 300], N, Hq, Hkv, D, 16, dtype)
    s.check(s.call())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("N,Hq,Hkv,D,page", [(1, 4, 2, 64, 16), (60, 8, 2, 128, 64), (64, 4, 2, 64, 16),
                                             (65, 2, 2, 128, 16), (200, 8, 1, 64, 32), (12, 16, 2, 128, 3),
                                             (6, 2, 1, 128, 16)])
def test_tree(dtype, N, Hq, Hkv, D, page):
    s = Setup(3, [0, 5, 64, 200], N, Hq, Hkv, D, page, dtype)
    parent = random_trees(s.rng, 4, N)
    mk = sv.tree_mask(s.dev(parent), N)
    res = s.call(tree_mask=mk.mask)
    words = mk.mask.cpu().numpy().view(np.uint8)
    sees = np.unpackbits(words, axis=-1, bitorder="little").reshape(4, N, -1)[:, :, :N].astype(bool)
    s.check(res, sees=sees)
    res = s.call(tree_mask=mk.mask[1])
    s.check(res, sees=sees[1])


@pytest.mark.parametrize("N", [3, 70])
def test_rows_that_see_nothing(N):
    s = Setup(4, [0, 0, 40, 3], N, 4, 2, 64, 16, "bf16")
    sees = s.rng.random((4, N, N)) < 0.3
    sees[0, ::3] = False
    sees[1] = False
    sees[2, 2] = False  # sees its context only
    res = s.call(tree_mask=s.dev(mask_words(sees)))
    s.check(res, sees=sees)
    assert (res.out[1] == 0).all() and (res.lse[1] == -math.inf).all()


@pytest.mark.parametrize("page", [16, 24, 1])
@pytest.mark.parametrize("N,window,sinks", [(1, 1, 0), (1, 7, 4), (1, 100, 0), (1, 100, 130), (1, 5000, 4),
                                            (6, 3, 2), (6, 64, 4), (3, 200, 17), (40, 17, 1), (150, 20, 5)])
def test_window(N, window, sinks, page):
    s = Setup(5, [0, 1, 20, 64, 130, 600], N, 4, 2, 64, page, "bf16")
    s.check(s.call(window=window, sinks=sinks), window=window, sinks=sinks)


@pytest.mark.parametrize("N,D", [(50, 64), (50, 128), (3, 128)])
def test_window_over_trees(N, D):
    s = Setup(6, [0, 9, 200], N, 6, 2, D, 16, "f16")
    parent = random_trees(s.rng, 3, N)
    mk = sv.tree_mask(s.dev(parent), N)
    sees = np.unpackbits(mk.mask.cpu().numpy().view(np.uint8), axis=-1,
                         bitorder="little").reshape(3, N, -1)[:, :, :N].astype(bool)
    for window, sinks in ((2, 0), (3, 12), (30, 1)):
        res = s.call(tree_mask=mk.mask, position=mk.position, window=window, sinks=sinks)
        s.check(res, sees=sees, position=mk.position.cpu().numpy(), window=window, sinks=sinks)


@pytest.mark.parametrize("N,Hq", [(3, 4), (7, 4), (30, 8)])
def test_ragged_new_tokens(N, Hq):
    n_new = [N, 0, 1, 3, 0, N - 1]
    s = Setup(7, [10, 50, 0, 300, 0, 17], N, Hq, 2, 64, 16, "bf16", n_new=n_new)
    out = torch.full(s.q.shape, 7.0, dtype=s.q.dtype, device="cuda")
    res = s.call(out=out)
    assert res.out is out
    s.check(res)
    for b, n in enumerate(n_new):
        assert (out[b, n:] == 7.0).all()


@pytest.mark.parametrize("N,Hq,Hkv,D,dtype", [(1, 4, 1, 128, "bf16"), (1, 8, 8, 64, "f16"), (3, 8, 2, 128, "f16"),
                                              (8, 4, 1, 128, "bf16"), (40, 8, 1, 128, "bf16"), (100, 4, 1, 64, "f16")])
def test_long_contexts_are_split_and_joined(N, Hq, Hkv, D, dtype):
    s = Setup(9, [20000, 1, 7000], N, Hq, Hkv, D, 16, dtype)
    res = s.call()
    # rows from both ends: the reference is slow
    s.check(res, only=sorted({0, N // 2, N - 1}))
    again = s.call()
    assert torch.equal(res.out, again.out) and torch.equal(res.lse, again.lse)


@pytest.mark.parametrize("dtype,N,D", [("bf16", 1, 128), ("f16", 4, 64), ("bf16", 40, 128), ("f16", 70, 64)])
def test_nan_and_inf_in_hidden_places(dtype, N, D):
    """Rows that a token does not see do not reach it, whatever they hold; the tokens
    that see them get them."""
    s = Setup(10, [60, 200], N, 4, 2, D, 16, dtype)
    sees = np.tril(np.ones((2, N, N), bool))
    hidden = N // 2  # seen by itself alone
    sees[:, hidden + 1:, hidden] = False
    kw = dict(tree_mask=s.dev(mask_words(sees)))
    clean = s.call(**kw)
    for b, bad in enumerate((math.nan, math.inf)):
        t = int(s.ctx[b]) + hidden
        s.put(s.k, b, t, 0, 3, 0.1, bad)
        s.put(s.v, b, t, 0, 1, 0.1, bad)
        s.put(s.v, b, t, 1, 0, bad, 0.0)
    res = s.call(**kw)
    others = [n for n in range(N) if n != hidden]
    assert torch.equal(res.out[:, others], clean.out[:, others]) and torch.equal(res.lse[:, others], clean.lse[:, others])
    each = D // 4
    # heads 2, 3 read key head 1, whose keys are fine
    for b in range(2):
        got = res.out[b, hidden, 2:]
        assert not torch.isfinite(got[:, :each]).any()
        near = clean.out[b, hidden, 2:, each:].float()
        assert ((got[:, each:].float() - near).abs() <= 2 * half_step(dtype) * near.abs() + 1e-7).all()
        assert torch.equal(res.lse[b, hidden, 2:], clean.lse[b, hidden, 2:])
        assert not torch.isfinite(res.out[b, hidden, :2, each:2 * each]).any()
    assert torch.isnan(res.lse[0, hidden, :2]).all() and torch.isnan(res.out[0, hidden, :2]).all()


@pytest.mark.parametrize("N", [1, 4, 40])
def test_values_that_every_row_sees(N):
    """Infinities in the context reach all rows."""
    s = Setup(11, [300, 40], N, 4, 1, 64, 16, "bf16")
    s.put(s.v, 0, 7, 0, 2, 0.0, math.inf)
    s.put(s.v, 1, 39, 0, 0, math.nan, 0.0)
    res = s.call()
    assert not torch.isfinite(res.out[0, :, :, 32:48]).any() and torch.isfinite(res.out[0, :, :, :32]).all()
    assert torch.isnan(res.out[1, :, :, :16]).all() and torch.isfinite(res.out[1, :, :, 16:]).all()
    assert torch.isfinite(res.lse).all()


@pytest.mark.parametrize("N", [1, 40])
def test_queries_of_any_size(N):
    s = Setup(12, [100, 33, 0], N, 4, 2, 128, 16, "bf16")
    for factor in (1e-20, 1e-4, 1.0, 30.0):
        s.q = (torch.randn_like(s.q.float()) * factor).to(torch.bfloat16)
        s.check(s.call())
    # values of one row 2^20 apart
    s.q = torch.randn_like(s.q.float()).mul_(torch.exp2(-20.0 * torch.rand_like(s.q.float()))).to(torch.bfloat16)
    s.check(s.call())
    # far beyond float16, with a scale that brings scores back
    s.q = (torch.randn_like(s.q.float()) * 1e9).to(torch.bfloat16)
    s.check(s.call(scale=1e-10), scale=1e-10)
    s.q[0, 0, 1, 5] = math.nan
    s.q[1, 0, 2, 7] = math.inf
    s.q[2] = 0
    res = s.call(scale=1e-10)
    for b, h in ((0, 1), (1, 2)):
        assert torch.isnan(res.out[b, 0, h]).all() and torch.isnan(res.lse[b, 0, h])
        res.out[b, 0, h], res.lse[b, 0, h] = 0.0, 0.0
    assert torch.isfinite(res.out).all() and torch.isfinite(res.lse).all()


@pytest.mark.parametrize("N", [1, 6, 40])
def test_a_long_tail_under_one_key_is_not_lost(N):
    """9000 equal keys 17.4 nats below one other add 1/4 of its weight: float16 weights
    that reached one at most would have rounded them to zero."""
    s = Setup(13, [9000], N, 4, 1, 64, 64, "bf16")
    for x in (s.k, s.v):
        x.zero_()
    s.q.fill_(1.0)
    for x, low in ((s.k, 0.0), (s.v, 1.0)):
        for g in range(4):
            x[..., 32 + 4 * g:36 + 4 * g] = torch.tensor([0.0, low], device="cuda").half().view(torch.uint8)
    for g in range(4):
        s.put(s.k, 0, 11, 0, g, 0.0, 17.4 * 8 / 64)
        s.put(s.v, 0, 11, 0, g, 0.0, 0.0)
    s.check(s.call())


@pytest.mark.parametrize("N", [1, 5, 40])
def test_bad_pages_and_lengths(N):
    s = Setup(14, [100, 100, 50], N, 4, 2, 64, 16, "bf16")
    s.table[0, 2] = -5
    s.table[1, 0] = 1 << 29
    ctx = s.ctx.copy()
    res = s.call()
    assert res.flags.tolist() == [sv.FLAG_BAD_PAGE, sv.FLAG_BAD_PAGE, 0]
    s.check(res)
    s.ctx[2] = 10 ** 6
    res = s.call()
    assert res.flags.tolist()[2] == sv.FLAG_BAD_LENGTH
    assert (res.out[2] == 0).all() and (res.lse[2] == -math.inf).all()
    s.ctx = ctx


@pytest.mark.parametrize("N,Hq,Hkv,D", [(1, 8, 2, 128), (1, 8, 2, 64), (4, 8, 2, 128), (5, 8, 2, 64), (40, 8, 2, 128)])
def test_many_sequences(N, Hq, Hkv, D):
    ctx = np.random.default_rng(15).integers(0, 400, 300)
    s = Setup(15, ctx, N, Hq, Hkv, D, 16, "bf16", max_pages=2000 // 16)
    res = s.call()
    sub = sorted(np.random.default_rng(1).choice(300, 25, replace=False).tolist())
    out = type(res)(res.out[sub], res.lse[sub], None)
    s.q, s.table, s.ctx = s.q[sub], s.table[sub], s.ctx[sub]
    s.check(out)


@pytest.mark.parametrize("N,Hq,Hkv,D", [(1, 4, 2, 64), (1, 8, 1, 128), (6, 4, 2, 128), (9, 4, 2, 64), (40, 4, 2, 64)])
def test_scales_of_every_size(N, Hq, Hkv, D):
    """Groups that span next to nothing, 60 and more, and thousands, in one cache; the
    queries are as small as the largest keys are large."""
    s = Setup(20, [50, 0, 700], N, Hq, Hkv, D, 16, "bf16")
    gen = torch.Generator("cuda")
    gen.manual_seed(20)
    for x in (s.k, s.v):
        pair = x[..., D // 2:].contiguous().view(torch.float16).reshape(*x.shape[:3], 4, 2)
        up = torch.randint(0, 4, pair.shape[:-1], generator=gen, device="cuda")
        by = torch.tensor([2.0 ** -9, 1.0, 16.0, 1024.0], device="cuda")[up]
        pair = (pair.float() * by[..., None]).half()
        x[..., D // 2:] = pair.flatten(-2).view(torch.uint8)
    s.q = (s.q.float() / 512).to(s.q.dtype)
    s.check(s.call())


@pytest.mark.parametrize("N,Hq,Hkv,D", [(1, 130, 1, 64), (3, 256, 1, 128), (1, 128, 1, 128), (5, 96, 2, 64)])
def test_groups_of_many_heads(N, Hq, Hkv, D):
    s = Setup(21, [33, 0, 900], N, Hq, Hkv, D, 16, "bf16")
    s.check(s.call(), only=sorted({0, N - 1}))


@pytest.mark.parametrize("N,G", [(2, 8), (3, 3), (32, 1), (11, 3), (8, 4), (9, 1), (16, 2), (12, 4), (25, 5),
                                 (64, 2), (100, 1), (2, 64), (16, 4)])
def test_units_of_one_row_tile(N, G):
    """Between nine and 128 rows: many short sequences, so that a thread block has units of
    one tile and of several behind one another, and long ones cut between blocks."""
    ctx = np.random.default_rng(22).integers(0, 90, 700)
    ctx[::97] = 3000 + np.arange(len(ctx[::97])) * 31
    s = Setup(22, ctx, N, 2 * G, 2, 64, 16, "f16", max_pages=3400 // 16)
    res = s.call()
    again = s.call()
    assert torch.equal(res.out, again.out) and torch.equal(res.lse, again.lse)
    sub = [0, 1, 2, 96, 97, 98, 194, 291, 500, 679, 680, 698, 699]
    out = type(res)(res.out[sub], res.lse[sub], None)
    s.q, s.table, s.ctx = s.q[sub], s.table[sub], s.ctx[sub]
    s.check(out, only=sorted({0, N // 2, N - 1}))


def test_two_calls_at_once_on_two_streams():
    a, b = (Setup(23 + i, [4000, 20, 900], n, 8, 2, 128, 16, "bf16") for i, n in enumerate((1, 8)))
    want = a.call(), b.call()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    args = [(x.q, x.k, x.v, x.dev(x.table), x.dev(x.ctx)) for x in (a, b)]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for st, x in zip(streams, args):
            with torch.cuda.stream(st):
                got.append(sv.paged_attention(*x, return_lse=True))
    torch.cuda.synchronize()
    for i, x in enumerate(got):
        assert torch.equal(x.out, want[i % 2].out) and torch.equal(x.lse, want[i % 2].lse)


@pytest.mark.parametrize("N", [16, 40])
def test_a_wait_that_gives_up(N):
    s = Setup(16, [300, 20, 5000], N, 8, 2, 128, 16, "bf16")
    before = s.call()
    try:
        sv.set_wait_limit(0)
        gave_up = s.call()
    finally:
        sv.set_wait_limit(None)
    assert gave_up.flags.tolist() == [sv.FLAG_TIMEOUT] * 3
    assert torch.isnan(gave_up.out).all() and torch.isnan(gave_up.lse).all()
    after = s.call()
    assert not after.flags.any() and torch.equal(after.out, before.out) and torch.equal(after.lse, before.lse)


@pytest.mark.parametrize("N", [1, 4, 40])
def test_a_captured_call_follows_lengths(N):
    s = Setup(17, [3000, 100], N, 8, 2, 64, 16, "f16")
    ctx, table = s.dev(s.ctx), s.dev(s.table)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sv.paged_attention(s.q, s.k, s.v, table, ctx)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            res = sv.paged_attention(s.q, s.k, s.v, table, ctx, return_lse=True)
    torch.cuda.synchronize()
    for lens in ([3000, 100], [5, 90], [0, 0], [1500, 33]):
        ctx.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = sv.paged_attention(s.q, s.k, s.v, table, ctx, return_lse=True)
        assert torch.equal(res.out, want.out) and torch.equal(res.lse, want.lse)
        s.ctx = np.asarray(lens, np.int32)
        if lens[0] < 100:
            s.check(res)


def test_refusals():
    s = Setup(18, [20], 2, 4, 2, 64, 16, "bf16")
    table, ctx = s.dev(s.table), s.dev(s.ctx)
    with pytest.raises(ValueError):
        sv.paged_attention(s.q.float(), s.k, s.v, table, ctx)
    with pytest.raises(ValueError):
        sv.paged_attention(s.q, s.k, s.v.view(torch.int8), table, ctx)
    with pytest.raises(ValueError):
        sv.paged_attention(s.q[..., :32], s.k, s.v, table, ctx)
    with pytest.raises(ValueError):
        sv.paged_attention(s.q, s.k[..., :40], s.v[..., :40], table, ctx)
    with pytest.raises(ValueError):
        sv.paged_attention(s.q.requires_grad_(), s.k, s.v, table, ctx)
    with pytest.raises(ValueError):
        sv.cache_4bit(4, 16, 2, 96)
    wide = torch.zeros(4, 16, 2, 50, dtype=torch.uint8, device="cuda")[..., 1:49]
    with pytest.raises(sv.SpecVerifyError):
        sv.paged_attention(s.q.detach(), wide, wide, table, ctx)


def test_decode_steps_together():
    """A prompt, then steps of a tree over a 4-bit cache: rotation, append, attention,
    compaction and pages, against the same steps on the values that the rows stand for."""
    B, N, Hq, Hkv, D, page = 3, 7, 8, 2, 128, 16
    gen = torch.Generator("cuda")
    gen.manual_seed(19)
    normal = lambda *shape: torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    k, v = sv.cache_4bit(40, page, Hkv, D)
    pool = sv.page_pool(B, 12, 40)
    f, amplitude = sv.rotary_frequency(D, scaling="turns", factor=4.0)
    ctx = torch.zeros(B, dtype=torch.int32, device="cuda")
    num = torch.tensor([50, 3, 17], device="cuda")
    assert not sv.cache_resize(pool, num, page).any()
    prompt = normal(B, 50, Hkv, D), normal(B, 50, Hkv, D)
    sv.cache_append_rotary(*prompt, k, v, pool.page_table, ctx, f, num_new=num)
    ctx = num.to(torch.int32)
    parent = torch.tensor([[-1, 0, 0, 1, 1, 2, 5]] * B, dtype=torch.int32, device="cuda")
    mk = sv.tree_mask(parent, 4)
    path = torch.tensor([[0, 1, 4, -1], [0, 2, 5, 6], [0, -1, -1, -1]], dtype=torch.int32, device="cuda")
    taken = torch.tensor([2, 3, 0], dtype=torch.int32, device="cuda")
    for _ in range(3):
        assert not sv.cache_resize(pool, ctx + N, page).any()
        new = normal(B, N, Hkv, D), normal(B, N, Hkv, D)
        q = normal(B, N, Hq, D)
        turned = sv.cache_append_rotary(*new, k, v, pool.page_table, ctx, f, q=q, position=mk.position).q
        assert torch.equal(turned, sv.rotary(q, ctx[:, None] + mk.position, f))
        at = sv.paged_attention(turned, k, v, pool.page_table, ctx, tree_mask=mk.mask)
        rows = sv.cache_read(k, v, pool.page_table, torch.zeros_like(ctx), 150, num=ctx + N, dtype=torch.float32)
        for b in range(B):
            T = int(ctx[b]) + N
            sees = torch.ones(N, T, dtype=torch.bool)
            for n in range(N):
                up, seen = n, set()
                while up >= 0:
                    seen.add(up)
                    up = int(parent[b, up])
                sees[n, T - N:] = torch.tensor([m in seen for m in range(N)])
            kk, vv = (x[b, :T].double().cpu() for x in (rows.k, rows.v))
            want, _, mean, reach, vmax = attention_reference(turned[b].cpu(), kk, vv, sees.numpy(), D ** -0.5)
            tol, _ = tolerance(want, reach, mean, reach, vmax, T, D, "bf16", False)
            assert ((at.out[b].cpu().double() - want).abs() <= tol).all()
        before = sv.cache_read(k, v, pool.page_table, ctx, N)
        r = sv.cache_compact(k, v, pool.page_table, ctx, path, taken)
        now = sv.cache_read(k, v, pool.page_table, ctx, 4, num=taken + 1)
        for b in range(B):
            n = int(taken[b]) + 1
            assert torch.equal(now.k[b, :n], before.k[b, path[b, :n].long()])
        ctx = r.context_len
        assert not sv.cache_resize(pool, ctx, page).any()
