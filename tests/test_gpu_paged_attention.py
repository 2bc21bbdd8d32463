"""Attention over a paged key-value cache against a plain 64-bit computation:
types, head layouts, page sizes, lengths from none to many splits, trees,
windows with sinks, ragged batches, and what must not be read."""

import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_temp_gb300 as sv

from cache_helpers import (DTYPES, check_attention, make_pages, mask_words, random_trees, visible)

pytestmark = pytest.mark.gpu


class Setup:
    """Inputs of a call; every slot behind a sequence's tokens holds NaN."""

    def __init__(self, seed, ctx, N, Hq, Hkv, D, page, dtype, n_new=None, layout="nhd",
                 max_pages=None):
        rng = np.random.default_rng(seed)
        gen = torch.Generator("cuda")
        gen.manual_seed(seed)
        self.rng, self.page, self.dtype, self.N = rng, page, dtype, N
        self.ctx = np.asarray(ctx, np.int32)
        B = len(self.ctx)
        self.n_new = None if n_new is None else np.asarray(n_new, np.int32)
        lens = self.ctx + (N if n_new is None else self.n_new)
        self.table, pages = make_pages(rng, lens, page, max_pages)
        dt = DTYPES[dtype]
        normal = lambda *s: torch.randn(s, generator=gen, device="cuda", dtype=torch.float32).to(dt)
        self.q = normal(B, N, Hq, D) * 1.5
        if layout == "nhd":
            self.k, self.v = normal(pages, page, Hkv, D), normal(pages, page, Hkv, D)
        elif layout == "hnd":
            self.k = normal(pages, Hkv, page, D).transpose(1, 2)
            self.v = normal(pages, Hkv, page, D).transpose(1, 2)
        else:  # keys and values of a token side by side
            kv = normal(pages, page, 2, Hkv, D)
            self.k, self.v = kv[:, :, 0], kv[:, :, 1]
        used = torch.zeros(pages, page, dtype=torch.bool)
        for b, n in enumerate(lens):
            for t in range(0, int(n), page):
                used[self.table[b, t // page], :min(page, int(n) - t)] = True
        for x in (self.k, self.v):
            x[~used.cuda()] = math.nan

    def dev(self, x):
        return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()

    def slot(self, b, t):
        return int(self.table[b, t // self.page]), t % self.page

    def call(self, **kw):
        res = sv.paged_attention(self.q, self.k, self.v, self.dev(self.table), self.dev(self.ctx),
                                 num_new=self.dev(self.n_new), return_lse=True, return_flags=True,
                                 **kw)
        torch.cuda.synchronize()
        return res

    def check(self, res, **kw):
        check_attention(res, self.q, self.k, self.v, self.table, self.ctx, self.page, self.dtype,
                        n_new=self.n_new, **kw)


LENS = [0, 1, 15, 16, 17, 63, 64, 65, 127, 129, 300, 1000]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,D,page", [
    (4, 4, 64, 16), (8, 2, 128, 16), (7, 1, 128, 64), (32, 2, 64, 5), (40, 2, 128, 1),
    (4, 2, 256, 16), (3, 1, 8, 16), (6, 2, 40, 32), (5, 5, 72, 128), (4, 1, 192, 7)])
def test_one_token(dtype, Hq, Hkv, D, page):
    s = Setup(1, LENS, 1, Hq, Hkv, D, page, dtype)
    res = s.call()
    assert not res.flags.any()
    s.check(res)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N,Hq,Hkv,D", [(2, 4, 2, 64), (5, 8, 8, 64), (8, 8, 2, 128), (33, 4, 1, 128),
                                        (130, 4, 4, 64), (70, 10, 2, 128), (9, 4, 2, 256),
                                        (40, 6, 1, 72)])
def test_chain(dtype, N, Hq, Hkv, D):
    s = Setup(2, [0, 1, 16, 77, 300], N, Hq, Hkv, D, 16, dtype)
    s.check(s.call())


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N,Hq,Hkv,D,page", [(1, 4, 2, 64, 16), (60, 8, 2, 128, 64), (64, 4, 2, 64, 16),
                                             (65, 2, 2, 128, 16), (200, 8, 1, 64, 32), (12, 16, 2, 128, 3)])
def test_tree(dtype, N, Hq, Hkv, D, page):
    s = Setup(3, [0, 5, 64, 200], N, Hq, Hkv, D, page, dtype)
    parent = random_trees(s.rng, 4, N)
    mk = sv.tree_mask(s.dev(parent), N)
    res = s.call(tree_mask=mk.mask)
    words = mk.mask.cpu().numpy().view(np.uint8)
    sees = np.unpackbits(words, axis=-1, bitorder="little").reshape(4, N, -1)[:, :, :N].astype(bool)
    s.check(res, sees=sees)
    # one tree for all sequences
    res = s.call(tree_mask=mk.mask[1])
    s.check(res, sees=sees[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_see_nothing(dtype):
    N = 70
    s = Setup(4, [0, 0, 40, 3], N, 4, 2, 64, 16, dtype)
    sees = s.rng.random((4, N, N)) < 0.3
    sees[0, ::3] = False
    sees[1] = False
    sees[2, 5] = False  # sees its context only
    res = s.call(tree_mask=s.dev(mask_words(sees)))
    s.check(res, sees=sees)
    assert (res.out[1] == 0).all() and (res.lse[1] == -math.inf).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N,window,sinks", [(1, 1, 0), (1, 7, 4), (1, 100, 0), (1, 100, 130), (1, 5000, 4),
                                            (6, 3, 2), (6, 64, 4), (40, 17, 1), (150, 20, 5)])
def test_window(dtype, N, window, sinks):
    s = Setup(5, [0, 1, 20, 64, 130, 600], N, 8, 2, 64, 16, dtype)
    s.check(s.call(window=window, sinks=sinks), window=window, sinks=sinks)


@pytest.mark.parametrize("D", [64, 128])
def test_window_over_trees(D):
    N = 50
    s = Setup(6, [0, 9, 200], N, 6, 2, D, 16, "bf16")
    parent = random_trees(s.rng, 3, N)
    mk = sv.tree_mask(s.dev(parent), N)
    sees = np.unpackbits(mk.mask.cpu().numpy().view(np.uint8), axis=-1,
                         bitorder="little").reshape(3, N, -1)[:, :, :N].astype(bool)
    for position in (mk.position, mk.position - 5, mk.position + 48):  # clamped into [0, N)
        pos = position.cpu().numpy()
        for window, sinks in ((2, 0), (3, 12), (30, 1)):
            res = s.call(tree_mask=mk.mask, position=position, window=window, sinks=sinks)
            s.check(res, sees=sees, position=pos, window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,Hq", [(7, 4), (30, 8)])
def test_ragged_new_tokens(dtype, N, Hq):
    n_new = [N, 0, 1, 3, 0, N - 1]
    s = Setup(7, [10, 50, 0, 300, 0, 17], N, Hq, 2, 64, 16, dtype, n_new=n_new)
    out = torch.full(s.q.shape, 7.0, dtype=s.q.dtype, device="cuda")
    res = s.call(out=out)
    assert res.out is out
    s.check(res)
    for b, n in enumerate(n_new):
        assert (out[b, n:] == 7.0).all()


@pytest.mark.parametrize("layout", ["hnd", "pairs"])
@pytest.mark.parametrize("N,D", [(1, 128), (9, 64), (40, 128)])
def test_layouts_and_strided_queries(layout, N, D):
    s = Setup(8, [33, 200, 0], N, 8, 2, D, 16, "bf16", layout=layout)
    fused = torch.randn(3, N, 12, D, device="cuda").to(torch.bfloat16)  # queries, keys, values
    fused[:, :, :8] = s.q
    s.q = fused[:, :, :8]
    assert not s.q.is_contiguous()
    s.check(s.call())
    # a table that is a view of a wider one
    wide = np.full((3, s.table.shape[1] + 5), -7, np.int32)
    wide[:, :s.table.shape[1]] = s.table
    table = s.dev(wide)[:, :s.table.shape[1]]
    again = sv.paged_attention(s.q, s.k, s.v, table, s.dev(s.ctx))
    assert torch.equal(again.out, s.call().out)


@pytest.mark.parametrize("N,Hq,Hkv,D,dtype", [(1, 4, 1, 128, "bf16"), (1, 8, 8, 64, "f16"),
                                              (3, 8, 2, 256, "bf16"), (5, 2, 1, 64, "f32"),
                                              (40, 8, 1, 128, "bf16"), (100, 4, 1, 64, "f16")])
def test_long_contexts_are_split_and_joined(N, Hq, Hkv, D, dtype):
    s = Setup(9, [30000, 1, 7000], N, Hq, Hkv, D, 16, dtype)
    res = s.call()
    s.check(res)
    again = s.call()
    assert torch.equal(res.out, again.out) and torch.equal(res.lse, again.lse)


@pytest.mark.parametrize("dtype,N,D", [("bf16", 1, 128), ("f16", 9, 64), ("f32", 4, 64), ("bf16", 40, 128),
                                       ("f16", 70, 64)])
def test_nan_and_inf_in_hidden_places(dtype, N, D):
    """Values that a token does not see do not reach it, whatever they hold; the
    tokens that see them get them."""
    s = Setup(10, [60, 200], N, 4, 2, D, 16, dtype)
    sees = np.tril(np.ones((2, N, N), bool))
    hidden = N // 2  # seen by itself alone
    sees[:, hidden + 1:, hidden] = False
    kw = dict(tree_mask=s.dev(mask_words(sees)), window=0)
    clean = s.call(**kw)
    for b, (kx, vx) in enumerate(((math.nan, math.inf), (math.inf, math.nan))):
        p, i = s.slot(b, int(s.ctx[b]) + hidden)
        s.k[p, i, 0, 3] = kx
        s.v[p, i, :, 5] = vx
    res = s.call(**kw)
    others = [n for n in range(N) if n != hidden]
    assert torch.equal(res.out[:, others], clean.out[:, others])
    assert torch.equal(res.lse[:, others], clean.lse[:, others])
    assert not torch.isfinite(res.out[:, hidden, :, 5]).any()
    # a value alone (heads 2 and 3 have clean keys) reaches its dimension only
    rest = [d for d in range(D) if d != 5]
    assert torch.equal(res.out[:, hidden, 2:][..., rest], clean.out[:, hidden, 2:][..., rest])
    assert (res.out[0, hidden, 2:, 5] == math.inf).all()
    assert torch.isnan(res.out[1, hidden, 2:, 5]).all()


@pytest.mark.parametrize("dtype,N", [("bf16", 1), ("f32", 2), ("bf16", 40)])
def test_infinite_scores(dtype, N):
    """Keys that score -infinity weigh nothing; rows of such keys alone are empty."""
    s = Setup(11, [40, 100], N, 4, 2, 64, 16, dtype)
    s.q[:] = s.q.abs() + 0.5
    for t in range(40 + N):
        p, i = s.slot(0, t)
        s.k[p, i, :, 0] = -math.inf
    for t in range(0, 100, 3):
        p, i = s.slot(1, t)
        s.k[p, i, :, 1] = -math.inf
    res = s.call()
    assert (res.out[0] == 0).all() and (res.lse[0] == -math.inf).all()
    kept = visible(100, N, N)
    kept[:, 0:100:3] = False
    clean = s.k.clone()
    clean[clean == -math.inf] = 0.0
    from cache_helpers import attention_reference, attention_tolerance, gather
    k, v = (gather(x.cpu(), s.table[1], 100 + N, 16) for x in (clean, s.v))
    want, lse, mean, reach, vmax = attention_reference(s.q[1].cpu(), k, v, kept, 64 ** -0.5)
    tol, lse_tol = attention_tolerance(want, lse, mean, reach, vmax, 100 + N, 64, dtype)
    assert ((res.out[1].cpu().double() - want).abs() <= tol).all()
    assert ((res.lse[1].cpu().double() - lse).abs() <= lse_tol).all()


@pytest.mark.parametrize("dtype,N", [("bf16", 1), ("f32", 3), ("f16", 40)])
def test_large_scores(dtype, N):
    """Scores of some hundreds: one key takes nearly all, the sums stay finite."""
    s = Setup(12, [100, 500], N, 4, 2, 128, 16, dtype)
    s.check(s.call(scale=2.0), scale=2.0)


@pytest.mark.parametrize("dtype,N", [("bf16", 1), ("f32", 2), ("bf16", 33)])
def test_bad_pages_and_lengths_are_flagged(dtype, N):
    s = Setup(13, [100, 90, 80, 70], N, 4, 2, 64, 16, dtype)
    s.table[1, 2] = -1
    s.table[2, 0] = s.k.shape[0]
    res = s.call()
    assert res.flags.tolist() == [0, sv.FLAG_BAD_PAGE, sv.FLAG_BAD_PAGE, 0]
    s.check(res)
    s.ctx[3] = s.table.shape[1] * 16 - N + 1  # one token too many
    s.ctx[1] = -1
    res = s.call()
    assert res.flags.tolist() == [0, sv.FLAG_BAD_LENGTH, sv.FLAG_BAD_PAGE, sv.FLAG_BAD_LENGTH]
    for b in (1, 3):
        assert (res.out[b] == 0).all() and (res.lse[b] == -math.inf).all()
    res = sv.paged_attention(s.q, s.k, s.v, s.dev(s.table), s.dev(np.array([100, 0, 0, 0], np.int32)),
                             num_new=s.dev(np.array([N, N + 3, -2, N], np.int32)), return_flags=True)
    # sequence 1's entry 2, the pages of tokens 32 to 47, is still the bad one
    bad_page = sv.FLAG_BAD_PAGE if N > 32 else 0
    assert res.flags.tolist()[1:3] == [sv.FLAG_BAD_LENGTH | bad_page, sv.FLAG_BAD_LENGTH]


def test_a_captured_call_follows_the_lengths():
    s = Setup(14, [500, 900], 4, 8, 2, 128, 16, "bf16", max_pages=80)
    table, ctx = s.dev(s.table), s.dev(s.ctx)
    sv.paged_attention(s.q, s.k, s.v, table, ctx, return_lse=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = sv.paged_attention(s.q, s.k, s.v, table, ctx, return_lse=True)
    for lens in ([500, 900], [3, 17], [0, 600]):
        ctx.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        # an eager call of other sizes between two replays
        sv.paged_attention(s.q[:1], s.k, s.v, table[:1], ctx[:1])
        torch.cuda.synchronize()
        s.ctx = np.asarray(lens, np.int32)
        s.check(res)


def test_calls_on_two_streams_at_once():
    a = Setup(15, [3000] * 4, 1, 8, 2, 128, 16, "bf16")
    b = Setup(16, [2000] * 4, 20, 8, 2, 128, 16, "bf16")
    dev = [(x, x.dev(x.table), x.dev(x.ctx)) for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(5):
        for (x, table, ctx), st in zip(dev, streams):
            with torch.cuda.stream(st):
                got.append((x, sv.paged_attention(x.q, x.k, x.v, table, ctx, return_lse=True)))
    torch.cuda.synchronize()
    for x, r in got[:2]:
        x.check(r)
    for x, r in got[2:]:
        first = got[0 if x is a else 1][1]
        assert torch.equal(r.out, first.out) and torch.equal(r.lse, first.lse)


def test_offsets_beyond_32_bits():
    """Pages far behind 2^31 elements of a cache."""
    page, Hkv, D = 64, 8, 128
    per_page = page * Hkv * D
    pages = (1 << 32) // per_page + 40
    k = torch.zeros(pages, page, Hkv, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    far = np.array([[pages - 1, 3, pages - 17], [pages // 2 + 1, pages - 2, 0]], np.int32)
    for p in far.reshape(-1):
        k[int(p)].normal_()
        v[int(p)].normal_()
    table, ctx = torch.from_numpy(far).cuda(), np.array([150, 100], np.int32)
    for N in (1, 20):
        q = torch.randn(2, N, 16, D, device="cuda").to(torch.bfloat16)
        res = sv.paged_attention(q, k, v, table, torch.from_numpy(ctx).cuda(), return_lse=True)
        torch.cuda.synchronize()
        used = np.unique(far)
        small = np.searchsorted(used, far).astype(np.int32)
        at = torch.from_numpy(used.astype(np.int64)).cuda()
        check_attention(res, q, k[at], v[at], small, ctx, page, "bf16")


def test_long_chains_from_an_empty_cache():
    """A prompt: every token is new."""
    s = Setup(17, [0, 37], 300, 4, 2, 128, 16, "bf16")
    s.check(s.call())


# bf16 and f16 at head_dim 64 and 128 with pages of 8 n tokens take the tensor
# memory kernels, other sizes the matrix kernel, float32 the FMA kernel; up to 32
# rows (new tokens times query heads per head) are split over lane quarters, up to
# 128 are a row tile, more are pairs of row tiles.
KERNELS = [("bf16", 1, 8, 2, 128, 16), ("f16", 4, 16, 2, 64, 8), ("bf16", 10, 16, 2, 128, 32),
           ("f16", 12, 10, 2, 64, 16), ("bf16", 40, 14, 2, 128, 64), ("f16", 70, 8, 2, 64, 16),
           ("bf16", 3, 6, 2, 72, 16), ("f16", 2, 4, 2, 128, 5), ("bf16", 2, 4, 2, 200, 16),
           ("f32", 3, 6, 2, 20, 16), ("f32", 1, 4, 2, 128, 3), ("f32", 2, 2, 1, 256, 16)]


@pytest.mark.parametrize("dtype,N,Hq,Hkv,D,page", KERNELS)
def test_many_short_sequences(dtype, N, Hq, Hkv, D, page):
    """More units than CTAs: a CTA goes from one to the next."""
    rng = np.random.default_rng(20)
    B = 40 if N >= 40 else 420
    s = Setup(20, rng.integers(0, 50, B), N, Hq, Hkv, D, page, dtype,
              n_new=rng.integers(0, N + 1, B))
    s.check(s.call())


@pytest.mark.parametrize("dtype,N,Hq,Hkv,D,page", KERNELS)
def test_ragged_batches_that_are_cut_anywhere(dtype, N, Hq, Hkv, D, page):
    rng = np.random.default_rng(21)
    s = Setup(21, [3, 2500, 0, 127, 128, 129, 900, 1, 1300], N, Hq, Hkv, D, page, dtype)
    sees = rng.random((9, N, N)) < 0.5
    res = s.call(tree_mask=s.dev(mask_words(sees)))
    s.check(res, sees=sees)
    again = s.call(tree_mask=s.dev(mask_words(sees)))
    assert torch.equal(res.out, again.out) and torch.equal(res.lse, again.lse)


@pytest.mark.parametrize("dtype,N,Hq,Hkv,D,page", KERNELS)
def test_windows_in_every_kernel(dtype, N, Hq, Hkv, D, page):
    s = Setup(22, [0, 5, 700, 333], N, Hq, Hkv, D, page, dtype)
    position = s.rng.integers(0, N, (4, N))
    for window, sinks, pos in ((100, 4, None), (30, 200, None), (2 ** 31 - 1, 3, None), (7, 1, position)):
        res = s.call(window=window, sinks=sinks, position=s.dev(pos))
        s.check(res, window=window, sinks=sinks, position=pos)


@pytest.mark.parametrize("dtype,N,Hq,Hkv,D,page", KERNELS)
def test_nothing_to_do(dtype, N, Hq, Hkv, D, page):
    s = Setup(23, [30, 0, 7], N, Hq, Hkv, D, page, dtype, n_new=[0, 0, 0])
    out = torch.full(s.q.shape, 3.0, dtype=s.q.dtype, device="cuda")
    s.call(out=out)
    assert (out == 3.0).all()
    none = sv.paged_attention(s.q[:0], s.k, s.v, s.dev(s.table)[:0], s.dev(s.ctx)[:0], return_flags=True)
    assert none.out.shape[0] == 0 and none.flags.numel() == 0


@pytest.mark.parametrize("page", [8, 32, 128, 256, 384, 24])
@pytest.mark.parametrize("N", [1, 20, 70])
def test_page_sizes(page, N):
    s = Setup(24, [0, 100, 383, 384, 900], N, 8, 2, 128, page, "bf16", layout="hnd" if N == 20 else "nhd")
    s.check(s.call())


@pytest.mark.parametrize("Hq,N,D", [(130, 1, 64), (300, 2, 128), (97, 3, 64), (128, 1, 128)])
def test_many_query_heads_to_one(Hq, N, D):
    s = Setup(25, [40, 300], N, Hq, 1, D, 16, "bf16")
    s.check(s.call())


def test_queries_that_have_to_be_copied():
    s = Setup(26, [50, 120], 3, 8, 2, 64, 16, "bf16")
    want = s.call()
    flat = torch.zeros(s.q.numel() + 3, dtype=s.q.dtype, device="cuda")
    odd = flat[3:].view(s.q.shape)
    odd.copy_(s.q)
    swapped = s.q.transpose(2, 3).contiguous().transpose(2, 3)
    for q in (odd, swapped):
        got = sv.paged_attention(q, s.k, s.v, s.dev(s.table), s.dev(s.ctx))
        assert torch.equal(got.out, want.out)
    one = s.q[:1].expand(2, -1, -1, -1)
    got = sv.paged_attention(one, s.k, s.v, s.dev(s.table), s.dev(s.ctx))
    assert torch.equal(got.out, sv.paged_attention(one.contiguous(), s.k, s.v, s.dev(s.table),
                                                   s.dev(s.ctx)).out)


def test_refused_tensors():
    s = Setup(27, [50, 120], 3, 8, 2, 64, 16, "bf16")
    table, ctx = s.dev(s.table), s.dev(s.ctx)
    good = dict(q=s.q, k_cache=s.k, v_cache=s.v, page_table=table, context_len=ctx)
    words = torch.zeros(2, 3, 1, dtype=torch.int64, device="cuda")
    grad = s.q.clone().requires_grad_()
    for bad in (dict(q=s.q.float()), dict(q=s.q[:, :, :, :32]), dict(q=s.q[0]), dict(q=s.q.cpu()),
                dict(v_cache=s.v[:, :, :1]), dict(v_cache=s.v.half()), dict(k_cache=s.k.cpu()),
                dict(k_cache=s.k[None], v_cache=s.v[None]), dict(page_table=table[:1]),
                dict(page_table=table.float()), dict(context_len=ctx[:1]), dict(context_len=ctx.float()),
                dict(num_new=ctx[:1]), dict(tree_mask=words[:, :2]), dict(tree_mask=words.int()),
                dict(position=ctx), dict(out=s.q[:1]), dict(q=grad),
                dict(k_cache=s.k.transpose(1, 3).contiguous().transpose(1, 3),
                     v_cache=s.v.transpose(1, 3).contiguous().transpose(1, 3))):
        with pytest.raises(ValueError):
            sv.paged_attention(**(good | bad))
    for bad in (dict(out=s.q), dict(window=3, tree_mask=words), dict(scale=0.0), dict(sinks=-1),
                dict(q=s.q[:, :, :7])):
        with pytest.raises(sv.SpecVerifyError):
            sv.paged_attention(**(good | bad))
    with torch.no_grad():
        assert torch.equal(sv.paged_attention(**(good | dict(q=grad))).out, s.call().out)


@pytest.mark.parametrize("Hq,Hkv,D", [(16, 2, 128), (14, 2, 64), (3, 1, 128)])
def test_trees_of_several_row_tiles(Hq, Hkv, D):
    """Row tiles with lines of work of their own; sequences with fewer of them."""
    N, n_new = 100, [100, 3, 0, 64, 33, 100]
    s = Setup(28, [700, 100, 5, 3000, 0, 90], N, Hq, Hkv, D, 16, "bf16", n_new=n_new)
    sees = s.rng.random((6, N, N)) < 0.4
    res = s.call(tree_mask=s.dev(mask_words(sees)))
    s.check(res, sees=sees)
    again = s.call(tree_mask=s.dev(mask_words(sees)))
    for b, n in enumerate(n_new):
        assert torch.equal(res.out[b, :n], again.out[b, :n])


def test_integers_beyond_32_bits_and_outputs_with_gradients():
    gen = torch.Generator("cuda")
    gen.manual_seed(5)
    k, v = (torch.randn(8, 16, 2, 64, generator=gen, device="cuda") for _ in "kv")
    q = torch.randn(1, 2, 4, 64, generator=gen, device="cuda")
    args = (q, k, v, torch.arange(8, dtype=torch.int32, device="cuda")[None],
            torch.tensor([100], dtype=torch.int32, device="cuda"))
    plain = sv.paged_attention(*args).out
    assert torch.equal(sv.paged_attention(*args, window=2 ** 32 + 5).out, plain)
    assert torch.equal(sv.paged_attention(*args, window=8, sinks=2 ** 32 + 1).out, plain)
    assert torch.equal(sv.paged_attention(*args, window=-2 ** 32 + 5).out, plain)
    with pytest.raises(Exception):
        sv.paged_attention(*args, window=8, sinks=-2 ** 32)
    pool = sv.page_pool(1, 8, 8)
    with pytest.raises(Exception):
        sv.cache_resize(pool, args[4], 2 ** 32 + 16)
    with pytest.raises(ValueError):
        sv.paged_attention(*args, out=torch.empty_like(q, requires_grad=True))


# Tokens of the widest page table whose units are not cut, for each of KERNELS.
WHOLE = [512, 512, 768, 768, 2048, 2048, 256, 256, 128, 128, 64, 32]


@pytest.mark.parametrize("kernel,tokens", list(zip(KERNELS, WHOLE)))
def test_units_whole_and_cut(kernel, tokens):
    """The same call through a page table as wide as whole units allow, a page
    wider, and one so wide that units are cut: NaN and infinities where no token
    sees, rows that see nothing, sequences without new tokens."""
    dtype, N, Hq, Hkv, D, page = kernel
    rng = np.random.default_rng(31)
    width = tokens // page
    room = width * page - N
    ctx = [room, 0, room - 1, room // 2, 1, room // 3, room]
    B = len(ctx)
    n_new = [N, N, N, max(N - 1, 0), N, 0, N]
    s = Setup(31, ctx, N, Hq, Hkv, D, page, dtype, n_new=n_new, max_pages=width)
    sees = rng.random((B, N, N)) < 0.7
    sees[:, :, N // 2] = False
    for b in range(B):
        if n_new[b] > N // 2:
            p, i = s.slot(b, ctx[b] + N // 2)
            s.k[p, i], s.v[p, i] = math.nan, math.inf
    position = rng.integers(0, N, (B, N))
    table = s.table
    for more in (0, 1, -(-9000 // page)):
        s.table = np.concatenate([table, np.full((B, more), -1, np.int32)], 1)
        s.check(s.call(tree_mask=s.dev(mask_words(sees))), sees=sees, label=f"{more} pages more")
        kw = dict(window=max(tokens // 4, 1), sinks=3, position=position)
        s.check(s.call(**(kw | {"tree_mask": s.dev(mask_words(sees)), "position": s.dev(position)})),
                sees=sees, label=f"window, {more} pages more", **kw)
    # a table of the captured call's width, whatever the lengths: the rows that
    # see nothing are written too
    s.ctx[:] = 0
    none = np.zeros((B, N, N), bool)
    res = s.call(tree_mask=s.dev(mask_words(none)))
    s.check(res, sees=none)


@pytest.mark.parametrize("dtype,N,Hq,Hkv,D,page", KERNELS)
def test_more_whole_units_than_ctas(dtype, N, Hq, Hkv, D, page):
    rng = np.random.default_rng(32)
    B = 60 if N >= 40 else 500
    width = -(-(N + 30) // page)
    s = Setup(32, rng.integers(0, width * page - N + 1, B), N, Hq, Hkv, D, page, dtype,
              n_new=rng.integers(0, N + 1, B), max_pages=width)
    s.check(s.call())
    s.check(s.call(window=9, sinks=2), window=9, sinks=2)


@pytest.mark.parametrize("layout", ["nhd", "hnd", "pairs"])
@pytest.mark.parametrize("page", [12, 24, 40, 48, 96, 136, 200, 320])
@pytest.mark.parametrize("N,D", [(1, 128), (9, 64), (20, 128), (70, 64)])
def test_pages_of_any_multiple_of_eight(N, D, page, layout):
    """Pages that end inside tiles; one page of each table is bad."""
    s = Setup(33, [0, 7, page - 1, page, 3 * page + 5, 1000, 511], N, 8, 2, D, page, "bf16", layout=layout)
    s.table[4, 1] = -1
    res = s.call()
    s.check(res)
    assert res.flags.tolist() == [0, 0, 0, 0, sv.FLAG_BAD_PAGE, 0, 0]
    s.check(s.call(window=150, sinks=5), window=150, sinks=5)
