"""Appending, compacting, resizing and forking a paged key-value cache against
plain computations on lists, and a decode step of all of them together."""

import numpy as np
import pytest
import torch

import speculative_decoding_verification_temp_gb300 as sv

from cache_helpers import DTYPES, check_attention, make_pages

pytestmark = pytest.mark.gpu


def gpu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def bits(x):
    """The tensor's bytes: moved rows are equal to the last bit, NaNs too."""
    x = x.contiguous()
    return x.view(torch.int32 if x.dtype == torch.float32 else torch.int16)


def random_rows(gen, *shape, dtype):
    """Any bit patterns."""
    if dtype == torch.float32:
        return torch.randint(-2 ** 31, 2 ** 31 - 1, shape, generator=gen, device="cuda",
                             dtype=torch.int64).to(torch.int32).view(torch.float32)
    return torch.randint(-2 ** 15, 2 ** 15, shape, generator=gen, device="cuda",
                         dtype=torch.int32).to(torch.int16).view(dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("layers,N,H,D,page", [(None, 1, 8, 128, 16), (3, 5, 2, 64, 16), (2, 70, 1, 8, 7),
                                               (1, 33, 5, 72, 1), (2, 4, 2, 256, 64)])
def test_append(dtype, layers, N, H, D, page):
    gen = torch.Generator("cuda")
    gen.manual_seed(1)
    rng = np.random.default_rng(1)
    dt = DTYPES[dtype]
    ctx = np.array([0, 1, 15, 16, 100, 3, 9], np.int32)
    n_new = np.array([N, 0, N, max(N - 1, 0), 1, N, N], np.int32)
    B = len(ctx)
    table, pages = make_pages(rng, ctx + N, page)
    lead = () if layers is None else (layers,)
    k, v = (random_rows(gen, *lead, pages, page, H, D, dtype=dt) for _ in "kv")
    fused = random_rows(gen, *lead, B, N, 3 * H, D, dtype=dt)  # queries, keys, values side by side
    kn, vn = fused[..., H:2 * H, :], fused[..., 2 * H:, :]
    table[5, 3 // page] = -5
    ctx[6] = table.shape[1] * page - N + 1
    want = []
    for cache, new in ((k, kn), (v, vn)):
        x = cache.clone().cpu().view(-1, pages, page, H, D)
        y = new.cpu().reshape(-1, B, N, H, D)
        for b in range(B - 1):
            for n in range(n_new[b]):
                t = int(ctx[b]) + n
                p = int(table[b, t // page])
                if 0 <= p < pages:
                    x[:, p, t % page] = y[:, b, n]
        want.append(x.view(cache.shape))
    flags = sv.cache_append(kn, vn, k, v, gpu(table), gpu(ctx), num_new=gpu(n_new), return_flags=True)
    torch.cuda.synchronize()
    assert flags.tolist() == [0, 0, 0, 0, 0, sv.FLAG_BAD_PAGE if N else 0, sv.FLAG_BAD_LENGTH]
    for x, y in zip((k, v), want):
        assert torch.equal(bits(x.cpu()), bits(y))
    before = k.clone()
    sv.cache_append(kn, vn, k, v, gpu(table), gpu(ctx), num_new=gpu(n_new))
    torch.cuda.synchronize()
    assert torch.equal(bits(k), bits(before))


@pytest.mark.parametrize("dtype,layers,H,D,page,layout", [
    ("bf16", None, 8, 128, 16, "nhd"), ("f32", 2, 2, 64, 5, "nhd"), ("f16", 3, 3, 72, 64, "hnd"),
    ("bf16", 2, 1, 8, 1, "nhd")])
def test_compact(dtype, layers, H, D, page, layout):
    gen = torch.Generator("cuda")
    gen.manual_seed(2)
    rng = np.random.default_rng(2)
    dt, N, width = DTYPES[dtype], 40, 12
    paths = [[0], [0, 1, 2, 3], [0, 5, 6, 39], [0, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12],
             [0, 7], list(range(0, 36, 3)), [0, 1, 3, 4, 9], [], [0, 4, 4], [1, 2], [0, 1, 39], [0, 20, 21]]
    B = len(paths)
    ctx = rng.integers(0, 100, B).astype(np.int32)
    ctx[0] = 0
    table, pages = make_pages(rng, ctx + N, page)
    path = np.full((B, width), -1, np.int32)
    taken = np.array([len(p) - 1 for p in paths], np.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    flags = np.zeros(B, np.int64)
    flags[8] = flags[9] = sv.FLAG_BAD_TREE
    ctx[10] = table.shape[1] * page - 39
    flags[10] = sv.FLAG_BAD_LENGTH
    table[11, (ctx[11] + 20) // page] = pages  # node 20's page
    flags[11] = sv.FLAG_BAD_PAGE
    lead = () if layers is None else (layers,)
    if layout == "nhd":
        k, v = (random_rows(gen, *lead, pages, page, H, D, dtype=dt) for _ in "kv")
    else:
        k, v = (random_rows(gen, *lead, pages, H, page, D, dtype=dt).transpose(-3, -2) for _ in "kv")
    want = []
    for cache in (k, v):
        x = cache.cpu().clone().view(-1, pages, page, H, D)
        old = x.clone()
        for b in range(B):
            if flags[b] not in (0, sv.FLAG_BAD_PAGE):
                continue
            for i in range(1, len(paths[b])):
                s, d = int(ctx[b]) + paths[b][i], int(ctx[b]) + i
                ps, pd = int(table[b, s // page]), int(table[b, d // page])
                if 0 <= ps < pages and 0 <= pd < pages:
                    x[:, pd, d % page] = old[:, ps, s % page]
        want.append(x.view(cache.shape))
    res = sv.cache_compact(k, v, gpu(table), gpu(ctx), gpu(path), gpu(taken))
    torch.cuda.synchronize()
    assert res.flags.tolist() == flags.tolist()
    for b in range(B):
        moved = flags[b] in (0, sv.FLAG_BAD_PAGE)
        assert int(res.context_len[b]) == ctx[b] + (len(paths[b]) if moved else 0), b
    for x, y in zip((k, v), want):
        assert torch.equal(bits(x.cpu()), bits(y))


def test_compact_of_a_long_path():
    """A chain of 4096 nodes with every second one accepted."""
    N, page = 4096, 16
    path = np.arange(0, N, 2, dtype=np.int32)[None]
    k = torch.arange((N + 5 + page) // page * page, device="cuda", dtype=torch.float32)
    k = k.view(-1, page, 1, 1).expand(-1, -1, 1, 4).contiguous()
    v = -k
    table = torch.arange(k.shape[0], device="cuda", dtype=torch.int32)[None]
    res = sv.cache_compact(k, v, table, gpu(np.array([5], np.int32)), gpu(path),
                           gpu(np.array([N // 2 - 1], np.int32)))
    torch.cuda.synchronize()
    got = k.view(-1, 4)[5:5 + N // 2, 0].cpu().numpy()
    assert np.array_equal(got, 5.0 + np.arange(0, N, 2))
    assert torch.equal(v, -k) and res.context_len.tolist() == [5 + N // 2]


class Pool:
    """The pool's definition, on lists."""

    def __init__(self, B, width, pages, page):
        self.width, self.page, self.pages = width, page, pages
        self.rows = [[] for _ in range(B)]
        self.refs = [0] * pages
        self.free = list(range(pages - 1, -1, -1))

    def resize(self, lengths):
        flags = [0] * len(lengths)
        need = [-(-n // self.page) for n in lengths]
        for b, n in enumerate(lengths):
            if n < 0 or need[b] > self.width:
                flags[b] = sv.FLAG_BAD_LENGTH
                need[b] = len(self.rows[b])
        gone = []
        for b in range(len(lengths)):
            gone += self.rows[b][need[b]:]
            self.rows[b] = self.rows[b][:max(need[b], 0)]
        for p in gone:
            self.refs[p] -= 1
        for p in gone:
            if self.refs[p] == 0 and p not in self.free:
                self.free.append(p)
        room, demand = len(self.free), 0
        for b in range(len(lengths)):
            want = max(need[b] - len(self.rows[b]), 0)
            demand += want
            if want and demand > room:
                flags[b] = sv.FLAG_NO_PAGES
            elif want:
                # the place of its pages does not depend on who was served
                for _ in range(want):
                    p = self.free.pop()
                    self.refs[p] = 1
                    self.rows[b].append(p)
        return flags

    def fork(self, ctx, src, dst):
        flags, old, oldctx = [0] * len(src), [list(r) for r in self.rows], list(ctx)
        B, room, demand, copies, named = len(ctx), len(self.free), 0, [], set()
        for f, (s, d) in enumerate(zip(src, dst)):
            if not (0 <= s < B and 0 <= d < B):
                flags[f] = sv.FLAG_BAD_SEQUENCE
                continue
            n = oldctx[s]
            if n < 0 or len(old[s]) < -(-n // self.page):
                flags[f] = sv.FLAG_BAD_LENGTH
                continue
            if old[d] or d in named:
                flags[f] = sv.FLAG_BAD_SEQUENCE
                continue
            named.add(d)
            full, rest = n // self.page, n % self.page
            demand += rest > 0
            if rest and demand > room:
                flags[f] = sv.FLAG_NO_PAGES
                continue
            for p in old[s][:full]:
                self.refs[p] += 1
            self.rows[d] = old[s][:full]
            if rest:
                p = self.free.pop()
                self.refs[p] = 1
                self.rows[d].append(p)
                copies.append((old[s][full], p, rest))
            ctx[d] = n
        return flags, copies

    def check(self, pool):
        torch.cuda.synchronize()
        table = np.full((len(self.rows), self.width), -1)
        for b, r in enumerate(self.rows):
            table[b, :len(r)] = r
        assert np.array_equal(pool.page_table.cpu().numpy(), table)
        assert pool.page_count.tolist() == [len(r) for r in self.rows]
        assert pool.ref_count.tolist() == self.refs
        assert pool.free_count.tolist() == [len(self.free)]
        assert pool.free_list.tolist() == self.free + [-1] * (self.pages - len(self.free))


@pytest.mark.parametrize("B,width,pages,page,seed", [(1, 8, 8, 16, 0), (5, 10, 30, 4, 1), (40, 70, 1500, 16, 2),
                                                     (1500, 5, 4000, 1, 3), (7, 100, 60, 3, 4)])
def test_resize_and_fork(B, width, pages, page, seed):
    rng = np.random.default_rng(seed)
    pool, want = sv.page_pool(B, width, pages), Pool(B, width, pages, page)
    want.check(pool)
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    k, v = (random_rows(gen, 2, pages, page, 2, 16, dtype=torch.bfloat16) for _ in "kv")
    length = np.zeros(B, np.int64)
    for step in range(12):
        grow = rng.random(B)
        new = np.where(grow < 0.15, 0, np.where(grow < 0.8, length + rng.integers(0, 3 * page + 2, B),
                                                rng.integers(0, length + 1)))
        if step % 4 == 3:
            new[rng.integers(0, B)] = -3
            new[rng.integers(0, B)] = width * page + 1
        flags = sv.cache_resize(pool, gpu(new.astype(np.int32)), page)
        expect = want.resize(new.tolist())
        want.check(pool)
        assert flags.tolist() == expect
        length = np.array([min(max(int(n), 0), len(r) * page) if f == 0 else max(len(r) * page - 1, 0)
                           for n, r, f in zip(new, want.rows, expect)])
        F = int(rng.integers(1, B + 3))
        src, dst = rng.integers(-1, B + 1, F), rng.integers(-1, B + 1, F)
        empty = [b for b in range(B) if not want.rows[b]]
        for i, b in enumerate(empty[:F]):
            dst[i] = b
        ctx = length.tolist()
        ctx_dev = gpu(length.astype(np.int32))
        flags = sv.cache_fork(pool, k, v, ctx_dev, gpu(src.astype(np.int32)), gpu(dst.astype(np.int32)))
        cache = [x.clone().cpu() for x in (k, v)] if step == 0 else cache
        expect, copies = want.fork(ctx, src.tolist(), dst.tolist())
        want.check(pool)
        assert flags.tolist() == expect
        assert ctx_dev.tolist() == ctx
        for x, y in zip(cache, (k, v)):
            if step > 0:
                for a, b, n in copies:
                    x[:, b, :n] = x[:, a, :n]
                assert torch.equal(bits(x), bits(y.cpu()))
            else:
                x.copy_(y.cpu())
        length = np.array(ctx)


def test_pages_named_twice_or_outside_are_flagged():
    pool = sv.page_pool(3, 4, 6)
    assert sv.cache_resize(pool, gpu(np.array([4, 4, 0], np.int32)), 2).tolist() == [0, 0, 0]
    pool.page_table[1, 0] = 77           # no page
    pool.page_table[1, 1] = pool.page_table[0, 1]  # given back twice, taken once
    flags = sv.cache_resize(pool, gpu(np.zeros(3, np.int32)), 2)
    torch.cuda.synchronize()
    assert flags[1] & sv.FLAG_BAD_PAGE
    n = int(pool.free_count)
    free = pool.free_list[:n].tolist()
    assert len(set(free)) == n and all(0 <= p < 6 for p in free)


def test_decode_steps_together():
    """Steps of a decode loop on two layers: pages, append, tree attention, tree
    verification, compaction, pages given back; then a fork that goes on.  After
    each step the attention of one token over the kept tokens is the plain one
    over a list of the kept keys and values."""
    rng = np.random.default_rng(5)
    gen = torch.Generator("cuda")
    gen.manual_seed(5)
    L, B, H, Hq, D, page, V, N = 2, 4, 2, 8, 64, 16, 512, 24
    seqs = B + 1
    pool = sv.page_pool(seqs, 20, 60)
    k = torch.full((L, 60, page, H, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    ctx = torch.zeros(seqs, dtype=torch.int32, device="cuda")
    kept = [[[] for _ in range(seqs)] for _ in range(2)]  # keys, values: [L, H, D] rows
    normal = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)
    first = np.array([5, 16, 33, 1, 0], np.int32)  # prompts of several lengths

    def add(kn, vn, rows):
        for x, new in zip(kept, (kn.cpu(), vn.cpu())):
            for b, at in enumerate(rows):
                x[b] += [new[:, b, i] for i in at]

    def look():
        q = normal(seqs, 1, Hq, D)
        lens = ctx.cpu().numpy()
        live = [b for b in range(seqs) if lens[b] > 0]
        for layer in range(L):
            at = torch.tensor(live, device="cuda")
            res = sv.paged_attention(q[at], k[layer], v[layer], pool.page_table[at],
                                     ctx[at] - 1, return_lse=True, return_flags=True)
            torch.cuda.synchronize()
            assert not res.flags.any()
            T = max(int(lens[b]) for b in live)
            plain = []
            for x in kept:
                flat = torch.zeros(len(live), T, H, D, dtype=torch.bfloat16)
                for i, b in enumerate(live):
                    assert len(x[b]) == lens[b]
                    flat[i, :lens[b]] = torch.stack([r[layer] for r in x[b]])
                plain.append(flat)
            table = np.arange(len(live), dtype=np.int32)[:, None]
            check_attention(res, q[at], *plain, table, lens[live] - 1, T, "bf16",
                            label=f"layer {layer}")

    def append(new, rows_of):
        assert not sv.cache_resize(pool, ctx + new, page).any()
        n = int(new.max())
        kn, vn = normal(L, seqs, n, H, D), normal(L, seqs, n, H, D)
        assert not sv.cache_append(kn, vn, k, v, pool.page_table, ctx, num_new=new,
                                   return_flags=True).any()
        return kn, vn

    new = gpu(first)
    kn, vn = append(new, None)
    add(kn, vn, [range(n) for n in first])
    ctx += new
    look()
    for step in range(3):
        live = (ctx > 0).to(torch.int32)
        trees = int(live.sum())
        parent = np.full((trees, N), -1, np.int32)
        for n in range(1, N):
            parent[:, n] = rng.integers(max(0, n - 5), n, trees)
        new = live * N
        kn, vn = append(new, None)
        mk = sv.tree_mask(gpu(parent), N)
        q = normal(seqs, N, Hq, D)
        mask = torch.zeros(seqs, N, 1, dtype=torch.int64, device="cuda")
        mask[:trees] = mk.mask
        for layer in range(L):
            res = sv.paged_attention(q, k[layer], v[layer], pool.page_table, ctx, num_new=new,
                                     tree_mask=mask, return_lse=True, return_flags=True)
            assert not res.flags.any()
            sees = np.unpackbits(mask.cpu().numpy().view(np.uint8), axis=-1,
                                 bitorder="little").reshape(seqs, N, -1)[:, :, :N].astype(bool)
            check_attention(res, q, k[layer], v[layer], pool.page_table.cpu().numpy(),
                            ctx.cpu().numpy(), page, "bf16", n_new=new.cpu().numpy(), sees=sees)
        logits = torch.randn(trees, N, V, generator=gen, device="cuda") * 2
        tokens = torch.randint(0, V, (trees, N), generator=gen, device="cuda", dtype=torch.int32)
        tokens[:, 1:] = logits.argmax(-1).to(torch.int32)[:, :1]  # some of them are accepted
        ver = sv.verify_tree(logits, logits, tokens, gpu(parent), N, 1.0, 1.0, seed=step)
        path = torch.full((seqs, N + 1), -1, dtype=torch.int32, device="cuda")
        path[:trees] = ver.path
        taken = torch.full((seqs,), -1, dtype=torch.int32, device="cuda")
        taken[:trees] = ver.num_accepted
        got = sv.cache_compact(k, v, pool.page_table, ctx, path, taken)
        assert not got.flags.any()
        add(kn, vn, [path[b, :int(taken[b]) + 1].tolist() for b in range(seqs)])
        ctx.copy_(got.context_len)
        assert not sv.cache_resize(pool, ctx, page).any()
        assert pool.page_count.tolist() == [-(-int(n) // page) for n in ctx]
        look()
        if step == 1:  # the empty sequence goes on from the third one's tokens
            flags = sv.cache_fork(pool, k, v, ctx, gpu(np.array([2], np.int32)),
                                  gpu(np.array([4], np.int32)))
            assert flags.tolist() == [0]
            for x in kept:
                x[4] = list(x[2])
            look()
    assert int(ctx[4]) > 0
    assert not sv.cache_resize(pool, torch.zeros_like(ctx), page).any()
    assert int(pool.free_count) == 60 and not pool.ref_count.any()


def test_a_captured_step_follows_its_inputs():
    """Pages, append, attention, compaction and pages given back, captured
    together and replayed over other lengths and paths, against the same calls
    outside a graph."""
    B, N, H, D, page, pages, width = 3, 6, 2, 64, 16, 64, 8
    gen = torch.Generator("cuda")
    gen.manual_seed(11)
    dt = torch.bfloat16
    new = [torch.randn(2, B, N, H, D, generator=gen, device="cuda").to(dt) for _ in "kv"]
    q = torch.randn(B, N, 4 * H, D, generator=gen, device="cuda").to(dt)
    parent = gpu(np.tile(np.array([-1, 0, 0, 1, 2, 4], np.int32), (B, 1)))
    mask = sv.tree_mask(parent, max_depth=8).mask
    ctx, path, taken = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((B,), (B, N), (B,)))
    start = [torch.randn(2, pages, page, H, D, generator=gen, device="cuda").to(dt) for _ in "kv"]

    def state():
        return sv.page_pool(B, width, pages), [x.clone() for x in start]

    def step(pool, kv):
        f0 = sv.cache_resize(pool, ctx + N, page)
        sv.cache_append(*new, *kv, pool.page_table, ctx)
        outs = [sv.paged_attention(q, kv[0][i], kv[1][i], pool.page_table, ctx, tree_mask=mask).out
                for i in range(2)]
        kept = sv.cache_compact(*kv, pool.page_table, ctx, path, taken)
        f1 = sv.cache_resize(pool, kept.context_len, page)
        return [*outs, kept.context_len, kept.flags, f0, f1]

    (pool_a, kv_a), (pool_b, kv_b) = state(), state()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = step(pool_a, kv_a)
    cases = [([0, 0, 0], [[0, 1, 3, -1, -1, -1], [0, 2, 4, 5, -1, -1], [0, -1, -1, -1, -1, -1]], [2, 3, 0]),
             ([3, 4, 1], [[0, 2, -1, -1, -1, -1], [0, -1, -1, -1, -1, -1], [0, 2, 4, 5, -1, -1]], [1, -1, 3]),
             ([100, 17, 5], [[0, 2, 4, 5, -1, -1], [0, 1, -1, -1, -1, -1], [0, 1, 3, -1, -1, -1]], [3, 1, 2]),
             ([90, 0, 122], [[0, 2, 4, -1, -1, -1], [0, 1, 3, -1, -1, -1], [0, 2, 4, 5, -1, -1]], [2, 2, 3])]
    for lengths, nodes, accepted in cases:
        ctx.copy_(torch.tensor(lengths, dtype=torch.int32))
        path.copy_(torch.tensor(nodes, dtype=torch.int32))
        taken.copy_(torch.tensor(accepted, dtype=torch.int32))
        graph.replay()
        want = step(pool_b, kv_b)
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
        for x, y in zip([*pool_a, *map(bits, kv_a)], [*pool_b, *map(bits, kv_b)]):
            assert torch.equal(x, y)
        assert not got[3].any() and not got[4].any() and not got[5].any()
        for x, y, t in zip(got[2].tolist(), lengths, accepted):
            assert x == y + t + 1


def test_a_shortened_sequence_goes_on_from_a_fork():
    """Appending behind a length inside a shared page would write the other
    holder's tokens; a fork at the shorter length has a page of its own there."""
    B, H, D, page, pages = 4, 2, 64, 16, 32
    gen = torch.Generator("cuda")
    gen.manual_seed(12)
    dt = torch.bfloat16
    kv = [torch.randn(pages, page, H, D, generator=gen, device="cuda").to(dt) for _ in "kv"]
    new = [torch.randn(B, 5, H, D, generator=gen, device="cuda").to(dt) for _ in "kv"]
    pool = sv.page_pool(B, 8, pages)
    ctx = gpu(np.array([32, 0, 0, 0], np.int32))
    assert not sv.cache_resize(pool, ctx, page).any()

    def row(b, n):
        return [x[pool.page_table[b].clamp(min=0).long()].flatten(0, 1)[:n].clone() for x in kv]

    first = row(0, 32)
    assert not sv.cache_fork(pool, *kv, ctx, gpu(np.array([0], np.int32)), gpu(np.array([1], np.int32))).any()
    ctx[1] = 20
    assert not sv.cache_fork(pool, *kv, ctx, gpu(np.array([1], np.int32)), gpu(np.array([2], np.int32))).any()
    assert ctx.tolist() == [32, 20, 20, 0]
    ctx[1] = 0
    assert not sv.cache_resize(pool, ctx, page).any()
    num = gpu(np.array([0, 0, 5, 0], np.int32))
    assert not sv.cache_resize(pool, ctx + num, page).any()
    assert not sv.cache_append(*new, *kv, pool.page_table, ctx, num_new=num, return_flags=True).any()
    torch.cuda.synchronize()
    table = pool.page_table.tolist()
    assert table[0][0] == table[2][0] and table[0][1] != table[2][1]
    for x, y in zip(row(0, 32), first):
        assert torch.equal(bits(x), bits(y))
    for x, y, z in zip(row(2, 25), first, new):
        assert torch.equal(bits(x[:20]), bits(y[:20])) and torch.equal(bits(x[20:]), bits(z[2]))


def test_the_first_calls_of_a_process_can_be_captured():
    """Nothing is set up, loaded or told to the driver before the capture."""
    import os
    import subprocess
    import sys
    script = """
import torch, speculative_decoding_verification_temp_gb300 as sv
cases = []
for dt, N, D in ((torch.bfloat16, 1, 128), (torch.float16, 9, 64), (torch.bfloat16, 70, 128), (torch.float32, 3, 64),
                 (torch.bfloat16, 2, 96)):
    g = torch.Generator("cuda"); g.manual_seed(N)
    k, v = (torch.randn(20, 16, 2, D, generator=g, device="cuda").to(dt) for _ in "kv")
    q = torch.randn(2, N, 8, D, generator=g, device="cuda").to(dt)
    cases.append((q, k, v, torch.arange(20, dtype=torch.int32, device="cuda").view(2, 10),
                  torch.tensor([5, 60], dtype=torch.int32, device="cuda")))
pool = sv.page_pool(2, 4, 8)
ctx = torch.tensor([20, 0], dtype=torch.int32, device="cuda")
kv = [torch.randn(8, 16, 2, 64, device="cuda") for _ in "kv"]
src, dst = (torch.tensor([x], dtype=torch.int32, device="cuda") for x in (0, 1))
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = [sv.paged_attention(*c).out for c in cases]
    flags = sv.cache_resize(pool, ctx, 16), sv.cache_fork(pool, *kv, ctx, src, dst)
graph.replay()
torch.cuda.synchronize()
for x, c in zip(got, cases):
    assert torch.equal(x, sv.paged_attention(*c).out)
assert not any(f.any() for f in flags) and ctx.tolist() == [20, 20]
print("captured")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", script], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and "captured" in done.stdout, done.stderr[-2000:]
