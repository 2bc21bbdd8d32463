"""The serving operators around a verification step: attention over a paged key-value cache, and the cache's pages.

A case is one pass of one of three kinds:
  attention  N new tokens of each of B sequences (one token, a chain of drafts, or a tree of them) attend to their
             sequence's pages; optionally a sliding window with a few first tokens that stay visible
  accept     what a step does to the cache around the verification: pages for the new tokens, their keys and values
             written, the accepted path moved together, the pages behind it given back
  fork       sequences that go on from another one's tokens: shared full pages, a copy of the last, partly filled one
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _attention(name, B, N, Hq, Hkv, D, dtype, page, lo, hi, tree=False, window=0, sinks=0):
    return {"name": name, "kind": "attention", "B": B, "N": N, "Hq": Hq, "Hkv": Hkv, "D": D, "dtype": dtype, "page": page,
            "lo": lo, "hi": hi, "tree": tree, "window": window, "sinks": sinks}


def _accept(name, L, B, N, Hkv, D, dtype, page, lo, hi, depth):
    return {"name": name, "kind": "accept", "L": L, "B": B, "N": N, "Hkv": Hkv, "D": D, "dtype": dtype, "page": page,
            "lo": lo, "hi": hi, "depth": depth}


def _fork(name, L, B, F, Hkv, D, dtype, page, lo, hi):
    return {"name": name, "kind": "fork", "L": L, "B": B, "F": F, "Hkv": Hkv, "D": D, "dtype": dtype, "page": page,
            "lo": lo, "hi": hi}


def listed():
    return [
        # one user, one token a step: the latency of a decode step
        _attention("token_one_sequence", 1, 1, 32, 8, 128, "bf16", 16, 1001, 1001),
        # the verifier's full batch decoding without drafts, contexts of every length
        _attention("token_batch_256", 256, 1, 32, 8, 128, "bf16", 16, 1, 4096),
        # long documents: two sequences share the whole card, seven query heads to a key head
        _attention("token_long", 2, 1, 28, 4, 128, "f16", 64, 65537, 131072),
        # a streaming drafter: long histories of which a window and four first tokens are visible
        _attention("token_window", 64, 1, 32, 8, 64, "bf16", 16, 200, 32768, window=1024, sinks=4),
        # a target scoring seven drafts and the token before them, in a batch
        _attention("chain_batch_64", 64, 8, 32, 8, 128, "bf16", 16, 1, 4096),
        # a small drafter in float32, five tokens a step, the smallest verification batch
        _attention("chain_f32", 4, 5, 8, 8, 64, "f32", 16, 17, 2000),
        # the verification workload's trees of sixty nodes
        _attention("tree_batch_32", 32, 60, 32, 8, 128, "bf16", 64, 64, 4096, tree=True),
        # the largest trees of the walk over long contexts: bound by the products
        _attention("tree_256_nodes", 16, 256, 64, 8, 128, "bf16", 64, 1000, 8192, tree=True),
        # a drafter of few layers, four sequences
        _accept("accept_small", 2, 4, 12, 8, 64, "bf16", 16, 1, 500, 4),
        # the verification workload's trees through all layers of a target
        _accept("accept_trees", 32, 32, 60, 8, 128, "bf16", 16, 64, 700, 6),
        # four continuations of one prompt
        _fork("fork_small", 4, 8, 3, 8, 128, "bf16", 16, 100, 400),
        # a batch of prompts forked at once through all layers
        _fork("fork_batch", 32, 128, 64, 8, 128, "bf16", 64, 33, 600),
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attention"] * 4 + ["accept", "fork"])
    dtype, page = rng.choice(["bf16", "bf16", "f16"]), rng.choice([8, 16, 32, 64, 128])
    Hkv, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    if kind == "accept":
        hi = _log_between(rng, 8, 700)
        N = rng.randint(2, 60)
        return _unnamed(_accept("", rng.randint(1, 32), rng.randint(1, 32), N, Hkv, D, dtype, page, rng.randint(0, hi), hi, rng.randint(1, min(6, N - 1))))
    if kind == "fork":
        hi, F = _log_between(rng, 8, 600), rng.randint(1, 64)
        return _unnamed(_fork("", rng.randint(1, 32), F + rng.randint(1, 64), F, Hkv, D, dtype, page, rng.randint(1, hi), hi))
    form = rng.choice(["token", "token", "window", "chain", "tree", "f32"])
    group = rng.choice([1, 2, 4, 5, 7, 8])
    B = _log_between(rng, 1, 256 if form == "token" else 64)
    hi = _log_between(rng, 16, min(131072, 1048576 // B) if form in ("token", "window") else min(8192, 131072 // B))
    lo = rng.randint(1, hi)
    if form == "token":
        return _unnamed(_attention("", B, 1, Hkv * group, Hkv, D, dtype, page, lo, hi))
    if form == "window":
        return _unnamed(_attention("", B, rng.randint(1, 4), Hkv * group, Hkv, D, dtype, page, lo, hi, window=_log_between(rng, 16, 4096), sinks=rng.randint(0, 8)))
    if form == "chain":
        return _unnamed(_attention("", B, rng.randint(2, 16), Hkv * group, Hkv, D, dtype, page, lo, hi))
    if form == "tree":
        return _unnamed(_attention("", min(B, 32), rng.randint(2, 128), Hkv * group, Hkv, D, dtype, page, lo, hi, tree=True))
    return _unnamed(_attention("", min(B, 16), rng.randint(1, 8), Hkv * group, Hkv, D, "f32", page, min(lo, 2000), min(hi, 2000)))


def _unnamed(case):
    return {k: v for k, v in case.items() if k != "name"}


def _spread(lo, hi, n):
    """n whole numbers spread evenly from lo to hi: the same ones for every seed, in an order that the seed gives."""
    return np.round(np.linspace(lo, hi, n)).astype(np.int64)


def _lengths(case, n):
    return _spread(case["lo"], case["hi"], n) if n > 1 else np.array([case["hi"]])


def _random_trees(rng, B, N):
    """parent, ancestor-or-self matrix and depth of random trees, the root node 0."""
    parent = np.full((B, N), -1, np.int64)
    sees = np.zeros((B, N, N), bool)
    depth = np.zeros((B, N), np.int64)
    rows = np.arange(B)
    sees[:, 0, 0] = True
    for n in range(1, N):
        parent[:, n] = np.minimum((rng.random(B) ** 2 * n).astype(np.int64), n - 1)
        sees[:, n] = sees[rows, parent[:, n]]
        sees[:, n, n] = True
        depth[:, n] = depth[rows, parent[:, n]] + 1
    return parent, sees, depth


def _mask_words(sees):
    """[B, N, N] truth values as the bit words of a tree mask: bit m % 64 of word m // 64."""
    B, N, _ = sees.shape
    bits = np.zeros((B, N, (N + 63) // 64 * 64), np.uint8)
    bits[:, :, :N] = sees
    return np.packbits(bits, axis=-1, bitorder="little").view("<i8").copy()


def _gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _views(flat, parts):
    """The arrays `parts`, as views of one tensor that holds them one behind another."""
    sizes = [x.size for x in parts]
    return [x.view(p.shape) for x, p in zip(flat.split(sizes), parts)]


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    B, page, Hkv, D, dt = case["B"], case["page"], case["Hkv"], case["D"], DTYPES[case["dtype"]]
    normal = lambda *shape: torch.randn(shape, generator=gen, device="cuda", dtype=dt)  # noqa: E731
    s = {"kind": case["kind"], "page": page}
    if case["kind"] == "attention":
        N, Hq = case["N"], case["Hq"]
        ctx = rng.permutation(_lengths(case, B))
        width = -(-(case["hi"] + N) // page)
        used = -(-(ctx + N) // page)
        pages = int(used.sum())
        order = rng.permutation(pages)
        table = np.zeros((B, width), np.int32)
        table[np.arange(width) < used[:, None]] = order
        s |= {"q": normal(B, N, Hq, D) * 1.5, "k": normal(pages, page, Hkv, D), "v": normal(pages, page, Hkv, D),
              "table": _gpu(table), "ctx": _gpu(ctx.astype(np.int32)), "window": case["window"], "sinks": case["sinks"],
              "mask": None, "position": None}
        if case["tree"]:
            _, sees, depth = _random_trees(rng, B, N)
            s |= {"mask": _gpu(_mask_words(sees)), "position": _gpu(depth.astype(np.int32))}
        return s
    # a pool in use: the sequences hold shuffled pages, the rest of them wait on the free list
    L = case["L"]
    live = case["F"] and B - case["F"] if case["kind"] == "fork" else B
    ctx = np.zeros(B, np.int64)
    ctx[:live] = rng.permutation(_lengths(case, live))
    count = -(-ctx // page)
    more = -(-(case["hi"] + case.get("N", 0)) // page) + 1
    pages = int(count.sum()) + (B * (more - case["lo"] // page) if case["kind"] == "accept" else case["F"])
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((B, more), -1, np.int32)
    held = int(count.sum())
    table[np.arange(more) < count[:, None]] = order[:held]
    refs = np.zeros(pages, np.int32)
    refs[order[:held]] = 1
    free = np.full(pages, -1, np.int32)
    free[:pages - held] = order[held:]
    parts = (table, count.astype(np.int32), refs, free, np.array([pages - held], np.int32), ctx.astype(np.int32))
    start = _gpu(np.concatenate([x.reshape(-1) for x in parts]))
    now = start.clone()
    s |= {"k": normal(L, pages, page, Hkv, D), "v": normal(L, pages, page, Hkv, D), "start": start, "all": now, "now": _views(now, parts)}
    if case["kind"] == "fork":
        F = case["F"]
        s |= {"src": _gpu(rng.integers(0, live, F).astype(np.int32)), "dst": _gpu((live + rng.permutation(F)).astype(np.int32))}
        return s
    N, depth = case["N"], case["depth"]
    taken = rng.permutation(_spread(0, depth, B))
    path = np.full((B, depth + 1), -1, np.int32)
    for b in range(B):
        path[b, 0] = 0
        path[b, 1:taken[b] + 1] = 1 + np.sort(rng.permutation(N - 1)[:taken[b]])
    s |= {"k_new": normal(L, B, N, Hkv, D), "v_new": normal(L, B, N, Hkv, D), "path": _gpu(path), "taken": _gpu(taken.astype(np.int32)),
          "N": N}
    return s


def run(s):
    if s["kind"] == "attention":
        if own:
            import speculative_decoding_verification_temp_gb300 as sv
            r = sv.paged_attention(s["q"], s["k"], s["v"], s["table"], s["ctx"], tree_mask=s["mask"], position=s["position"],
                                   window=s["window"], sinks=s["sinks"], return_lse=True)
            return {"out": r.out, "lse": r.lse}
        return _plain_attention(s)
    # the pass starts from the same pool each time
    s["all"].copy_(s["start"])
    table, count, refs, free, top, ctx = s["now"]
    if s["kind"] == "fork":
        if own:
            import speculative_decoding_verification_temp_gb300 as sv
            sv.cache_fork(sv.PagePool(table, count, refs, free, top), s["k"], s["v"], ctx, s["src"], s["dst"])
        else:
            _plain_fork(s)
        return {"k": s["k"], "v": s["v"], "table": table, "count": count, "refs": refs, "free": free, "top": top, "ctx": ctx}
    if own:
        import speculative_decoding_verification_temp_gb300 as sv
        pool = sv.PagePool(table, count, refs, free, top)
        sv.cache_resize(pool, ctx + s["N"], s["page"])
        sv.cache_append(s["k_new"], s["v_new"], s["k"], s["v"], table, ctx)
        length = sv.cache_compact(s["k"], s["v"], table, ctx, s["path"], s["taken"]).context_len
        sv.cache_resize(pool, length, s["page"])
    else:
        _plain_resize(s, ctx + s["N"])
        _plain_append(s)
        length = _plain_compact(s)
        _plain_resize(s, length)
    return {"k": s["k"], "v": s["v"], "table": table, "count": count, "refs": refs, "free": free, "top": top, "length": length}


def _plain_attention(s):
    q, ctx, table = s["q"], s["ctx"].long(), s["table"].long()
    B, N, Hq, D = q.shape
    page, Hkv = s["k"].shape[1:3]
    Lmax = table.shape[1] * page
    at = torch.arange(Lmax, device=q.device)
    inside = at[None, :] - ctx[:, None]  # place among the new tokens, negative in the context
    m = inside.clamp(0, N - 1)
    n = torch.arange(N, device=q.device)
    if s["mask"] is not None:
        words = torch.gather(s["mask"], 2, (m // 64)[:, None, :].expand(B, N, Lmax))
        sees = ((words >> (m % 64)[:, None, :]) & 1).bool()
        depth = s["position"].long()
    else:
        sees = m[:, None, :] <= n[None, :, None]
        depth = n[None, :].expand(B, N)
    sees = torch.where((inside < 0)[:, None, :], True, sees) & (inside < N)[:, None, :]
    if s["window"]:
        place = torch.where(inside < 0, at[None, :], ctx[:, None] + torch.gather(depth, 1, m))
        gap = (ctx[:, None] + depth)[:, :, None] - place[:, None, :]
        sees = sees & ((gap < s["window"]) | (place < s["sinks"])[:, None, :])
    k = s["k"][table].reshape(B, Lmax, Hkv, D).permute(0, 2, 3, 1).float()
    v = s["v"][table].reshape(B, Lmax, Hkv, D).permute(0, 2, 1, 3).float()
    rows = q.float().reshape(B, N, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    score = (rows @ k).mul_(D ** -0.5).reshape(B, Hkv, Hq // Hkv, N, Lmax)
    score.masked_fill_(~sees[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    weight = score.sub_(top).exp_()
    total = weight.sum(-1, keepdim=True)
    out = (weight.reshape(B, Hkv, -1, Lmax) @ v).reshape(B, Hkv, Hq // Hkv, N, D) / torch.where(total == 0, 1.0, total)
    lse = (top + total.log()).squeeze(-1)
    return {"out": out.permute(0, 3, 1, 2, 4).reshape(B, N, Hq, D).to(q.dtype), "lse": lse.permute(0, 3, 1, 2).reshape(B, N, Hq)}


def _plain_resize(s, length):
    """Gives pages back behind `length`, takes the missing ones before it; both in the order of sequences and their pages."""
    table, count, refs, free, top, _ = s["now"]
    B, width = table.shape
    pages, dev = refs.numel(), table.device
    need = (length.long() + s["page"] - 1) // s["page"]
    have = count.long()
    at = torch.arange(width, device=dev)[None, :]
    # pages given back: one reference less; a page without references goes to the free list at its first mention
    gone = ((at >= need[:, None]) & (at < have[:, None])).reshape(-1)
    spare = torch.full((), pages, device=dev)
    which = torch.where(gone, table.reshape(-1).long(), spare)
    wide = torch.cat([refs, refs.new_zeros(1)])
    wide.index_add_(0, which, -gone.to(torch.int32))
    mention = torch.arange(B * width, device=dev)
    first = torch.full((pages + 1,), B * width, device=dev).scatter_reduce_(0, which, mention, "amin")
    freed = gone & (wide[which] == 0) & (first[which] == mention)
    stack = torch.cat([free, free.new_zeros(1)])
    place = top.long() + freed.long().cumsum(0) - 1
    stack.scatter_(0, torch.where(freed, place, spare), which.to(torch.int32))
    filled = top.long() + freed.sum()
    table = torch.where(gone.reshape(B, width), -1, table)
    # pages taken, from the end of the list
    want = (need - have).clamp(min=0)
    upto = want.cumsum(0)
    served = upto <= filled
    took = torch.where(served, want, 0)
    fresh = (at >= have[:, None]) & (at < (have + took)[:, None])
    deep = filled - 1 - (upto - want)[:, None] - (at - have[:, None])
    deep = torch.where(fresh, deep, spare)
    table = torch.where(fresh, stack[deep], table)
    wide.scatter_(0, torch.where(fresh, table.long(), spare).reshape(-1), torch.ones(B * width, dtype=torch.int32, device=dev))
    stack.scatter_(0, deep.reshape(-1), torch.full((B * width,), -1, dtype=torch.int32, device=dev))
    for x, y in zip(s["now"], (table, torch.where(want > 0, have + took, torch.minimum(have, need)), wide[:-1], stack[:-1], filled - took.sum())):
        x.copy_(y)


def _slots(s, at):
    """Row numbers in [pages * page) of the token places at [B, n]."""
    table = s["now"][0].long()
    return torch.gather(table, 1, at // s["page"]) * s["page"] + at % s["page"]


def _plain_append(s):
    N, ctx = s["N"], s["now"][5].long()
    rows = _slots(s, ctx[:, None] + torch.arange(N, device=ctx.device)).reshape(-1)
    for cache, new in ((s["k"], s["k_new"]), (s["v"], s["v_new"])):
        L, _, _, H, D = cache.shape
        cache.view(L, -1, H, D)[:, rows] = new.reshape(L, -1, H, D)


def _plain_compact(s):
    ctx, path, taken = s["now"][5].long(), s["path"].long(), s["taken"].long()
    i = torch.arange(path.shape[1], device=ctx.device)[None, :]
    src = _slots(s, ctx[:, None] + torch.where(i <= taken[:, None], path, i)).reshape(-1)
    dst = _slots(s, ctx[:, None] + i).reshape(-1)
    for cache in (s["k"], s["v"]):
        flat = cache.view(cache.shape[0], -1, *cache.shape[3:])
        flat[:, dst] = flat[:, src]
    return (ctx + taken + 1).to(torch.int32)


def _plain_fork(s):
    table, count, refs, free, top, ctx = s["now"]
    page, src, dst = s["page"], s["src"].long(), s["dst"].long()
    length = ctx.long()[src]
    full, rest = length // page, length % page
    at = torch.arange(table.shape[1], device=table.device)[None, :]
    old = table[src].long()
    shared = at < full[:, None]
    spare = torch.full((), refs.numel(), device=table.device)
    wide = torch.cat([refs, refs.new_zeros(1)])
    wide.index_add_(0, torch.where(shared, old, spare).reshape(-1), shared.reshape(-1).to(torch.int32))
    part = rest > 0
    deep = torch.where(part, top.long() - part.long().cumsum(0), spare)
    stack = torch.cat([free, free.new_zeros(1)])
    fresh = stack[deep].long()
    stack.scatter_(0, deep, torch.full_like(dst, -1, dtype=torch.int32))
    wide.scatter_(0, torch.where(part, fresh, spare), torch.ones_like(dst, dtype=torch.int32))
    new = torch.where(shared, old, torch.where(part[:, None] & (at == full[:, None]), fresh[:, None], -1))
    table[dst] = new.to(torch.int32)
    count[dst] = (full + part).to(torch.int32)
    ctx[dst] = length.to(torch.int32)
    for x, y in ((refs, wide[:-1]), (free, stack[:-1]), (top, top - part.sum())):
        x.copy_(y)
    # the rows of the last pages; rows that a page does not hold yet keep what they have
    last = torch.gather(old, 1, torch.where(part, full, 0)[:, None]).squeeze(1)
    into = torch.where(part, fresh, last)
    filled = torch.arange(page, device=table.device)[None, :] < torch.where(part, rest, 0)[:, None]
    for cache in (s["k"], s["v"]):
        cache[:, into] = torch.where(filled[None, :, :, None, None], cache[:, last], cache[:, into])


def work(case):
    size = torch.empty(0, dtype=DTYPES[case["dtype"]]).element_size()
    B, Hkv, D, page = case["B"], case["Hkv"], case["D"], case["page"]
    row = 2 * Hkv * D * size  # a token's key and value
    if case["kind"] == "attention":
        N, Hq = case["N"], case["Hq"]
        ctx = _lengths(case, B)
        seen, read = ctx, ctx
        if case["window"]:
            seen = np.minimum(ctx, case["window"] - 1 + np.minimum(case["sinks"], np.maximum(ctx - case["window"] + 1, 0)))
            read = np.minimum(ctx, seen + N - 1)
        among = 0.5 * N * (N + 1) if not case["tree"] else N * (1 + math.log2(N + 1))
        pairs = float(seen.sum()) * N + B * (min(among, N * case["window"]) if case["window"] else among)
        moved = (float(read.sum()) + B * N) * row + B * N * Hq * (2 * D * size + 4)
        moved += 4.0 * B + 4 * float((-(-(read + N) // page)).sum()) + (8.0 * B * N * ((N + 63) // 64) if case["tree"] else 0)
        return {"bytes": moved, "flops": 4.0 * D * Hq * pairs}
    L = case["L"]
    if case["kind"] == "accept":
        moves = float(_spread(0, case["depth"], B).sum())
        return {"bytes": 2.0 * L * row * (B * case["N"] + moves) + 16.0 * B * (case["depth"] + 4), "flops": 0.0}
    # half a page in the mean
    return {"bytes": 2.0 * L * row * case["F"] * page / 2 + 8.0 * case["F"] * (case["lo"] + case["hi"]) / 2 / page, "flops": 0.0}


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "attention":
        return _exact_attention(case, s)
    page, L = case["page"], case["L"]
    table, count, refs, free, top, ctx = [x.cpu().numpy().astype(np.int64) for x in s["now"]]
    stack = [int(p) for p in free[:top[0]]]
    hold = [[int(p) for p in table[b, :count[b]]] for b in range(case["B"])]
    k, v = s["k"], s["v"]
    flat = lambda x: x.view(L, -1, case["Hkv"], case["D"])  # noqa: E731

    def rows(b, places):
        return torch.tensor([hold[b][int(t) // page] * page + int(t) % page for t in places], device="cuda", dtype=torch.long)

    if case["kind"] == "fork":
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            n = int(ctx[a])
            hold[b] = hold[a][:n // page] + ([stack.pop()] if n % page else [])
            tail = range(n // page * page, n)
            if n % page:
                for x in (k, v):
                    flat(x)[:, rows(b, tail)] = flat(x)[:, rows(a, tail)]
    else:
        N = case["N"]
        path, taken = s["path"].tolist(), s["taken"].tolist()
        for b in range(case["B"]):
            while len(hold[b]) * page < ctx[b] + N:
                hold[b].append(stack.pop())
            for x, new in ((k, s["k_new"]), (v, s["v_new"])):
                flat(x)[:, rows(b, range(ctx[b], ctx[b] + N))] = new[:, b]
                for i in range(taken[b] + 1):
                    flat(x)[:, rows(b, [ctx[b] + i])] = new[:, b, path[b][i]:path[b][i] + 1]
    # the whole numbers have to be equal as they are
    none = {name: None for name in ("table", "count", "refs", "free", "top", "ctx" if case["kind"] == "fork" else "length")}
    return {"k": k, "v": v, **none}


def _exact_attention(case, s):
    B, N, Hq, Hkv, D = (case[x] for x in ("B", "N", "Hq", "Hkv", "D"))
    out = torch.zeros(B, N, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, N, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, ctx in enumerate(s["ctx"].tolist()):
        T = ctx + N
        ids = s["table"][b, :-(-T // case["page"])].long()
        k = s["k"][ids].flatten(0, 1)[:T].double()
        v = s["v"][ids].flatten(0, 1)[:T].double()
        place = torch.arange(T, device="cuda")
        visible = torch.ones(N, T, dtype=torch.bool, device="cuda")
        if s["mask"] is None:
            visible[:, ctx:] = torch.ones(N, N, dtype=torch.bool, device="cuda").tril()
        else:
            bits = np.unpackbits(s["mask"][b].cpu().numpy().view(np.uint8), axis=-1, bitorder="little")[:, :N]
            visible[:, ctx:] = torch.from_numpy(bits.astype(bool)).cuda()
            place[ctx:] = ctx + s["position"][b].long()
        if case["window"]:
            visible &= (place[ctx:, None] - place[None, :] < case["window"]) | (place[None, :] < case["sinks"])
        for h in range(Hq):
            key, value = k[:, h // (Hq // Hkv)], v[:, h // (Hq // Hkv)]
            z = torch.where(visible, s["q"][b, :, h].double() @ key.T / math.sqrt(D), -math.inf)
            lse[b, :, h] = torch.logsumexp(z, -1)
            out[b, :, h] = torch.softmax(z, -1) @ value
    return {"out": out, "lse": lse}
