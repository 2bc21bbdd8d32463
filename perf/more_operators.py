"""The serving operators next to the paged key-value cache: the position rotation, appending with it, and a cache in 4 bits.

A case is one pass of one of four kinds:
  rotary     packed tokens' heads rotated by their positions (half or interleaved pairs, all or part of the head, plain or scaled frequencies)
  append     new tokens of each sequence: queries rotated, keys rotated and written to their pages, values written
  append4    the same into a cache of 4-bit rows, and the new tokens' rows read back as the values that they stand for
  attention4 attention of new tokens (one, a chain, a tree) over a cache of 4-bit rows

A 4-bit row of a head of D values is D/8 little-endian words of 32 bits, then four pairs (scale, minimum) of float16, one for each group of D/4
values.  Bits 4i of word w hold the code of value 8w + 2i, bits 16 + 4i that of value 8w + 2i + 1 (i = 0..3); a code n stands for minimum + scale n.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BASE = 10000.0
LIMIT = 61440.0  # of what a 4-bit row holds


def _rotary(name, T, H, D, dim, dtype, far, interleaved=False, factor=1.0):
    return {"name": name, "kind": "rotary", "T": T, "H": H, "D": D, "dim": dim, "dtype": dtype, "far": far, "interleaved": interleaved,
            "factor": factor}


def _append(name, bits, B, N, Hq, Hkv, D, dim, dtype, page, lo, hi, tree=False, ragged=False, interleaved=False, factor=1.0):
    return {"name": name, "kind": "append4" if bits == 4 else "append", "B": B, "N": N, "Hq": Hq, "Hkv": Hkv, "D": D, "dim": dim, "dtype": dtype,
            "page": page, "lo": lo, "hi": hi, "tree": tree, "ragged": ragged, "interleaved": interleaved, "factor": factor}


def _attention(name, B, N, Hq, Hkv, D, dtype, page, lo, hi, tree=False, window=0, sinks=0):
    return {"name": name, "kind": "attention4", "B": B, "N": N, "Hq": Hq, "Hkv": Hkv, "D": D, "dtype": dtype, "page": page, "lo": lo, "hi": hi,
            "tree": tree, "window": window, "sinks": sinks}


def listed():
    return [
        # one token of one user: queries and keys of a layer in one projection
        _rotary("rotary_step", 1, 40, 128, 128, "bf16", 4096),
        # packed prompts of a batch, with frequencies scaled for long contexts
        _rotary("rotary_prompts", 16384, 40, 128, 128, "bf16", 131072, factor=8.0),
        # one user, one token a step: the latency of a decode step
        _append("append_step", 16, 1, 1, 32, 8, 128, 128, "bf16", 16, 1001, 1001),
        # the verification workload's trees of sixty nodes, whose positions are depths
        _append("append_trees", 16, 32, 60, 32, 8, 128, 128, "bf16", 64, 64, 4096, tree=True),
        # prompts of different lengths, half of each head rotated in interleaved pairs
        _append("append_prompts", 16, 5, 4001, 32, 8, 128, 64, "f16", 16, 0, 1000, ragged=True, interleaved=True),
        # the verifier's full batch decoding without drafts, into 4 bits
        _append("append4_batch_256", 4, 256, 1, 32, 8, 128, 128, "bf16", 16, 1, 4096),
        # a chunk of a prompt in each of sixteen sequences, into 4 bits
        _append("append4_chunks", 4, 16, 512, 32, 8, 64, 64, "f16", 32, 0, 3000, factor=4.0),
        # one user, one token a step over a 4-bit cache
        _attention("token4_one_sequence", 1, 1, 32, 8, 128, "bf16", 16, 1001, 1001),
        # the verifier's full batch decoding without drafts, contexts of every length
        _attention("token4_batch_256", 256, 1, 32, 8, 128, "bf16", 16, 1, 4096),
        # long documents, what 4 bits are for: two sequences share the whole card, seven query heads to a key head
        _attention("token4_long", 2, 1, 28, 4, 128, "f16", 64, 65537, 131072),
        # a target scoring seven drafts and the token before them, in a batch
        _attention("chain4_batch_64", 64, 8, 32, 8, 128, "bf16", 16, 1, 4096),
        # the verification workload's trees of sixty nodes
        _attention("tree4_batch_32", 32, 60, 32, 8, 128, "bf16", 64, 64, 4096, tree=True),
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rotary", "append", "append4", "attention4", "attention4", "attention4"])
    factor = rng.choice([1.0, 4.0, 16.0])
    if kind == "rotary":
        dtype = rng.choice(["bf16", "f16", "f32"])
        D = rng.choice([64, 80, 96, 128, 256])
        T, H = _log_between(rng, 1, 16384), rng.randint(1, 40)
        while T * H * D * (2 if dtype == "f32" else 1) > 16384 * 40 * 128:
            T = T // 2 + 1
        return _unnamed(_rotary("", T, H, D, rng.choice([D, D, D // 2]), dtype, _log_between(rng, 2, 131072), rng.random() < 0.5, factor))
    page = rng.choice([8, 16, 32, 64, 128])
    Hkv, group, D = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 7, 8]), rng.choice([64, 128])
    if kind in ("append", "append4"):
        B = _log_between(rng, 1, 256)
        N = _log_between(rng, 1, min(4001, max(1, 8192 // B)))
        hi = _log_between(rng, 1, 4096)
        while Hkv * group > 40:
            group -= 1
        return _unnamed(_append("", 4 if kind == "append4" else 16, B, N, Hkv * group, Hkv, D, rng.choice([D, D // 2]),
                                rng.choice(["bf16", "f16", "f32"] if kind == "append" else ["bf16", "f16"]), page, rng.randint(0, hi), hi,
                                tree=rng.random() < 0.3 and N <= 128, ragged=rng.random() < 0.3, interleaved=rng.random() < 0.5, factor=factor))
    dtype = rng.choice(["bf16", "bf16", "f16"])
    form = rng.choice(["token", "token", "window", "chain", "tree"])
    B = _log_between(rng, 1, 256 if form == "token" else 64)
    hi = _log_between(rng, 16, min(131072, 1048576 // B) if form in ("token", "window") else min(8192, 131072 // B))
    lo = rng.randint(1, hi)
    if form == "token":
        return _unnamed(_attention("", B, 1, Hkv * group, Hkv, D, dtype, page, lo, hi))
    if form == "window":
        return _unnamed(_attention("", B, rng.randint(1, 4), Hkv * group, Hkv, D, dtype, page, lo, hi, window=_log_between(rng, 16, 4096), sinks=rng.randint(0, 8)))
    if form == "chain":
        return _unnamed(_attention("", B, rng.randint(2, 16), Hkv * group, Hkv, D, dtype, page, lo, hi))
    return _unnamed(_attention("", min(B, 32), rng.randint(2, 96), Hkv * group, Hkv, D, dtype, page, lo, hi, tree=True))


def _unnamed(case):
    return {k: v for k, v in case.items() if k != "name"}


def _spread(lo, hi, n):
    """n whole numbers spread evenly from lo to hi: the same ones for every seed, in an order that the seed gives."""
    return np.round(np.linspace(lo, hi, n)).astype(np.int64) if n > 1 else np.array([hi])


def _fresh(case):
    """New tokens of the sequences, before the seed orders them."""
    return _spread(0, case["N"], case["B"]) if case["ragged"] else np.full(case["B"], case["N"])


def _frequency(case):
    """Radians a token of each pair; those of long waves divided by the factor, those of short waves kept, the ones between mixed."""
    dim, factor = case["dim"], case["factor"]
    f = BASE ** (-np.arange(0, dim, 2) / dim)
    turns = f * 4096 / (2 * math.pi)  # over the context that the model was trained on
    keep = np.clip((turns - 1) / 31, 0, 1)
    return f * keep + f / factor * (1 - keep)


def _random_trees(rng, B, N):
    """ancestor-or-self matrix and depth of random trees, the root node 0."""
    sees = np.zeros((B, N, N), bool)
    depth = np.zeros((B, N), np.int64)
    rows = np.arange(B)
    sees[:, 0, 0] = True
    for n in range(1, N):
        parent = np.minimum((rng.random(B) ** 2 * n).astype(np.int64), n - 1)
        sees[:, n] = sees[rows, parent]
        sees[:, n, n] = True
        depth[:, n] = depth[rows, parent] + 1
    return sees, depth


def _mask_words(sees):
    """[B, N, N] truth values as the bit words of a tree mask: bit m % 64 of word m // 64."""
    B, N, _ = sees.shape
    bits = np.zeros((B, N, (N + 63) // 64 * 64), np.uint8)
    bits[:, :, :N] = sees
    return np.packbits(bits, axis=-1, bitorder="little").view("<i8").copy()


def _gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    normal = lambda *shape: torch.randn(shape, generator=gen, device="cuda", dtype=dt)  # noqa: E731
    s = {"kind": case["kind"]}
    if case["kind"] == "rotary":
        # sequences one behind another, from places of their own
        T = case["T"]
        ends = np.sort(rng.integers(0, T, max(1, T // 700)))
        start = rng.integers(0, case["far"], len(ends) + 1)
        which = np.searchsorted(ends, np.arange(T), side="right")
        begin = np.concatenate([[0], ends])[which]
        position = np.minimum(start[which] + np.arange(T) - begin, case["far"] - 1)
        return s | {"x": normal(T, case["H"], case["D"]), "position": _gpu(position.astype(np.int32)), "frequency": _gpu(_frequency(case)),
                    "interleaved": case["interleaved"]}
    B, N, Hq, Hkv, D, page = (case[x] for x in ("B", "N", "Hq", "Hkv", "D", "page"))
    ctx = rng.permutation(_spread(case["lo"], case["hi"], B))
    width = -(-(case["hi"] + N) // page)
    used = -(-(ctx + N) // page)
    pages = int(used.sum())
    table = np.zeros((B, width), np.int32)
    table[np.arange(width) < used[:, None]] = rng.permutation(pages)
    sees, depth = _random_trees(rng, B, N) if case["tree"] else (None, None)
    s |= {"q": normal(B, N, Hq, D) * 1.5, "table": _gpu(table), "ctx": _gpu(ctx.astype(np.int32)),
          "position": _gpu(depth.astype(np.int32)) if case["tree"] else None, "dtype": dt}
    if case["kind"] == "attention4":
        # what real keys have, channels with a level and a spread of their own
        level = torch.randn(2, Hkv, 1, D, generator=gen, device="cuda")
        spread = torch.rand(2, Hkv, 1, D, generator=gen, device="cuda") + 0.5
        k, v = (torch.empty(pages, Hkv, page, D // 2 + 16, dtype=torch.uint8, device="cuda") for _ in "kv")
        step = max(1, (1 << 26) // (Hkv * page * D))
        for i in range(0, pages, step):
            for j, x in enumerate((k, v)):
                part = x[i:i + step]
                rows = torch.randn(*part.shape[:3], D, generator=gen, device="cuda")
                part.copy_(_pack(rows * spread[j] + level[j]))
        return s | {"k": k.transpose(1, 2), "v": v.transpose(1, 2), "mask": _gpu(_mask_words(sees)) if case["tree"] else None,
                    "window": case["window"], "sinks": case["sinks"]}
    if case["kind"] == "append":
        k, v = normal(pages, page, Hkv, D), normal(pages, page, Hkv, D)
    else:
        k, v = (torch.zeros(pages, Hkv, page, D // 2 + 16, dtype=torch.uint8, device="cuda").transpose(1, 2) for _ in "kv")
    return s | {"k": k, "v": v, "k_new": normal(B, N, Hkv, D), "v_new": normal(B, N, Hkv, D), "out": torch.zeros_like(s["q"]),
                "fresh": _gpu(rng.permutation(_fresh(case)).astype(np.int32)) if case["ragged"] else None,
                "frequency": _gpu(_frequency(case)), "interleaved": case["interleaved"], "N": N}


def run(s):
    if s["kind"] == "rotary":
        if own:
            import speculative_decoding_verification_temp_gb300 as sv
            return sv.rotary(s["x"], s["position"], s["frequency"], interleaved=s["interleaved"])
        return _plain_rotate(s["x"], s["position"], s["frequency"], s["interleaved"])
    if s["kind"] == "attention4":
        if own:
            import speculative_decoding_verification_temp_gb300 as sv
            return sv.paged_attention(s["q"], s["k"], s["v"], s["table"], s["ctx"], tree_mask=s["mask"], position=s["position"],
                                      window=s["window"], sinks=s["sinks"]).out
        return _plain_attention(s)
    if own:
        import speculative_decoding_verification_temp_gb300 as sv
        sv.cache_append_rotary(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["ctx"], s["frequency"], q=s["q"], out=s["out"],
                               position=s["position"], num_new=s["fresh"], interleaved=s["interleaved"])
        if s["kind"] == "append4":
            r = sv.cache_read(s["k"], s["v"], s["table"], s["ctx"], s["N"], num=s["fresh"], dtype=s["dtype"])
            return {"q": s["out"], "k": r.k, "v": r.v}
    else:
        _plain_append(s)
        if s["kind"] == "append4":
            k, v = _plain_read(s)
            return {"q": s["out"], "k": k, "v": v}
    return {"q": s["out"], "k": s["k"], "v": s["v"]}


def _plain_rotate(x, position, frequency, interleaved):
    """x [..., heads, D] by position [...]; the angles in 64 bits."""
    angle = position.double()[..., None, None] * frequency
    cos, sin = angle.cos().float(), angle.sin().float()
    half = frequency.numel()
    y = x.float()
    turn, rest = y[..., :2 * half], y[..., 2 * half:]
    a, b = (turn[..., 0::2], turn[..., 1::2]) if interleaved else (turn[..., :half], turn[..., half:])
    a, b = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, rest], -1).to(x.dtype)


def _pack(x):
    """Rows of values [..., D] as 4-bit rows [..., D/2 + 16] of bytes."""
    D = x.shape[-1]
    group = x.float().clamp(-LIMIT, LIMIT).unflatten(-1, (4, D // 4))
    low = group.amin(-1, keepdim=True).half()
    scale = ((group.amax(-1, keepdim=True) - low.float()) / 15).half()
    code = ((group - low.float()) * torch.where(scale == 0, 0.0, 1 / scale.float())).round().clamp(0, 15)
    code = code.to(torch.uint8).flatten(-2).unflatten(-1, (D // 8, 4, 2))
    # a word's bytes: even values two by two, then odd ones
    pairs = (code[..., 0::2, :] | code[..., 1::2, :] << 4).transpose(-1, -2).flatten(-3)
    return torch.cat([pairs, torch.cat([scale, low], -1).flatten(-2).contiguous().view(torch.uint8)], -1)


def _unpack(rows):
    """4-bit rows as float32 values."""
    D = (rows.shape[-1] - 16) * 2
    pair = rows[..., D // 2:].contiguous().view(torch.float16).float().unflatten(-1, (4, 1, 2))
    pieces = rows[..., :D // 2].unflatten(-1, (D // 8, 2, 2)).transpose(-1, -2)  # [word, byte, even or odd]
    code = torch.stack([pieces & 15, pieces >> 4], -2).flatten(-4).float().unflatten(-1, (4, D // 4))
    return (pair[..., 1] + pair[..., 0] * code).flatten(-2)


def _places(s):
    """Row numbers in [pages * page) of the new tokens, [B, N], and which of them there are."""
    N, page, table = s["N"], s["k"].shape[1], s["table"].long()
    n = torch.arange(N, device=table.device)
    at = s["ctx"].long()[:, None] + n
    there = n < (s["fresh"][:, None] if s["fresh"] is not None else N)
    return torch.gather(table, 1, at // page) * page + at % page, there.expand(at.shape)


def _plain_append(s):
    rows, there = _places(s)
    place = s["ctx"].long()[:, None] + (s["position"] if s["position"] is not None else torch.arange(s["N"], device=rows.device))
    turn = lambda x: _plain_rotate(x, place, s["frequency"], s["interleaved"])  # noqa: E731
    s["out"].copy_(torch.where(there[..., None, None], turn(s["q"]), s["out"]))
    for cache, new in ((s["k"], turn(s["k_new"])), (s["v"], s["v_new"])):
        page = cache.shape[1]
        new = _pack(new) if s["kind"] == "append4" else new
        old = cache[rows // page, rows % page]
        cache[rows // page, rows % page] = torch.where(there[..., None, None], new, old)


def _plain_read(s):
    rows, there = _places(s)
    page = s["k"].shape[1]
    return [torch.where(there[..., None, None], _unpack(x[rows // page, rows % page]), 0.0).to(s["dtype"]) for x in (s["k"], s["v"])]


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
    k = _unpack(s["k"][table]).reshape(B, Lmax, Hkv, D).permute(0, 2, 3, 1)
    rows = q.float().reshape(B, N, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    score = (rows @ k).mul_(D ** -0.5).reshape(B, Hkv, Hq // Hkv, N, Lmax)
    del k
    score.masked_fill_(~sees[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    weight = score.sub_(top).exp_()
    total = weight.sum(-1, keepdim=True)
    v = _unpack(s["v"][table]).reshape(B, Lmax, Hkv, D).permute(0, 2, 1, 3)
    out = (weight.reshape(B, Hkv, -1, Lmax) @ v).reshape(B, Hkv, Hq // Hkv, N, D) / torch.where(total == 0, 1.0, total)
    return out.permute(0, 3, 1, 2, 4).reshape(B, N, Hq, D).to(q.dtype)


def work(case):
    size = torch.empty(0, dtype=DTYPES[case["dtype"]]).element_size()
    if case["kind"] == "rotary":
        values = case["T"] * case["H"]
        return {"bytes": 2.0 * values * case["D"] * size + 4.0 * case["T"], "flops": 3.0 * values * case["dim"]}
    B, N, Hq, Hkv, D, page = (case[x] for x in ("B", "N", "Hq", "Hkv", "D", "page"))
    row = 2 * Hkv * (D // 2 + 16)  # a token's key and value in 4 bits
    if case["kind"] != "attention4":
        tokens = float(_fresh(case).sum())
        fresh = 2 * Hkv * D * size
        # 4-bit rows are written, read back and returned; rows of no token are returned as zeros
        moved = tokens * (2 * Hq * D * size + fresh) + (tokens * 2 * row + B * N * fresh if case["kind"] == "append4" else tokens * fresh)
        return {"bytes": moved + 4.0 * B + 4.0 * tokens / page, "flops": 3.0 * tokens * (Hq + Hkv) * case["dim"]}
    ctx = _spread(case["lo"], case["hi"], B)
    seen, read = ctx, ctx
    if case["window"]:
        seen = np.minimum(ctx, case["window"] - 1 + np.minimum(case["sinks"], np.maximum(ctx - case["window"] + 1, 0)))
        read = np.minimum(ctx, seen + N - 1)
    among = 0.5 * N * (N + 1) if not case["tree"] else N * (1 + math.log2(N + 1))
    pairs = float(seen.sum()) * N + B * (min(among, N * case["window"]) if case["window"] else among)
    moved = (float(read.sum()) + B * N) * row + B * N * Hq * 2 * D * size
    moved += 4.0 * B + 4 * float((-(-(read + N) // page)).sum()) + (8.0 * B * N * ((N + 63) // 64) if case["tree"] else 0)
    return {"bytes": moved, "flops": 4.0 * D * Hq * pairs}


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "rotary":
        return _exact_rotation(s["x"], s["position"], s["frequency"], s["interleaved"])
    if case["kind"] == "attention4":
        return _exact_attention(case, s)
    B, N, page = case["B"], case["N"], case["page"]
    ctx, table = s["ctx"].tolist(), s["table"].cpu().numpy()
    fresh = s["fresh"].tolist() if case["ragged"] else [N] * B
    q = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    if case["kind"] == "append":
        k, v = s["k"].double(), s["v"].double()
    else:
        k, v = (torch.zeros(s["k_new"].shape, dtype=torch.float64, device="cuda") for _ in "kv")
    for b in range(B):
        n = fresh[b]
        place = ctx[b] + (s["position"][b, :n] if case["tree"] else torch.arange(n, device="cuda"))
        turn = lambda x: _exact_rotation(x, place, s["frequency"], s["interleaved"])  # noqa: E731, B023
        q[b, :n] = turn(s["q"][b, :n])
        key, value = turn(s["k_new"][b, :n]), s["v_new"][b, :n].double()
        if case["kind"] == "append4":
            # the rows are made of keys in the type that they come in
            k[b, :n], v[b, :n] = (_exact_four_bits(x.to(s["dtype"]).double()) for x in (key, value))
        else:
            at = np.arange(ctx[b], ctx[b] + n)
            slot = _gpu(table[b, at // page].astype(np.int64) * page + at % page)
            k.flatten(0, 1)[slot], v.flatten(0, 1)[slot] = key, value
    return {"q": q, "k": k, "v": v}


def _exact_rotation(x, position, frequency, interleaved):
    half = frequency.numel()
    angle = position.double()[:, None, None] * frequency
    y = x.double().clone()
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    z = torch.complex(y[..., first], y[..., second]) * torch.polar(torch.ones_like(angle), angle)
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_four_bits(x):
    """The values that the 4-bit rows of x stand for."""
    out = []
    for g in x.chunk(4, -1):
        low = g.min(-1, keepdim=True).values.half().double()
        scale = ((g.max(-1, keepdim=True).values - low) / 15).half().double()
        n = torch.where(scale == 0, 0.0, torch.round((g - low) / scale)).clamp(0, 15)
        out.append(low + scale * n)
    return torch.cat(out, -1)


def _exact_values(rows):
    """4-bit rows in float64, from the bits of their words."""
    D = (rows.shape[-1] - 16) * 2
    word = rows[..., :D // 2].contiguous().view(torch.int32)
    bits = [4 * (i // 2) + 16 * (i % 2) for i in range(8)]
    code = torch.stack([(word >> at) & 15 for at in bits], -1).flatten(-2).double()
    pairs = rows[..., D // 2:].contiguous().view(torch.float16).double()
    scale, low = (pairs[..., i::2].repeat_interleave(D // 4, -1) for i in (0, 1))
    return low + scale * code


def _exact_attention(case, s):
    B, N, Hq, Hkv, D = (case[x] for x in ("B", "N", "Hq", "Hkv", "D"))
    out = torch.zeros(B, N, Hq, D, dtype=torch.float64, device="cuda")
    for b, ctx in enumerate(s["ctx"].tolist()):
        T = ctx + N
        ids = s["table"][b, :-(-T // case["page"])].long()
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
        for h in range(Hkv):
            key, value = (_exact_values(x[ids, :, h]).flatten(0, 1)[:T] for x in (s["k"], s["v"]))
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            z = torch.where(visible[:, None], s["q"][b, :, heads].double() @ key.T / math.sqrt(D), -math.inf)
            out[b, :, heads] = torch.softmax(z, -1) @ value
    return out
