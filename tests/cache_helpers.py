"""Helpers of the key-value cache tests: caches with shuffled pages and plain
64-bit references, written from the operators' definitions."""

import math

import numpy as np
import torch

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def make_pages(rng, lens, page, max_pages=None, spare=3):
    """A page table for sequences of `lens` tokens on shuffled pages; unused
    entries hold an id outside the cache.  Returns (table, num_pages)."""
    used = [-(-int(n) // page) for n in lens]
    width = max(max(used), 1) if max_pages is None else max_pages
    pages = sum(used) + spare
    order = rng.permutation(pages)
    table = np.full((len(used), width), 1 << 30, np.int32)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pages


def random_trees(rng, B, N):
    parent = np.full((B, N), -1, np.int32)
    for n in range(1, N):
        parent[:, n] = (rng.random(B) ** 2 * n).astype(np.int32)
    return parent


def mask_words(sees):
    """[B, N, N] truth values as tree mask words [B, N, ceil(N/64)]."""
    B, N, _ = sees.shape
    bits = np.zeros((B, N, -(-N // 64) * 64), np.uint8)
    bits[:, :, :N] = sees
    return np.packbits(bits, axis=-1, bitorder="little").view("<i8").reshape(B, N, -1).copy()


def visible(ctx, n_new, N, sees=None, position=None, window=0, sinks=0):
    """[n_new, ctx + n_new] truth values, from the definition, element by element
    along the new tokens."""
    T = ctx + n_new
    out = np.ones((n_new, T), bool)
    block = np.tril(np.ones((n_new, n_new), bool)) if sees is None else sees[:n_new, :n_new]
    out[:, ctx:] = block
    if window > 0:
        pos = np.arange(N) if position is None else np.clip(position, 0, N - 1)
        place = np.arange(T)
        place[ctx:] = ctx + pos[:n_new]
        for n in range(n_new):
            out[n] &= (place < sinks) | (ctx + pos[n] - place < window)
    return out


def gather(cache, table_row, T, page):
    """[T, heads, D] rows of a cache tensor [pages, page_size, heads, D] in
    float64; rows on pages outside the cache are NaN."""
    pages = cache.shape[0]
    out = torch.full((T, *cache.shape[2:]), math.nan, dtype=torch.float64)
    for t in range(0, T, page):
        p = int(table_row[t // page])
        if 0 <= p < pages:
            n = min(page, T - t)
            out[t:t + n] = cache[p, :n].double()
    return out


def attention_reference(q, k, v, sees, scale):
    """out, lse and the error scales of each output, in float64: q [n, Hq, D],
    k and v [T, Hkv, D], sees [n, T].  What a token does not see is left out
    before any product."""
    n, Hq, D = q.shape
    G = Hq // k.shape[1]
    out = torch.zeros(n, Hq, D, dtype=torch.float64)
    lse = torch.full((n, Hq), -math.inf, dtype=torch.float64)
    mean = torch.zeros(n, Hq, D, dtype=torch.float64)   # sum of w |v| over sum of w
    reach = torch.zeros(n, Hq, dtype=torch.float64)     # largest scale * sum |q k|
    vmax = torch.zeros(n, Hq, dtype=torch.float64)
    q = q.double()
    sees = torch.from_numpy(np.ascontiguousarray(sees))
    for i in range(n):
        at = sees[i].nonzero()[:, 0]
        if not len(at):
            continue
        kk, vv = k[at], v[at]
        for h in range(k.shape[1]):
            z = q[i, h * G:(h + 1) * G] @ kk[:, h].T * scale
            reach[i, h * G:(h + 1) * G] = (q[i, h * G:(h + 1) * G].abs() @ kk[:, h].abs().T
                                           * scale).amax(1)
            m = z.amax(1, keepdim=True)
            w = torch.where(m == -math.inf, 0.0, (z - m).exp())
            s = w.sum(1, keepdim=True)
            some = s > 0
            lse[i, h * G:(h + 1) * G] = torch.where(some, m + s.log(), -math.inf)[:, 0]
            div = torch.where(some, s, 1.0)
            out[i, h * G:(h + 1) * G] = w @ vv[:, h] / div
            mean[i, h * G:(h + 1) * G] = w @ vv[:, h].abs() / div
            vmax[i, h * G:(h + 1) * G] = vv[:, h].abs().max()
    return out, lse, mean, reach, vmax


def attention_tolerance(out, lse, mean, reach, vmax, T, D, dtype):
    """Bounds on |out| and |lse| errors.

    Each weight is off by a factor 1 + d: the score's float32 sum of D products
    (half a step 2^-24 each; twice that for hardware sums that cut instead of
    rounding), its product with scale log2(e) and the exponent (2^-24 of a value
    of up to `reach` log2(e), three roundings), the exponential (2^-22 relative)
    and the rescaling by later maxima (covered by another 2^-21); the float32 sums
    over T keys add T 2^-24 (2^-23 where they are cut).  Numerator and
    denominator are off by that much of sum w |v| and sum w.  16-bit types round
    each weight by half a step (float16 also by half of its smallest step 2^-24,
    of weights that are at most 1, with a sum of at least 1 at the maximum's
    key) and the output by half a step.
    """
    d = (D + 8) * 2.0 ** -23 * reach + 2.0 ** -20 + T * 2.0 ** -23
    half = torch.finfo(DTYPES[dtype]).eps / 2
    tol = (mean + out.abs()) * (d[..., None] + 2.0 ** -22) + out.abs() * half * (1 + 2.0 ** -6)
    if dtype != "f32":
        tol = tol + mean * half * (1 + 2.0 ** -6)
    if dtype == "f16":
        tol = tol + (T * 2.0 ** -25 * vmax + 2.0 ** -25)[..., None]
    lse_tol = d + 2.0 ** -22 * (1 + lse.abs())
    return tol + 1e-30, lse_tol


def check_attention(res, q, k_cache, v_cache, table, ctx, page, dtype, n_new=None, sees=None,
                    position=None, window=0, sinks=0, scale=None, label=""):
    """Compares an AttentionResult (with lse) with the reference, sequence by
    sequence.  Tokens behind n_new are not looked at."""
    q, k_cache, v_cache = q.cpu(), k_cache.cpu(), v_cache.cpu()
    out, lse = res.out.cpu().double(), res.lse.cpu().double()
    B, N, Hq, D = q.shape
    for b in range(B):
        n = N if n_new is None else int(n_new[b])
        if n == 0:
            continue
        c = int(ctx[b])
        T = c + n
        pos = None if position is None else (position[b] if position.ndim == 2 else position)
        m = None if sees is None else (sees[b] if sees.ndim == 3 else sees)
        vis = visible(c, n, N, m, pos, window, sinks)
        good = np.array([0 <= int(table[b, t // page]) < k_cache.shape[0] for t in range(T)], bool)
        vis = vis & good
        k, v = (gather(x, table[b], T, page) for x in (k_cache, v_cache))
        want, want_lse, mean, reach, vmax = attention_reference(
            q[b, :n], k, v, vis, D ** -0.5 if scale is None else scale)
        tol, lse_tol = attention_tolerance(want, want_lse, mean, reach, vmax, T, D, dtype)
        where = f"{label} sequence {b} ctx {c} new {n}"
        empty = want_lse == -math.inf
        assert (lse[b, :n][empty] == -math.inf).all(), where
        assert (out[b, :n][empty] == 0).all(), where
        err = (out[b, :n] - want).abs()
        assert torch.isfinite(out[b, :n]).all(), where
        assert (err <= tol).all(), f"{where}: {(err / tol).max().item():.3g} of the tolerance"
        e = (lse[b, :n] - want_lse).abs()[~empty]
        assert (e <= lse_tol[~empty]).all(), f"{where}: lse off by {e.max().item():.3g}"
