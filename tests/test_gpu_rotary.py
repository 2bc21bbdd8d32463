"""Rotation by position, and appending with it, against plain 64-bit computations."""

import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_temp_gb300 as sv

from cache_helpers import make_pages
from rows_helpers import (DTYPES, check_four_bits, half_step, rotated, rotation_tolerance, stands_for)

pytestmark = pytest.mark.gpu


def normal(seed, shape, dtype):
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").to(DTYPES[dtype])


def check(got, x, position, f, dtype, interleaved=False, amplitude=1.0, inverse=False):
    want = rotated(x, position, f, interleaved, amplitude, inverse)
    tol = rotation_tolerance(x, want, f.numel(), interleaved, dtype, amplitude)
    err = (got.double().cpu() - want).abs()
    assert got.dtype == DTYPES[dtype] and (err <= tol).all(), (err / tol).nan_to_num(0).max()
    rest = 2 * f.numel()
    assert torch.equal(got[..., rest:], x[..., rest:])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,H,D,dim", [(1, 1, 64, 64), (1, 40, 128, 128), (7, 3, 128, 64), (300, 5, 80, 40),
                                       (33, 2, 96, 48), (5, 1, 256, 256), (2, 3, 10, 6), (3, 2, 2, 2),
                                       (1000, 1, 64, 32), (4, 2, 600, 512), (9, 17, 40, 30)])
def test_rotary(T, H, D, dim, dtype, interleaved):
    x = normal(T + D, (T, H, D), dtype)
    f = sv.rotary_frequency(dim).frequency
    position = torch.from_numpy(np.random.default_rng(T).integers(0, 131072, T)).cuda()
    check(sv.rotary(x, position, f, interleaved=interleaved), x, position, f, dtype, interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_and_negative_positions(interleaved):
    x = normal(3, (6, 2, 64), "f32")
    f = sv.rotary_frequency(64, base=500000.0).frequency
    position = torch.tensor([2 ** 31 - 1, 2 ** 30 + 1, 2 ** 24 + 1, -1, -2 ** 31, 0], device="cuda")
    # longdouble turns of 2^31 tokens are off by 2^-63 2^31 or less
    check(sv.rotary(x, position, f, interleaved=interleaved), x, position, f, "f32", interleaved)
    assert torch.equal(sv.rotary(x, position, f, interleaved=interleaved)[5], x[5])


def test_amplitude_inverse_and_gradient():
    x = normal(4, (9, 4, 128), "f32")
    f, a = sv.rotary_frequency(128, scaling="index", factor=16.0)
    position = torch.arange(100, 109, device="cuda")
    assert a > 1.2
    y = sv.rotary(x, position, f, amplitude=a)
    check(y, x, position, f, "f32", amplitude=a)
    check(sv.rotary(x, position, f, amplitude=-0.5, inverse=True), x, position, f, "f32", amplitude=-0.5,
          inverse=True)
    # the rotation is orthogonal: its inverse is its gradient
    back = sv.rotary(sv.rotary(x, position, f), position, f, inverse=True)
    # two rotations of 2^-21 (|a| + |b|) and two roundings
    assert (back - x).abs().max() <= 2.0 ** -19 * 2 * x.abs().max()
    g = normal(5, x.shape, "f32")
    left = (sv.rotary(x, position, f).double() * g).sum()
    right = (x.double() * sv.rotary(g, position, f, inverse=True)).sum()
    assert (left - right).abs() <= 2.0 ** -19 * (x.double().abs() * g.abs().amax()).sum()


def test_shapes_strides_and_places():
    f = sv.rotary_frequency(32).frequency
    fused = normal(6, (3, 5, 12, 64), "bf16")
    position = torch.arange(15, device="cuda").reshape(3, 5) * 7
    q = fused[:, :, 2:8]
    want = sv.rotary(q.contiguous(), position, f)
    assert torch.equal(sv.rotary(q, position, f), want)
    # one position for all sequences; a token; no token; transposed heads (copied)
    assert torch.equal(sv.rotary(q, position[1], f)[1], want[1])
    assert torch.equal(sv.rotary(q[1, 2], position[1, 2], f), want[1, 2])
    assert sv.rotary(q[:, :0], position[:, :0], f).shape == (3, 0, 6, 64)
    assert torch.equal(sv.rotary(q.transpose(2, 3).contiguous().transpose(2, 3), position, f), want)
    # expanded heads
    one = q[:, :, :1].expand(3, 5, 4, 64)
    assert torch.equal(sv.rotary(one, position, f), want[:, :, :1].expand(3, 5, 4, 64))
    # rows at odd offsets take the scalar path
    flat = torch.empty(q.numel() + 1, dtype=q.dtype, device="cuda")
    odd = flat[1:].view(q.shape)
    odd.copy_(q)
    assert torch.equal(sv.rotary(odd, position, f), want)
    # in place, the other heads stay
    before = fused.clone()
    assert sv.rotary(q, position, f, out=q) is q
    assert torch.equal(q, want)
    assert torch.equal(fused[:, :, :2], before[:, :, :2]) and torch.equal(fused[:, :, 8:], before[:, :, 8:])
    assert torch.equal(sv.rotary(odd, position, f, out=odd), want)


@pytest.mark.parametrize("scaling", [None, "linear", "base", "turns", "index"])
def test_frequencies(scaling):
    dim, factor, context = 64, 8.0, 2048
    f, a = sv.rotary_frequency(dim, 10000.0, scaling, factor, context, 1.0, 16.0, device="cpu")
    for i in range(dim // 2):
        plain = 10000.0 ** (-2 * i / dim)
        turns = context * plain / (2 * math.pi)
        if scaling is None:
            want = plain
        elif scaling == "linear":
            want = plain / factor
        elif scaling == "base":
            want = (10000.0 * factor ** (dim / (dim - 2))) ** (-2 * i / dim)
        else:
            if turns <= 0.9:
                want = plain / factor
            elif turns >= 18:
                want = plain
            else:
                assert plain / factor <= f[i] <= plain
                continue
        assert abs(float(f[i]) - want) <= 1e-14 * plain + (1e-3 * plain if scaling == "index" else 0)
    if scaling == "base":
        # the longest wave is factor times longer
        assert abs(float(f[-1]) * factor - 10000.0 ** (-(dim - 2) / dim)) < 1e-12
    assert a == (0.1 * math.log(factor) + 1 if scaling == "index" else 1.0)


def test_frequencies_that_are_not_finite():
    x = normal(7, (3, 2, 8), "f32")
    f = torch.tensor([1.0, math.nan, math.inf, 0.0], dtype=torch.float64, device="cuda")
    y = sv.rotary(x, torch.arange(3, device="cuda"), f)
    for i in (1, 2):
        assert torch.isnan(y[..., [i, i + 4]]).all()
    assert torch.isfinite(y[..., [0, 4, 3, 7]]).all() and torch.equal(y[..., [3, 7]], x[..., [3, 7]])


# ---------------------------------------------------------------------------
# appending
# ---------------------------------------------------------------------------


class Append:
    def __init__(self, seed, ctx, N, Hq, Hkv, D, page, dtype, four, n_new=None, layers=None, layout="hnd",
                 new_dtype=None):
        rng = np.random.default_rng(seed)
        self.ctx, self.N, self.page, self.four, self.dtype = np.asarray(ctx), N, page, four, dtype
        B = len(ctx)
        self.n_new = None if n_new is None else np.asarray(n_new, np.int32)
        count = np.full(B, N) if n_new is None else np.clip(n_new, 0, N)
        self.count = count
        self.table, pages = make_pages(rng, self.ctx + count, page)
        lead = () if layers is None else (layers,)
        self.lead = lead
        width = D // 2 + 16 if four else D
        gen = torch.Generator("cuda")
        gen.manual_seed(seed)

        def cache():
            shape = (*lead, pages, Hkv, page, width) if layout == "hnd" else (*lead, pages, page, Hkv, width)
            if four:
                x = torch.randint(0, 256, shape, generator=gen, device="cuda", dtype=torch.uint8)
            else:
                x = torch.randn(shape, generator=gen, device="cuda").to(DTYPES[dtype])
            return x.transpose(-3, -2) if layout == "hnd" else x

        self.k, self.v = cache(), cache()
        self.q = normal(seed + 1, (*lead, B, N, Hq, D), dtype)
        self.k_new = normal(seed + 2, (*lead, B, N, Hkv, D), dtype) * 2 + 0.5
        self.v_new = normal(seed + 3, (*lead, B, N, Hkv, D), dtype)
        self.dev = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()
        self.args = (self.dev(self.table), self.dev(self.ctx.astype(np.int32)))

    def slot(self, b, t):
        return int(self.table[b, t // self.page]), t % self.page

    def check_caches(self, before, f, place, interleaved, amplitude=1.0):
        """place [B, N]: positions."""
        k, v = self.k.clone(), self.v.clone()
        for b in range(len(self.ctx)):
            n = int(self.count[b])
            if n == 0:
                continue
            pos = torch.as_tensor(place[b][:n])
            k_new = self.k_new[..., b, :n, :, :].reshape(-1, n, *self.k_new.shape[-2:])
            key = rotated(k_new, pos.expand(k_new.shape[0], n), f, interleaved, amplitude)
            tol = rotation_tolerance(k_new, key, f.numel(), interleaved, self.dtype, amplitude)
            for i in range(n):
                p, t = self.slot(b, int(self.ctx[b]) + i)
                at = (Ellipsis, p, t, slice(None), slice(None))
                got_k, got_v = (x[at].reshape(-1, *x.shape[-2:]) for x in (k, v))
                want_v = self.v_new[..., b, i, :, :].reshape(-1, *self.v_new.shape[-2:])
                if self.four:
                    check_four_bits(got_k, key[:, i], tol[:, i])
                    check_four_bits(got_v, want_v)
                else:
                    assert ((got_k.double().cpu() - key[:, i]).abs() <= tol[:, i]).all()
                    assert torch.equal(got_v, want_v)
                k[at] = before[0][at]
                v[at] = before[1][at]
        # nothing else was written
        assert torch.equal(k, before[0]) and torch.equal(v, before[1])


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("dtype,Hq,Hkv,D,dim,page,interleaved", [
    ("bf16", 8, 2, 128, 128, 16, False), ("f16", 4, 4, 64, 64, 8, True), ("f32", 3, 3, 64, 32, 5, False),
    ("bf16", 7, 1, 128, 64, 64, True), ("bf16", 2, 1, 64, 24, 1, False), ("f16", 5, 5, 128, 6, 16, True),
    ("f32", 6, 2, 128, 128, 16, True)])
def test_append(four, dtype, Hq, Hkv, D, dim, page, interleaved):
    n_new = [3, 0, 5, 1, 5]
    s = Append(D + dim, [0, 40, 15, 16, 63], 5, Hq, Hkv, D, page, dtype, four, n_new=n_new)
    f = sv.rotary_frequency(dim).frequency
    before = (s.k.clone(), s.v.clone())
    out = torch.full_like(s.q, 7.0)
    r = sv.cache_append_rotary(s.k_new, s.v_new, s.k, s.v, *s.args, f, q=s.q, out=out, num_new=s.dev(s.n_new),
                               interleaved=interleaved, return_flags=True)
    assert r.q is out and not r.flags.any()
    place = s.ctx[:, None] + np.arange(5)
    s.check_caches(before, f, place, interleaved)
    for b, n in enumerate(n_new):
        assert (out[b, n:] == 7.0).all()
        check(out[b, :n], s.q[b, :n], torch.as_tensor(place[b, :n]), f, dtype, interleaved)
    # reading gives what the rows stand for, and zeros behind num
    got = sv.cache_read(s.k, s.v, *s.args, 5, num=s.dev(s.n_new), dtype=DTYPES[dtype], return_flags=True)
    assert not got.flags.any()
    for b, n in enumerate(n_new):
        for x, y in ((got.k, s.k), (got.v, s.v)):
            assert (x[b, n:] == 0).all()
            for i in range(n):
                row = y[s.slot(b, int(s.ctx[b]) + i)]
                if four:
                    want = stands_for(row)
                    # a float32 rounding and one to the type
                    assert ((x[b, i].double().cpu() - want).abs() <= want.abs() * (half_step(dtype) + 2.0 ** -23) + 2.0 ** -25).all()
                else:
                    assert torch.equal(x[b, i], row)


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
def test_trees_layers_and_layouts(four, layout):
    s = Append(11, [5, 130, 0], 12, 4, 2, 64, 16, "bf16", four, layers=3, layout=layout)
    parent = torch.tensor([[-1, 0, 0, 1, 1, 2, 2, 3, 4, 4, 7, 0]] * 3, device="cuda", dtype=torch.int32)
    depth = sv.tree_mask(parent, 12).position
    f = sv.rotary_frequency(64).frequency
    before = (s.k.clone(), s.v.clone())
    r = sv.cache_append_rotary(s.k_new, s.v_new, s.k, s.v, *s.args, f, q=s.q, position=depth)
    place = s.ctx[:, None] + depth.cpu().numpy()
    s.check_caches(before, f, place, False)
    assert r.flags is None
    for layer in range(3):
        check(r.q[layer], s.q[layer], torch.as_tensor(place), f, "bf16")
    # one tree for all, positions outside [0, N) clamped, and no queries
    k, v = s.k.clone(), s.v.clone()
    one = depth[0].clone()
    one[0], one[11] = -3, 99
    r = sv.cache_append_rotary(s.k_new, s.v_new, s.k, s.v, *s.args, f, position=one)
    assert r.q is None and torch.equal(s.v, v)
    moved = sv.cache_read(s.k, s.v, *s.args, 12).k
    there = sv.cache_read(k, v, *s.args, 12).k
    assert torch.equal(moved[:, :, :11], there[:, :, :11]) and not torch.equal(moved[:, :, 11], there[:, :, 11])
    again = sv.rotary(s.k_new[0, :, 11], s.args[1] + 11, f)
    if not four:
        assert torch.equal(moved[0, :, 11], again)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_plain_append_into_four_bits(dtype):
    s = Append(12, [0, 33], 70, 1, 3, 128, 16, dtype, True)
    before = (s.k.clone(), s.v.clone())
    assert sv.cache_append(s.k_new, s.v_new, s.k, s.v, *s.args) is None
    f = torch.zeros(1, dtype=torch.float64, device="cuda")
    s.check_caches(before, f, s.ctx[:, None] + np.arange(70), False)


def test_extreme_values_in_four_bits():
    s = Append(13, [0], 6, 1, 1, 64, 8, "f32", True)
    x = s.k_new[0, :, 0]
    x[0] = 5.0                     # constant: scale 0
    x[1, :16] = 1e30               # beyond the limit
    x[1, 16:32] = torch.linspace(-1e30, 1e30, 16)
    x[2, :16] = math.nan
    x[2, 20] = math.inf
    x[2, 40] = -math.inf
    x[3] = torch.linspace(0, 1e-9, 64)
    x[4] = 1000.0 + torch.rand(64, device="cuda")
    x[5] = 0.0
    sv.cache_append(s.k_new, s.v_new, s.k, s.v, *s.args)
    rows = torch.stack([s.k[s.slot(0, t)][0] for t in range(6)])
    for t in (0, 1, 3, 4, 5):
        check_four_bits(rows[t], x[t])
    got = sv.cache_read(s.k, s.v, *s.args, 6, dtype=torch.float32).k[0, :, 0]
    assert torch.isnan(got[2, :48]).all() and torch.isfinite(got[2, 48:]).all()
    assert torch.isfinite(got[[0, 1, 3, 4, 5]]).all()
    assert (got[0] == 5.0).all() and (got[1, :16] == 61440.0).all() and (got[5] == 0).all()


def test_flags_and_what_is_left_alone():
    f = sv.rotary_frequency(64).frequency
    for four in (False, True):
        s = Append(14, [10, 20, 30, 3], 4, 2, 2, 64, 16, "bf16", four)
        before = (s.k.clone(), s.v.clone())
        table = s.args[0].clone()
        table[1] = 10 ** 6
        ctx = s.args[1].clone()
        ctx[2] = 10 ** 6
        ctx[3] = -1
        num = torch.tensor([2, 4, 4, 9], device="cuda")
        r = sv.cache_append_rotary(s.k_new, s.v_new, s.k, s.v, table, ctx, f, q=s.q, num_new=num, return_flags=True)
        assert r.flags.tolist() == [0, sv.FLAG_BAD_PAGE, sv.FLAG_BAD_LENGTH, sv.FLAG_BAD_LENGTH]
        for x, y in zip((s.k, s.v), before):
            changed = (x != y).flatten(2).any(-1).nonzero().tolist()
            assert sorted(changed) == sorted(list(s.slot(0, 10 + i)) for i in range(2))
        check(r.q[1], s.q[1], 20 + torch.arange(4), f, "bf16")
        got = sv.cache_read(s.k, s.v, table, ctx, 4, return_flags=True)
        assert got.flags.tolist() == [0, sv.FLAG_BAD_PAGE, sv.FLAG_BAD_LENGTH, sv.FLAG_BAD_LENGTH]
        assert (got.k[1:] == 0).all() and (got.v[1:] == 0).all()


def test_queries_in_place_of_a_fused_projection():
    s = Append(15, [7, 0], 3, 4, 2, 128, 16, "bf16", True)
    f = sv.rotary_frequency(128).frequency
    fused = torch.cat([s.q, s.k_new, s.v_new], 2)
    q, k, v = fused.split([4, 2, 2], 2)
    want = sv.cache_append_rotary(s.k_new, s.v_new, s.k, s.v, *s.args, f, q=s.q).q
    rows = (s.k.clone(), s.v.clone())
    s.k.zero_(), s.v.zero_()
    assert sv.cache_append_rotary(k, v, s.k, s.v, *s.args, f, q=q, out=q).q is q
    assert torch.equal(q, want) and torch.equal(k, s.k_new)
    for b in range(2):
        for i in range(3):
            at = s.slot(b, int(s.ctx[b]) + i)
            assert torch.equal(s.k[at], rows[0][at]) and torch.equal(s.v[at], rows[1][at])


def test_another_stream_and_a_captured_graph():
    s = Append(16, [7, 100], 3, 4, 2, 64, 16, "bf16", True)
    f = sv.rotary_frequency(64).frequency
    out = torch.empty_like(s.q)
    call = lambda: sv.cache_append_rotary(s.k_new, s.v_new, s.k, s.v, *s.args, f, q=s.q, out=out)  # noqa: E731
    call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
            read = sv.cache_read(s.k, s.v, *s.args, 3)
    torch.cuda.synchronize()
    for seed in (1, 2):
        s.k_new.copy_(normal(seed, s.k_new.shape, "bf16"))
        s.q.copy_(normal(seed + 5, s.q.shape, "bf16"))
        s.args[1].copy_(torch.tensor([7 + seed, 90], device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = read.k.clone(), out.clone()
        call()
        assert torch.equal(sv.cache_read(s.k, s.v, *s.args, 3).k, got[0]) and torch.equal(out, got[1])
        check(out, s.q, s.args[1].cpu()[:, None] + torch.arange(3), f, "bf16")


def test_long_batches_cross_the_batches_of_tokens():
    s = Append(17, list(range(0, 900, 9)), 31, 3, 1, 64, 16, "bf16", False)
    f = sv.rotary_frequency(64).frequency
    r = sv.cache_append_rotary(s.k_new, s.v_new, s.k, s.v, *s.args, f, q=s.q)
    place = torch.as_tensor(s.ctx[:, None] + np.arange(31))
    check(r.q, s.q, place, f, "bf16")
    got = sv.cache_read(s.k, s.v, *s.args, 31)
    check(got.k, s.k_new, place, f, "bf16")
    assert torch.equal(got.v, s.v_new)


def test_compaction_and_forks_move_four_bit_rows():
    s = Append(18, [21, 9], 8, 1, 2, 64, 8, "bf16", True, layers=2)
    sv.cache_append(s.k_new, s.v_new, s.k, s.v, *s.args)
    path = torch.tensor([[0, 2, 5, -1], [0, 7, -1, -1]], device="cuda", dtype=torch.int32)
    rows = sv.cache_read(s.k, s.v, *s.args, 8)
    r = sv.cache_compact(s.k, s.v, *s.args, path, torch.tensor([2, 1], device="cuda"))
    assert r.context_len.tolist() == [24, 11] and not r.flags.any()
    now = sv.cache_read(s.k, s.v, *s.args, 3)
    assert torch.equal(now.k[:, 0], rows.k[:, 0, [0, 2, 5]]) and torch.equal(now.v[:, 1, :2], rows.v[:, 1, [0, 7]])
    # a fork shares full pages and copies the last one
    pool = sv.page_pool(3, 6, 12)
    k, v = sv.cache_4bit(12, 8, 2, 64, num_layers=2)
    ctx = torch.tensor([19, 0, 0], dtype=torch.int32, device="cuda")
    assert not sv.cache_resize(pool, ctx, 8).any()
    new = normal(1, (2, 3, 19, 2, 64), "bf16")
    zero = torch.zeros(3, dtype=torch.int32, device="cuda")
    sv.cache_append(new, -new, k, v, pool.page_table, zero, num_new=ctx)
    flags = sv.cache_fork(pool, k, v, ctx, torch.tensor([0], device="cuda"), torch.tensor([2], device="cuda"))
    assert not flags.any() and ctx.tolist() == [19, 0, 19]
    got = sv.cache_read(k, v, pool.page_table, zero, 19, num=ctx)
    assert torch.equal(got.k[:, 0], got.k[:, 2]) and torch.equal(got.v[:, 0], got.v[:, 2])
    # values of normal rows lie within half a step of what came in: 4.5 / 15 / 2 and roundings
    assert (got.k[:, 0] - new[:, 0]).abs().max() < 0.4 and (got.k[:, 1] == 0).all()


def test_no_query_heads():
    """Queries without heads: the rows are appended all the same."""
    k, v = sv.cache_4bit(4, 16, 2, 64)
    new = torch.randn(1, 3, 2, 64, device="cuda", dtype=torch.float16)
    f, _ = sv.rotary_frequency(64)
    table = torch.arange(4, device="cuda", dtype=torch.int32)[None]
    ctx = torch.tensor([5], device="cuda", dtype=torch.int32)
    res = sv.cache_append_rotary(new, new, k, v, table, ctx, f, q=new[:, :, :0])
    assert res.q.shape == (1, 3, 0, 64)
    want = sv.rotary(new, ctx[:, None] + torch.arange(3, device="cuda"), f)
    got = sv.cache_read(k, v, table, ctx, 3, dtype=torch.float16)
    for x, y in ((got.k, want), (got.v, new)):
        span = (y.float().amax() - y.float().amin()).item()
        assert ((x.float() - y.float()).abs() <= span / 30 * 1.1 + 1e-2).all() and x.abs().sum() > 0


@pytest.mark.parametrize("four", [False, True])
def test_offsets_beyond_32_bits(four):
    """Pages more than 2^32 bytes into the cache: append, read, compaction and attention."""
    page, heads, D, pages = 16, 8, 128, 160_000 if not four else 450_000
    if four:
        k, v = (torch.empty(pages, heads, page, 80, dtype=torch.uint8, device="cuda").transpose(1, 2) for _ in "kv")
    else:
        k, v = (torch.empty(pages, page, heads, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    assert k.numel() * k.element_size() > 2 ** 32
    gen = torch.Generator("cuda")
    gen.manual_seed(5)
    new = lambda n: torch.randn(2, n, heads, D, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    table = torch.tensor([[pages - 1, 3, pages - 7], [pages - 2, pages - 5, 0]], dtype=torch.int32, device="cuda")
    small = torch.tensor([[0, 1, 2], [3, 4, 5]], dtype=torch.int32, device="cuda")
    ks, vs = sv.cache_4bit(6, page, heads, D) if four else (k[:6].clone().zero_(), v[:6].clone().zero_())
    f, _ = sv.rotary_frequency(D)
    ctx = torch.tensor([0, 0], dtype=torch.int32, device="cuda")
    rows, more = (new(36), new(36)), (new(5), new(5))
    at = torch.tensor([36, 36], dtype=torch.int32, device="cuda")
    path = torch.tensor([[0, 2, 4], [0, 3, -1]], dtype=torch.int32, device="cuda")
    taken = torch.tensor([2, 1], dtype=torch.int32, device="cuda")
    q = torch.randn(2, 5, 32, D, generator=gen, device="cuda").to(torch.bfloat16)
    got = []
    for kc, vc, t in ((k, v, table), (ks, vs, small)):
        out = []
        sv.cache_append_rotary(*rows, kc, vc, t, ctx, f)
        sv.cache_append_rotary(*more, kc, vc, t, at, f)
        out += sv.paged_attention(q, kc, vc, t, at, return_lse=True)[:2]
        out += sv.paged_attention(q[:, :1], kc, vc, t, at, return_lse=True)[:2]
        sv.cache_compact(kc, vc, t, at, path, taken)
        out += sv.cache_read(kc, vc, t, ctx, 39)[:2]
        got.append(out)
    for x, y in zip(*got):
        assert torch.equal(x, y)
