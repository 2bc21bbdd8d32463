"""Outputs over 4-bit rows dimension by dimension, each measured by its own values: groups of
small and of large scales, a long tail under one heavy key, a key of huge values that no
token looks at."""

import math

import numpy as np
import pytest
import torch

from cache_helpers import visible
from rows_helpers import four_bits, half_step
from test_gpu_attention_q4 import Setup

pytestmark = pytest.mark.gpu


def check(s, res, only=None, groups=(0, 1, 2, 3), window=0, sinks=0):
    """|out - want| of each output against bounds from the values of its own dimension.

    With weights w (summing to one) of the seen keys, and mean = sum of w (|m| + s n):
    - scores off by d, as in tolerance() of the attention's tests: (mean + |out|) d;
    - weights, and their products with the scales (or, on tensor memory, the values), are
      float16: 2^-11 of each, 2 mean 2^-11; on tensor memory its minimum and the value itself
      are also off by 2^-21 each, half of float16's smallest step for their sixteenth;
    - up to 8 rows, what float16 cannot hold: half of its smallest step, 2^-25, for each key's
      product with code 15 and its product with the minimum, 8 scales at most: 23 2^-25.  The
      key of the largest weight times scale has a weight of 2^6 at least, and either scales
      of 2^-7 and more, or ones of which the largest was brought to [1, 2), the group's own, s, to
      2^-7 or more there too (of groups up to 2^14 apart in all keys, or 2^7 in some):
      T 23 2^-25 2^-6 2^7 s < T 2^-19 s;
    - on tensor memory, weights below 2^-32 of the largest: 2^-32 of every value;
    - the output's own type.
    """
    out = res.out.cpu().double()
    B, N, Hq, D = out.shape
    q = s.q[:B].double().cpu()
    Hkv = s.k.shape[2]
    wide = N * (Hq // Hkv) > 8
    for b in range(B):
        c, T = int(s.ctx[b]), int(s.ctx[b]) + N
        vis = torch.from_numpy(visible(c, N, N, window=window, sinks=sinks))
        slots = [s.slot(b, t) for t in range(T)]
        pages, places = (torch.tensor(x, device="cuda") for x in zip(*slots))
        k, v = ([x.repeat_interleave(D // 4, -1) if x.shape[-1] == 4 else x for x in four_bits(cache[pages, places])]
                for cache in (s.k, s.v))
        keys, size, values = k[2] + k[1] * k[0], v[2].abs() + v[1].abs() * v[0], v[2] + v[1] * v[0]
        for n in (range(N) if only is None else only):
            at = vis[n].nonzero()[:, 0]
            for h in range(Hq):
                g = h // (Hq // Hkv)
                z = keys[at, g] @ q[b, n, h] / math.sqrt(D)
                w = torch.softmax(z, 0)
                want, mean = w @ values[at, g], w @ size[at, g]
                reach = float((keys[at, g].abs() @ q[b, n, h].abs()).max()) / math.sqrt(D)
                top = int((w * v[1][at, g].abs().amax(-1)).argmax())
                d = (D + 16) * 2.0 ** -22 * reach + 2.0 ** -20 + T * 2.0 ** -23
                tol = 2 * mean * 2.0 ** -11 * (1 + 2.0 ** -6) + want.abs() * half_step(s.dtype) * (1 + 2.0 ** -6) + 2.0 ** -25
                if wide:
                    d += reach * 2.0 ** -11 * 1.01
                    tol = tol + 2.0 ** -20 + 2.0 ** -32 * values[at, g].abs().sum(0)
                else:
                    tol = tol + T * 2.0 ** -19 * v[1][at[top], g].abs()
                tol = tol + (mean + want.abs()) * (d + 2.0 ** -22)
                worst = ((out[b, n, h] - want).abs() / tol).view(4, -1)[list(groups)].amax(-1)
                assert (worst <= 1).all(), f"sequence {b} token {n} head {h}: {worst.tolist()} of the tolerance"


def put_groups(cache, scale, low, at=None):
    """Scales and minima [4] of the rows of head dimension groups, NaN rows staying NaN."""
    D = (cache.shape[-1] - 16) * 2
    rows = cache if at is None else cache[at[0], at[1]]
    pair = rows[..., D // 2:].contiguous().view(torch.float16).unflatten(-1, (4, 2))
    new = torch.stack([torch.as_tensor(scale), torch.as_tensor(low)], -1).cuda().half().expand_as(pair)
    pair = torch.where(torch.isnan(pair), pair, new).flatten(-2).contiguous().view(torch.uint8)
    if at is None:
        cache[..., D // 2:] = pair
    else:
        cache[at[0], at[1], :, D // 2:] = pair


SIZES = [(1, 4, 1, 64), (1, 4, 1, 128), (2, 4, 1, 128), (1, 8, 1, 64), (16, 4, 1, 128), (40, 4, 1, 64)]
GROUPS = {"small": [2.0 ** -11, 1.3 * 2.0 ** -11, 1.7 * 2.0 ** -11, 1.1 * 2.0 ** -12], "smallest": [1.7 * 2.0 ** -14] * 4,
          "usual": [0.21, 0.34, 0.13, 0.55], "uneven": [1.3 * 2.0 ** -11, 1.7 * 2.0 ** -7, 0.15, 3.0],
          "large": [3000.0, 4000.0, 2500.0, 4090.0], "around one": [0.9, 1.1, 1.9, 2.1], "zeros": [0.0, 0.0, 0.3, 0.0]}


@pytest.mark.parametrize("groups", GROUPS)
@pytest.mark.parametrize("N,Hq,Hkv,D", SIZES)
def test_each_group_by_its_own_values(N, Hq, Hkv, D, groups):
    s = Setup(51, [50, 0, 400], N, Hq, Hkv, D, 16, "f16")
    scale = torch.tensor(GROUPS[groups])
    put_groups(s.v, scale, -7.0 * scale)
    check(s, s.call(), only=sorted({0, N - 1}))


@pytest.mark.parametrize("N,Hq,Hkv,D", SIZES)
def test_scales_that_differ_from_key_to_key(N, Hq, Hkv, D):
    s = Setup(52, [50, 0, 400], N, Hq, Hkv, D, 16, "f16")
    gen = torch.Generator("cuda")
    gen.manual_seed(52)
    pair = s.v[..., D // 2:].contiguous().view(torch.float16).unflatten(-1, (4, 2)).float()
    by = torch.exp2(torch.rand(pair.shape[:3], generator=gen, device="cuda") * 22 - 11)[..., None, None]
    pair[..., 1] = 2.0 * pair[..., 0]
    s.v[..., D // 2:] = (pair * by).half().flatten(-2).view(torch.uint8)
    check(s, s.call(), only=sorted({0, N - 1}))


@pytest.mark.parametrize("unrelated", [None, 4096.0, 2.0 ** -13])
@pytest.mark.parametrize("groups", ["small", "usual", "uneven", "large"])
@pytest.mark.parametrize("N,Hq,Hkv,D", SIZES)
def test_a_long_tail_under_one_heavy_key(N, Hq, Hkv, D, groups, unrelated):
    """9000 keys, alike, 9 nats below one other, together weigh 1.1 of it; a further key of
    other scales lies 20 nats below them.  2048 sequences on the same pages: none is cut into
    pieces so short that the key is alone in its own."""
    s = Setup(53, [9000], N, Hq, Hkv, D, 64, "f16")
    s.q, s.table, s.ctx = s.q.repeat(2048, 1, 1, 1), s.table.repeat(2048, 0), s.ctx.repeat(2048)
    s.q.fill_(1.0)
    s.k[..., :D // 2] = 0
    s.v[..., :D // 2] = 0xFF
    put_groups(s.k, [0.0] * 4, [0.0] * 4)
    put_groups(s.v, GROUPS[groups], [0.0] * 4)
    p, i = s.slot(0, 11)
    put_groups(s.k, [0.0] * 4, [9.0 / math.sqrt(D)] * 4, (p, i))
    s.v[p, i, :, :D // 2] = 0x11
    if unrelated is not None:
        p, i = s.slot(0, 5000)
        put_groups(s.k, [0.0] * 4, [-20.0 / math.sqrt(D)] * 4, (p, i))
        put_groups(s.v, [unrelated] * 4, [0.0] * 4, (p, i))
    res = s.call()
    for b in (0, 1000):  # at its own place of the workers' runs
        one = type(res)(res.out[b:b + 1], None, None)
        check(s, one, only=[0])


@pytest.mark.parametrize("places", [range(32), range(32, 64), range(0, 400, 3), range(40, 400)], ids=str)
@pytest.mark.parametrize("N,Hq,Hkv,D", SIZES[:4])
def test_groups_that_change_along_a_sequence(N, Hq, Hkv, D, places):
    """Keys whose groups lie apart, in other tiles than, or among, keys whose groups are alike."""
    s = Setup(55, [400], N, Hq, Hkv, D, 16, "f16")
    scale = torch.tensor(GROUPS["usual"])
    put_groups(s.v, scale, -7.0 * scale)
    scale = torch.tensor([0.002, 0.02, 0.1, 0.25])
    for t in places:
        put_groups(s.v, scale, -7.0 * scale, s.slot(0, t))
    check(s, s.call())
    check(s, s.call(window=90, sinks=5), window=90, sinks=5)


@pytest.mark.parametrize("N,Hq,Hkv,D", SIZES[:4])
def test_large_minima_beside_small_scales(N, Hq, Hkv, D):
    s = Setup(54, [50, 0, 400], N, Hq, Hkv, D, 16, "f16")
    put_groups(s.v, [2.0 ** -11, 0.3, 2.0 ** -9, 2.0 ** -14], [0.0, -60000.0, 1.0, 40000.0])
    s.check(s.call())
    check(s, s.call(), groups=(0,))
