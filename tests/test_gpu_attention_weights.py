"""float16 weights far below a row's largest: many of them together count."""

import math

import pytest
import torch

import speculative_decoding_verification_temp_gb300 as sv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("N,G,D,page", [(1, 4, 128, 16), (4, 8, 64, 16), (12, 5, 64, 16), (20, 6, 128, 32),
                                        (70, 4, 64, 64), (40, 7, 128, 16), (3, 3, 72, 16), (2, 2, 128, 5),
                                        (2, 4, 256, 16)])
def test_a_long_tail_under_one_key(N, G, D, page, first):
    """One key scores 17.375, the others 0: e^-17.375 = 2^-25.07 of the largest each.
    The one key's values are 0, the others' 64.

    Bound: float16 rounds a weight by at most half a step of its value, 2^-11, or by
    half of its smallest step, 2^-25, where the row's largest weight is at least 2^7:
    2^-32 of it, T times, times 64.  The output is rounded by 2^-11 of itself; the
    rest is as in the other tests: (D + 8) 2^-23 of the largest score, T 2^-23 for
    the sums.  (Without the lifted weights the tail is lost: all of the output in the
    kernels of whole rows, a quarter of it where quarters of the lanes share a row.)
    """
    T, B, Hkv, gap, value = 9000, 200, 2, 17.375, 64.0
    pages = -(-(T + N) // page)
    k = torch.zeros(pages, page, Hkv, D, dtype=torch.float16, device="cuda")
    v = torch.full_like(k, value)
    at = 0 if first else T - 1
    k[at // page, at % page, :, 0] = gap
    v[at // page, at % page] = 0.0
    q = torch.zeros(B, N, Hkv * G, D, dtype=torch.float16, device="cuda")
    q[..., 0] = 1.0
    # enough sequences, all on the same pages, that units are whole or nearly so
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None].expand(B, -1)
    ctx = torch.full((B,), T, dtype=torch.int32, device="cuda")
    res = sv.paged_attention(q, k, v, table, ctx, scale=1.0, return_lse=True)
    tail = (T - 1 + 1 + torch.arange(N, dtype=torch.float64)) * math.exp(-gap)
    out = (tail * value / (1 + tail))[None, :, None, None]
    lse = (gap + torch.log1p(tail))[None, :, None]
    small = (D + 8) * 2.0 ** -23 * gap + 2.0 ** -20 + (T + N) * 2.0 ** -23
    tol = (T + N) * 2.0 ** -32 * value + out * (2 * 2.0 ** -11 * (1 + 2.0 ** -6) + 2 * small)
    err = (res.out.cpu().double() - out).abs()
    assert (err <= tol).all(), f"off by {err.max().item():.3g} of {out.max().item():.3g}"
    assert ((res.lse.cpu().double() - lse).abs() <= small + 2.0 ** -22 * (1 + lse)).all()
