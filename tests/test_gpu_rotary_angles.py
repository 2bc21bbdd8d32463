"""Angles of frequencies of any size at any position, against arithmetic on whole numbers."""

from fractions import Fraction

import numpy as np
import pytest
import torch

import speculative_decoding_verification_temp_gb300 as sv

from rows_helpers import rotation_tolerance

pytestmark = pytest.mark.gpu

BITS = 400


def _arctan(x):
    """2^BITS arctan(1 / x), by its series."""
    total, term, n = 0, (1 << BITS) // x, 0
    while term:
        total += (-1) ** n * (term // (2 * n + 1))
        term //= x * x
        n += 1
    return total


PI = Fraction(16 * _arctan(5) - 4 * _arctan(239), 1 << BITS)


def turned(x, position, frequency):
    """x [T, heads, D] float64 turned by position [T]; pairs of halves."""
    half, out = len(frequency), x.clone()
    for t, at in enumerate(position):
        for i, f in enumerate(frequency):
            turns = at * Fraction(f) / (2 * PI)
            angle = float((turns - round(turns)) * 2 * PI)
            c, s = np.cos(angle), np.sin(angle)
            a, b = x[t, :, i], x[t, :, i + half]
            out[t, :, i], out[t, :, i + half] = a * c - b * s, a * s + b * c
    return out


FREQUENCIES = [[1.0, 0.7498942093324559, 6.283185307179586, 100.0], [1000.0, 12345.678, -250.5, 1e6],
               [3.0, -1.0, -1e-3, 2.0 ** -40], [2.0 ** 52 + 1, 1e17, -7e22, 5e-324]]


@pytest.mark.parametrize("frequency", FREQUENCIES, ids=str)
def test_frequencies_of_every_size(frequency):
    position = [2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, 999999937, -123456789, 131071, 1, -1, 0]
    gen = torch.Generator("cuda")
    gen.manual_seed(81)
    x = torch.randn(len(position), 3, 8, generator=gen, device="cuda")
    f = torch.tensor(frequency, dtype=torch.float64, device="cuda")
    got = sv.rotary(x, torch.tensor(position, device="cuda"), f).double().cpu()
    want = turned(x.double().cpu(), position, frequency)
    # a turn is held to 2^-64 and its fraction to 2^-65 a token, 2^-32 turns at most of these
    # positions: nothing next to float32's 2^-25.  Frequencies of 2^53 and more are off by
    # 2^-106 of themselves besides, 2^-29 turns a token at 1e23: only near positions
    tol = rotation_tolerance(x, want, 4, False, "f32")
    if max(map(abs, frequency)) > 2.0 ** 53:
        got, want, tol = got[-3:], want[-3:], tol[-3:]
    assert ((got - want).abs() <= tol).all(), ((got - want).abs() / tol).nan_to_num(0).amax((1, 2))
