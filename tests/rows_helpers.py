"""Plain references of the rotation and of 4-bit rows, in 64 bits, from their definitions."""

import math

import numpy as np
import torch

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def half_step(dtype):
    return torch.finfo(DTYPES[dtype]).eps / 2


def rotated(x, position, frequency, interleaved=False, amplitude=1.0, inverse=False):
    """x [..., heads, D] turned by position [...], value by value, in float64; the
    angles in the widest type that numpy has, wrapped before sine and cosine."""
    x = x.double().cpu()
    pos = np.asarray(position.cpu(), dtype=np.int64)
    f = frequency.cpu().numpy()
    out = x.clone()
    half = len(f)
    # exact: position * frequency as whole numbers of 2^-1100
    for p, freq in enumerate(f):
        num, den = float(freq).as_integer_ratio()
        two_pi = 2 * np.longdouble(math.pi) + np.longdouble(2.4492935982947064e-16)
        turns = (np.longdouble(1) * num / den / two_pi) * pos.astype(np.longdouble)
        angle = ((turns - np.rint(turns)) * two_pi).astype(np.float64)
        c = torch.from_numpy(np.asarray(np.cos(angle)))[..., None] * amplitude
        s = torch.from_numpy(np.asarray(np.sin(angle)))[..., None] * amplitude * (-1 if inverse else 1)
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + half)
        a, b = x[..., i], x[..., j]
        out[..., i], out[..., j] = a * c - b * s, a * s + b * c
    return out


def rotation_tolerance(x, want, pairs, interleaved, dtype, amplitude=1.0):
    """Bounds on the error of rotated values: the angle in float32 half turns is off by
    2^-25 of itself, pi 2^-25 radians at most, sine and cosine by two steps of 2^-24
    (2^-22 covers both), their product with the amplitude by 2^-24 of itself, two
    products and a sum by 2^-24 of |a| + |b| each: 2^-21 (|a| + |b|) amplitude in all;
    the result is rounded to its type."""
    x = x.double().cpu().abs()
    y = torch.zeros_like(x)
    if interleaved:
        s = x[..., 0:2 * pairs:2] + x[..., 1:2 * pairs:2]
        y[..., 0:2 * pairs:2] = y[..., 1:2 * pairs:2] = s
    else:
        s = x[..., :pairs] + x[..., pairs:2 * pairs]
        y[..., :pairs] = y[..., pairs:2 * pairs] = s
    tiny = 2.0 ** -25 if dtype == "f16" else 0.0  # half of float16's smallest step
    return y * abs(amplitude) * 2.0 ** -21 + want.abs() * half_step(dtype) * (1 + 2.0 ** -8) + tiny


def four_bits(rows):
    """codes [..., D], scale and minimum [..., 4] (float64) of 4-bit rows, bit by bit."""
    rows = rows.cpu().numpy()
    D = (rows.shape[-1] - 16) * 2
    words = np.ascontiguousarray(rows[..., :D // 2]).view("<u4").astype(np.int64)
    codes = np.zeros((*rows.shape[:-1], D))
    for i in range(4):
        codes[..., 2 * i::8] = words >> (4 * i) & 15
        codes[..., 2 * i + 1::8] = words >> (16 + 4 * i) & 15
    pairs = np.ascontiguousarray(rows[..., D // 2:]).view("<f2").astype(np.float64)
    return [torch.from_numpy(x.copy()) for x in (codes, pairs[..., 0::2], pairs[..., 1::2])]


def stands_for(rows):
    """The values of 4-bit rows."""
    codes, scale, low = four_bits(rows)
    each = codes.shape[-1] // 4
    return low.repeat_interleave(each, -1) + scale.repeat_interleave(each, -1) * codes


def check_four_bits(rows, x, slack=0.0):
    """Whether 4-bit rows are those of x (float64), each known to within `slack`
    [same shape] or 0: minimum and scale are float16's nearest, codes the nearest."""
    codes, scale, low = four_bits(rows)
    x = x.double().cpu().clamp(-61440, 61440)
    slack = torch.zeros_like(x) + slack
    each = x.shape[-1] // 4
    g, sl = x.unflatten(-1, (4, each)), slack.unflatten(-1, (4, each)).amax(-1)
    lo, hi = g.amin(-1), g.amax(-1)
    half = 2.0 ** -11  # float16's half step, relative
    # minimum: half a step of float16 (2^-25 where it is below float16's normal values)
    assert ((low - lo).abs() <= sl + lo.abs() * half * (1 + 2.0 ** -8) + 2.0 ** -25).all()
    # scale: a float32 difference, a product with 1/15 (three roundings of 2^-24), a float16
    want = (hi - low) / 15
    assert ((scale - want).abs() <= sl / 15 * 1.01 + want.abs() * (half + 2.0 ** -21) * (1 + 2.0 ** -8) + 2.0 ** -25).all()
    # codes: the nearest of those that there are, up to the roundings of (x - m) (1 / s)
    s, m = scale.repeat_interleave(each, -1), low.repeat_interleave(each, -1)
    at = torch.where(s == 0, 0.0, (x - m) / torch.where(s == 0, 1.0, s)).clamp(0, 15)
    off = torch.where(s == 0, 0.0, slack / torch.where(s == 0, 1.0, s))
    assert ((codes - at).abs() <= 0.5 + off + 2.0 ** -19).all()
    assert (codes == codes.round()).all()
