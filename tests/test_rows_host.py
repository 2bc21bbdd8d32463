"""Host checks of the rotation and of the 4-bit cache: refused calls launch nothing.
No GPU; the pointers below are never dereferenced."""

import ctypes

import pytest
import torch

import speculative_decoding_verification_temp_gb300 as sv
from speculative_decoding_verification_temp_gb300 import _abi
from speculative_decoding_verification_temp_gb300 import build as build_mod

OK, INV, UNS = _abi.SPEC_OK, _abi.SPEC_ERR_INVALID_ARG, _abi.SPEC_ERR_UNSUPPORTED
F32, BF16, F16, Q4 = _abi.SPEC_F32, _abi.SPEC_BF16, _abi.SPEC_F16, _abi.SPEC_Q4
P = 0x10000
FAR = P << 8


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return _abi.load()


def cache(**kw):
    """A 4-bit cache; strides in bytes."""
    page, heads, D, pages, layers = 16, 2, 64, 10, 1
    row = D // 2 + 16
    d = dict(k=P, v=P, dtype=Q4, num_layers=layers, num_pages=pages, page_size=page, num_heads=heads, head_dim=D)
    for x in "kv":
        d |= {f"{x}_layer_stride": pages * page * heads * row, f"{x}_page_stride": page * heads * row,
              f"{x}_token_stride": heads * row, f"{x}_head_stride": row}
    return _abi.spec_kv_cache(**(d | kw))


def table(**kw):
    return _abi.spec_page_table(**(dict(table=P, ld=8, max_pages=8) | kw))


def rows(heads=2, D=64, B=2, N=3, data=P, **kw):
    d = dict(data=data, layer_stride=B * N * heads * D, seq_stride=N * heads * D, token_stride=heads * D, head_stride=D)
    return _abi.spec_rows(**(d | kw))


def rotation(**kw):
    return _abi.spec_rotation(**(dict(frequency=P, dim=64, interleaved=0, inverse=0, amplitude=1.0) | kw))


BAD_CACHES = [(dict(k=None), INV), (dict(v=None), INV), (dict(num_pages=0), INV), (dict(page_size=0), INV),
              (dict(num_heads=0), INV), (dict(num_layers=0), INV), (dict(dtype=3), INV), (dict(dtype=5), INV),
              (dict(head_dim=32), UNS), (dict(head_dim=96), UNS), (dict(head_dim=256), UNS),
              (dict(k=P + 8), UNS), (dict(v=P + 2), UNS), (dict(k_token_stride=100), UNS),
              (dict(k_head_stride=32), UNS), (dict(v_page_stride=0), UNS), (dict(v_token_stride=-96), UNS)]
BAD_TABLES = [dict(table=None), dict(max_pages=0), dict(ld=7), dict(max_pages=1 << 27, ld=1 << 27)]
BAD_ROTATIONS = [dict(dim=0), dict(dim=3), dict(dim=66), dict(dim=-2), dict(frequency=P + 4)]


def attention(lib, B=2, N=3, Hq=4, q=P, qs=(12 * 64, 4 * 64, 64), dtype=BF16, c=None, t=None, ctx=P, mask=None,
              ms=0, pos=None, ps=0, scale=0.125, window=0, sinks=0, out=FAR, ws=P, ws_bytes=None):
    need = lib.spec_paged_attention_q4_workspace_size(max(B, 0), min(max(N, 1), 4096), 4, 2, 64, BF16)
    return lib.spec_paged_attention_q4(q, *qs, Hq, dtype, c or cache(), t or table(), ctx, None, B, N, mask, ms,
                                       pos, ps, scale, window, sinks, out, None, None, ws,
                                       need if ws_bytes is None else ws_bytes, None)


def test_attention_refuses(lib):
    assert attention(lib, B=0) == OK
    for kw, want in BAD_CACHES:
        assert attention(lib, c=cache(**kw)) == want, kw
    for kw in BAD_TABLES:
        assert attention(lib, t=table(**kw)) == INV, kw
    bf16 = cache(dtype=BF16, k_token_stride=128, v_token_stride=128, k_head_stride=64, v_head_stride=64)
    for kw in (dict(c=cache(num_layers=2)), dict(c=bf16), dict(dtype=F32), dict(dtype=Q4), dict(dtype=9),
               dict(B=-1), dict(N=0), dict(N=4097), dict(Hq=0), dict(Hq=3), dict(q=None), dict(out=None),
               dict(ctx=None), dict(scale=0.0), dict(scale=float("nan")), dict(scale=3e38), dict(sinks=-1),
               dict(ws=None), dict(ws=P + 4), dict(ws_bytes=0), dict(window=4, mask=P), dict(ms=-1), dict(ps=-1),
               dict(out=P), dict(B=1 << 17, N=4096)):
        assert attention(lib, **kw) == INV, kw
    for kw in (dict(q=P + 8), dict(out=FAR + 8), dict(qs=(12 * 64, 4 * 64, 60)), dict(qs=(0, 4 * 64, 64))):
        assert attention(lib, **kw) == UNS, kw


def test_the_16_bit_entries_refuse_four_bits(lib):
    need = lib.spec_paged_attention_workspace_size(2, 3, 4, 2, 64, BF16)
    assert lib.spec_paged_attention(P, 768, 256, 64, 4, cache(), table(), P, None, 2, 3, None, 0, None, 0, 0.125, 0,
                                    0, FAR, None, None, P, need, None) == INV
    assert lib.spec_cache_append(P, 768, 384, 128, 64, P, 768, 384, 128, 64, cache(), table(), P, None, 2, 3, None,
                                 None) == INV
    assert lib.spec_paged_attention_workspace_size(1, 1, 8, 2, 128, Q4) == 0


def test_attention_workspace_sizes(lib):
    size = lib.spec_paged_attention_q4_workspace_size
    for n in (1, 2, 3, 4, 8, 9, 60, 4096):
        assert size(1, n, 8, 2, 128, BF16) > 0 and size(1, n, 8, 2, 64, F16) > 0
    assert size(1, 2, 256, 1, 128, BF16) > 0  # more heads than a row tile
    for bad in ((-1, 1, 8, 2, 128, BF16), (1, 0, 8, 2, 128, BF16), (1, 4097, 8, 2, 128, BF16),
                (1, 1, 7, 2, 128, BF16), (1, 1, 8, 0, 128, BF16), (1, 1, 8, 2, 96, BF16), (1, 1, 8, 2, 256, BF16),
                (1, 1, 8, 2, 128, F32), (1, 1, 8, 2, 128, Q4), (1 << 20, 4096, 8, 2, 128, BF16)):
        assert size(*bad) == 0, bad


def rotary(lib, x=None, out=None, dtype=BF16, B=2, N=3, heads=2, D=64, position=P, stride=0, r=None):
    return lib.spec_rotary(x or rows(), out or rows(data=FAR), dtype, B, N, heads, D, position, stride,
                           r or rotation(), None)


def test_rotary_refuses(lib):
    for kw in (dict(B=0), dict(N=0), dict(heads=0)):
        assert rotary(lib, **kw) == OK, kw
    for kw in BAD_ROTATIONS + [dict(frequency=None), dict(dim=514)]:
        assert rotary(lib, r=rotation(**kw)) == INV, kw
    for kw in (dict(dtype=Q4), dict(dtype=3), dict(B=-1), dict(N=-1), dict(heads=-1), dict(heads=65537), dict(D=0),
               dict(D=65537), dict(B=1 << 15, N=1 << 15), dict(position=None), dict(stride=-1),
               dict(x=rows(data=None)), dict(out=rows(data=None)), dict(x=rows(data=P + 1)),
               dict(x=rows(head_stride=32)), dict(out=rows(data=FAR, token_stride=0)),
               dict(x=rows(seq_stride=1 << 60)),
               # rows that overlap, the same rows in another order
               dict(out=rows(data=P + 64)), dict(out=rows(data=P, token_stride=64, head_stride=192))):
        assert rotary(lib, **kw) == INV, kw


def append(lib, q=None, out_q=None, heads=4, k=None, v=None, dtype=BF16, c=None, t=None, ctx=P, position=P, stride=0,
           B=2, N=3, r=None):
    return lib.spec_cache_append_rotary(q or rows(4), out_q or rows(4, data=FAR), heads, k or rows(), v or rows(),
                                        dtype, c or cache(), t or table(), ctx, None, position, stride, B, N,
                                        r or rotation(), None, None)


def test_append_rotary_refuses(lib):
    assert append(lib, B=0) == OK
    for kw, want in BAD_CACHES:
        assert append(lib, c=cache(**kw)) == want, kw
    for kw in BAD_TABLES:
        assert append(lib, t=table(**kw)) == INV, kw
    for kw in BAD_ROTATIONS:
        assert append(lib, r=rotation(**kw)) == INV, kw
    for kw in (dict(dtype=Q4), dict(dtype=3), dict(B=-1), dict(N=-1), dict(N=4097), dict(B=1 << 17, N=2048),
               dict(ctx=None), dict(k=rows(data=None)), dict(v=rows(data=None)), dict(stride=-1),
               dict(heads=0), dict(heads=65537), dict(out_q=rows(4, data=None)), dict(out_q=rows(4, data=P + 256)),
               dict(c=cache(dtype=F16, k_token_stride=128, v_token_stride=128, k_head_stride=64, v_head_stride=64))):
        assert append(lib, **kw) == INV, kw
    for kw in (dict(k=rows(data=P + 8)), dict(v=rows(token_stride=60)), dict(q=rows(4, head_stride=68)),
               dict(out_q=rows(4, data=FAR + 8)), dict(k=rows(seq_stride=0))):
        assert append(lib, **kw) == UNS, kw


def read(lib, c=None, t=None, start=P, B=2, N=3, dtype=BF16, k=None, v=None):
    return lib.spec_cache_read(c or cache(), t or table(), start, None, B, N, dtype, k or rows(), v or rows(), None,
                               None)


def test_read_refuses(lib):
    assert read(lib, B=0) == OK
    for kw, want in BAD_CACHES:
        assert read(lib, c=cache(**kw)) == want, kw
    for kw in BAD_TABLES:
        assert read(lib, t=table(**kw)) == INV, kw
    for kw in (dict(dtype=Q4), dict(dtype=3), dict(B=-1), dict(N=-1), dict(N=4097), dict(B=1 << 17, N=2048),
               dict(start=None), dict(k=rows(data=None)), dict(v=rows(data=None))):
        assert read(lib, **kw) == INV, kw
    for kw in (dict(k=rows(data=P + 8)), dict(v=rows(head_stride=8)), dict(k=rows(token_stride=0))):
        assert read(lib, **kw) == UNS, kw


def test_structs_have_the_headers_layout():
    assert ctypes.sizeof(_abi.spec_rotation) == 8 + 4 * 4
    assert ctypes.sizeof(_abi.spec_rows) == 5 * 8


def test_the_binding_refuses():
    x = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16)
    pos = torch.zeros(3, dtype=torch.int32)
    f = torch.ones(32, dtype=torch.float64)
    ints = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        sv.rotary(x, pos, f)  # not on the GPU
    k, v = sv.cache_4bit(4, 16, 2, 64, device="cpu")
    assert k.shape == (4, 16, 2, 48) and k.dtype == torch.uint8
    with pytest.raises(ValueError):
        sv.cache_append_rotary(x[:, :, :2], x[:, :, :2], k, v, ints[None], ints, f)
    with pytest.raises(ValueError):
        sv.cache_read(k, v, ints[None], ints, 3)
    with pytest.raises(ValueError):
        sv.paged_attention(x, k, v, ints[:, None], ints)
    for bad in ((4, 16, 2, 32), (4, 16, 2, 96), (4, 16, 2, 256)):
        with pytest.raises(ValueError):
            sv.cache_4bit(*bad, device="cpu")
    for kw in (dict(base=0.0), dict(scaling="none of these"), dict(scaling="turns", factor=0.0)):
        with pytest.raises(ValueError):
            sv.rotary_frequency(64, device="cpu", **kw)
    with pytest.raises(ValueError):
        sv.rotary_frequency(63, device="cpu")
