"""Host checks of the key-value cache operators: refused calls launch nothing.
No GPU; the pointers below are never dereferenced."""

import ctypes

import pytest
import torch

import speculative_decoding_verification_temp_gb300 as sv
from speculative_decoding_verification_temp_gb300 import _abi
from speculative_decoding_verification_temp_gb300 import build as build_mod

OK, INV, UNS = _abi.SPEC_OK, _abi.SPEC_ERR_INVALID_ARG, _abi.SPEC_ERR_UNSUPPORTED
P = 0x10000


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return _abi.load()


def cache(**kw):
    page, heads, D, pages, layers = 16, 2, 64, 10, 1
    d = dict(k=P, v=P, dtype=_abi.SPEC_BF16, num_layers=layers, num_pages=pages, page_size=page,
             num_heads=heads, head_dim=D)
    for x in "kv":
        d |= {f"{x}_layer_stride": pages * page * heads * D, f"{x}_page_stride": page * heads * D,
              f"{x}_token_stride": heads * D, f"{x}_head_stride": D}
    return _abi.spec_kv_cache(**(d | kw))


def table(**kw):
    return _abi.spec_page_table(**(dict(table=P, ld=8, max_pages=8) | kw))


BAD_CACHES = [
    (dict(k=None), INV), (dict(v=None), INV), (dict(dtype=3), INV), (dict(dtype=-1), INV),
    (dict(num_pages=0), INV), (dict(page_size=0), INV), (dict(page_size=65537), INV),
    (dict(num_heads=0), INV), (dict(head_dim=0), INV), (dict(num_layers=0), INV),
    (dict(head_dim=264), UNS), (dict(head_dim=60), UNS), (dict(k=P + 8), UNS), (dict(v=P + 2), UNS),
    (dict(k_token_stride=132), UNS), (dict(v_page_stride=16 * 2 * 64 + 4), UNS),
    (dict(k_head_stride=32), UNS), (dict(k_page_stride=-2048), UNS), (dict(v_token_stride=0), UNS),
    (dict(v_page_stride=1 << 60), UNS)]
BAD_TABLES = [dict(table=None), dict(max_pages=0), dict(ld=7), dict(max_pages=1 << 27, ld=1 << 27)]


def attention(lib, B=2, N=3, Hq=4, q=P, qs=(12 * 64, 4 * 64, 64), c=None, t=None, ctx=P, mask=None,
              ms=0, pos=None, ps=0, scale=0.125, window=0, sinks=0, out=P << 4, ws=P, ws_bytes=None):
    need = lib.spec_paged_attention_workspace_size(max(B, 0), min(max(N, 1), 4096), 4, 2, 64, 1)
    return lib.spec_paged_attention(q, *qs, Hq, c or cache(), t or table(), ctx, None, B, N, mask, ms,
                                    pos, ps, scale, window, sinks, out, None, None, ws,
                                    need if ws_bytes is None else ws_bytes, None)


def test_attention_refuses(lib):
    assert attention(lib, B=0) == OK
    for kw, want in BAD_CACHES:
        assert attention(lib, c=cache(**kw)) == want, kw
    for kw in BAD_TABLES:
        assert attention(lib, t=table(**kw)) == INV, kw
    assert attention(lib, c=cache(num_layers=2)) == INV
    for kw in (dict(B=-1), dict(N=0), dict(N=4097), dict(Hq=0), dict(Hq=3), dict(q=None), dict(out=None),
               dict(ctx=None), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(sinks=-1), dict(ws=None), dict(ws=P + 4),
               dict(window=4, mask=P), dict(ms=-1), dict(ps=-1), dict(B=1 << 17, N=4096),
               dict(out=P), dict(out=P + 12 * 64 * 2 + 2 * 4 * 64 * 2), dict(q=(P << 4) + 16)):
        assert attention(lib, **kw) == INV, kw
    need = lib.spec_paged_attention_workspace_size(2, 3, 4, 2, 64, 1)
    assert attention(lib, ws_bytes=need - 1) == INV
    for kw in (dict(q=P + 8), dict(out=(P << 4) + 8), dict(qs=(12 * 64, 4 * 64, 60)), dict(qs=(0, 4 * 64, 64)),
               dict(qs=(12 * 64, 8, 64))):
        assert attention(lib, **kw) == UNS, kw


def test_attention_workspace_sizes(lib):
    size = lib.spec_paged_attention_workspace_size
    assert size(1, 1, 8, 2, 128, _abi.SPEC_BF16) > 0
    assert size(1, 1, 8, 2, 256, _abi.SPEC_F32) > 0
    for bad in ((-1, 1, 8, 2, 128, 1), (1, 0, 8, 2, 128, 1), (1, 4097, 8, 2, 128, 1),
                (1, 1, 7, 2, 128, 1), (1, 1, 8, 0, 128, 1), (1, 1, 8, 2, 257, 1), (1, 1, 8, 2, 129, 1),
                (1, 1, 8, 2, 128, 3), (1 << 20, 4096, 8, 2, 128, 1)):
        assert size(*bad) == 0, bad


def append(lib, B=2, N=3, kn=P, vn=P, ks=(768, 384, 128, 64), vs=(768, 384, 128, 64), c=None, t=None,
           ctx=P):
    return lib.spec_cache_append(kn, *ks, vn, *vs, c or cache(), t or table(), ctx, None, B, N, None,
                                 None)


def test_append_refuses(lib):
    assert append(lib, B=0) == OK
    for kw, want in BAD_CACHES:
        assert append(lib, c=cache(**kw)) == want, kw
    for kw in BAD_TABLES:
        assert append(lib, t=table(**kw)) == INV, kw
    for kw in (dict(B=-1), dict(N=-1), dict(N=4097), dict(B=1 << 17, N=2048), dict(kn=None),
               dict(vn=None), dict(ctx=None)):
        assert append(lib, **kw) == INV, kw
    for kw in (dict(kn=P + 8), dict(vn=P + 4), dict(ks=(768, 384, 128, 60)), dict(vs=(768, 380, 128, 64)),
               dict(ks=(768, 384, 0, 64))):
        assert append(lib, **kw) == UNS, kw


def compact(lib, B=2, c=None, t=None, ctx=P, path=P, width=4, taken=P, out=P + 64):
    return lib.spec_cache_compact(c or cache(), t or table(), ctx, path, width, taken, B, out, None,
                                  None)


def test_compact_refuses(lib):
    assert compact(lib, B=0) == OK
    for kw, want in BAD_CACHES:
        assert compact(lib, c=cache(**kw)) == want, kw
    for kw in BAD_TABLES:
        assert compact(lib, t=table(**kw)) == INV, kw
    for kw in (dict(B=-1), dict(width=0), dict(width=4098), dict(ctx=None), dict(path=None),
               dict(taken=None), dict(out=None), dict(out=P)):
        assert compact(lib, **kw) == INV, kw


def pool(**kw):
    return _abi.spec_page_pool(**(dict(page_table=P, ld_table=8, max_pages=8, page_count=P, ref_count=P,
                                       free_list=P, free_count=P, num_seqs=3, num_pages=10,
                                       page_size=16) | kw))


BAD_POOLS = [dict(page_table=None), dict(page_count=None), dict(ref_count=None), dict(free_list=None),
             dict(free_count=None), dict(max_pages=0), dict(ld_table=7), dict(num_pages=0),
             dict(page_size=0), dict(page_size=65537), dict(num_seqs=4097),
             dict(max_pages=1 << 27, ld_table=1 << 27), dict(num_seqs=-1)]


def test_resize_and_fork_refuse(lib):
    fork = lambda p=None, c=None, ctx=P, src=P, dst=P, F=2, ws=P, n=None: lib.spec_cache_fork(
        p or pool(), c or cache(), ctx, src, dst, F, None, ws,
        lib.spec_cache_fork_workspace_size(2) if n is None else n, None)
    assert lib.spec_cache_resize(pool(num_seqs=0), P, None, None) == OK
    assert lib.spec_cache_resize(pool(), None, None, None) == INV
    assert fork(F=0) == OK
    for kw in BAD_POOLS:
        assert lib.spec_cache_resize(pool(**kw), P, None, None) == INV, kw
        assert fork(p=pool(**kw)) == INV, kw
    for kw, want in BAD_CACHES:
        assert fork(c=cache(**kw)) == want, kw
    for kw in (dict(F=-1), dict(F=4097), dict(ctx=None), dict(src=None), dict(dst=None), dict(ws=None),
               dict(ws=P + 2), dict(n=lib.spec_cache_fork_workspace_size(2) - 1),
               dict(c=cache(num_pages=11)), dict(c=cache(page_size=8))):
        assert fork(**kw) == INV, kw
    assert lib.spec_cache_fork_workspace_size(-1) == 0
    assert lib.spec_cache_fork_workspace_size(4097) == 0
    assert lib.spec_cache_fork_workspace_size(1) > 0


def test_structs_have_the_headers_layout():
    assert ctypes.sizeof(_abi.spec_kv_cache) == 2 * 8 + 8 * 8 + 6 * 4
    assert ctypes.sizeof(_abi.spec_page_table) == 24
    assert ctypes.sizeof(_abi.spec_page_pool) == 8 + 8 + 8 + 4 * 8 + 16


def test_the_binding_refuses_tensors_off_the_gpu():
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    ints = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        sv.paged_attention(torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16), k, k, ints[None], ints)
    with pytest.raises(ValueError):
        sv.cache_append(k[None, 0], k[None, 0], k, k, ints[None], ints)
    with pytest.raises(ValueError):
        sv.cache_compact(k, k, ints[None], ints, ints[None], ints)
    pool = sv.page_pool(1, 2, 4, device="cpu")
    assert pool.free_list.tolist() == [3, 2, 1, 0] and pool.page_table.tolist() == [[-1, -1]]
    with pytest.raises(ValueError):
        sv.cache_resize(pool, ints, 16)
    with pytest.raises(ValueError):
        sv.cache_fork(pool, k, k, ints, ints, ints)


def test_sizes_beyond_32_bits_are_refused(lib):
    # 2^34 pieces of 16 bytes in a page: more than the copy of a page counts
    huge = dict(num_pages=2, page_size=65536, num_heads=4096, head_dim=256, dtype=_abi.SPEC_F32)
    for x in "kv":
        huge |= {f"{x}_layer_stride": 1 << 41, f"{x}_page_stride": 1 << 40, f"{x}_token_stride": 1 << 20,
                 f"{x}_head_stride": 256}
    assert compact(lib, c=cache(**huge)) == UNS
    assert lib.spec_cache_fork(pool(num_pages=2, page_size=65536), cache(**huge), P, P, P, 2, None, P, 64,
                               None) == UNS
    # finite, but not times log2(e), which the kernels take the scores times
    assert attention(lib, scale=3e38) == INV


@pytest.mark.parametrize("x,want", [(5, 5), (0, 0), (-3, -1), (2 ** 31 - 1, 2 ** 31 - 1),
                                    (2 ** 31, 2 ** 31 - 1), (2 ** 32 + 5, 2 ** 31 - 1), (-2 ** 40, -1)])
def test_the_bindings_integers_do_not_wrap(x, want):
    from speculative_decoding_verification_temp_gb300 import cache as binding
    assert binding._c_int(x) == want


def test_the_binding_refuses_shapes_beyond_32_bits():
    from speculative_decoding_verification_temp_gb300 import cache as binding
    dev = torch.device("meta")
    wide = torch.empty(1, 2 ** 31, dtype=torch.int32, device=dev)
    with pytest.raises(ValueError):
        binding._table(wide, 1, dev)
    with pytest.raises(ValueError):
        binding._sizes((2 ** 32 + 1, 16, 2, 64))


@pytest.mark.parametrize("dtype,values,want", [
    (torch.int64, [5, -1, 2 ** 31 - 1, 2 ** 31, 2 ** 32 + 3, 2 ** 63 - 1, -2 ** 31 - 1, -2 ** 32 + 5],
     [5, -1, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, -2 ** 31, -2 ** 31]),
    (torch.uint64, [5, 2 ** 32 + 3, 2 ** 63, 2 ** 64 - 1], [5] + 3 * [2 ** 31 - 1]),
    (torch.uint32, [5, 2 ** 31 + 3, 2 ** 32 - 1], [5] + 2 * [2 ** 31 - 1]),
    (torch.uint16, [5, 2 ** 16 - 1], [5, 2 ** 16 - 1]), (torch.int16, [5, -7], [5, -7]),
    (torch.uint8, [5, 255], [5, 255])])
def test_the_bindings_integer_tensors_do_not_wrap(dtype, values, want):
    from speculative_decoding_verification_temp_gb300 import cache as binding
    x = torch.tensor(values, dtype=dtype)
    dev = torch.device("cpu")
    got = binding._ints(x, x.shape, dev, "x")
    assert got.dtype == torch.int32 and got.tolist() == want
    got, table = binding._table(x[None], 1, dev)
    assert got.dtype == torch.int32 and got.tolist() == [want] and table.max_pages == len(values)
