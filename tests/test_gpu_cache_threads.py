"""Calls of the page operators from several host threads at once, with sizes
whose shared memory has to be allowed: no thread's call lowers what another's
may use."""

import threading

import pytest
import torch

import speculative_decoding_verification_temp_gb300 as sv
from speculative_decoding_verification_temp_gb300 import _abi
from speculative_decoding_verification_temp_gb300 import cache as binding

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)


def ints(*shape, value=0):
    return torch.full(shape, value, dtype=torch.int32, device=DEV)


def compact(lib, width):
    k, v = (torch.zeros(2, 16, 1, 8, dtype=torch.bfloat16, device=DEV) for _ in "kv")
    table, path, out = ints(1, 1), ints(1, width), ints(1)
    taken, ctx = ints(1), ints(1, value=3)
    args = (binding._cache(k, v, False), binding._table(table, 1, DEV)[1], ctx.data_ptr(), path.data_ptr(),
            width, taken.data_ptr(), 1, out.data_ptr(), None)
    return lib.spec_cache_compact, args, (k, v, table, path, out, taken, ctx), lambda: out.tolist() == [4]


def resize(lib, B):
    pool = sv.page_pool(B, 1, B, device=DEV)
    length = ints(B, value=5)
    return (lib.spec_cache_resize, (binding._pool(pool, 16), length.data_ptr(), None), (pool, length),
            lambda: bool((pool.page_count == 1).all()))


def fork(lib, F):
    pool = sv.page_pool(2, 1, 4, device=DEV)
    k, v = (torch.zeros(4, 16, 1, 8, dtype=torch.bfloat16, device=DEV) for _ in "kv")
    ctx, src, dst = ints(2), ints(F, value=7), ints(F)  # no such source: nothing is forked
    ws = torch.empty(lib.spec_cache_fork_workspace_size(F), dtype=torch.uint8, device=DEV)
    flags = ints(F)
    args = (binding._pool(pool, 16), binding._cache(k, v, True), ctx.data_ptr(), src.data_ptr(),
            dst.data_ptr(), F, flags.data_ptr(), ws.data_ptr(), ws.numel())
    return (lib.spec_cache_fork, args, (pool, k, v, ctx, src, dst, ws, flags),
            lambda: bool((flags == sv.FLAG_BAD_SEQUENCE).all()))


@pytest.mark.parametrize("make,sizes", [(compact, (4097, 2600)), (resize, (4096, 2100)),
                                        (fork, (4096, 3500))], ids=["compact", "resize", "fork"])
def test_two_threads(make, sizes):
    lib = _abi.load()
    calls = [make(lib, n) for n in sizes]
    streams = [torch.cuda.Stream(DEV) for _ in sizes]
    torch.cuda.synchronize()
    go, failed = threading.Barrier(len(sizes)), [0] * len(sizes)

    def work(i):
        fn, args, _, _ = calls[i]
        with torch.cuda.device(DEV):
            go.wait()
            for _ in range(3000):
                failed[i] += fn(*args, streams[i].cuda_stream) != _abi.SPEC_OK

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sizes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert failed == [0] * len(sizes)
    assert all(done() for _, _, _, done in calls)
