"""Thin torch binding of the paged key-value cache operators: argument
marshalling only, as in ``api``.

A cache is a pair of tensors [num_pages, page_size, num_heads, head_dim] (one
layer) or [num_layers, num_pages, page_size, num_heads, head_dim]; any strides
whose last is 1 (a transposed [.., num_heads, page_size, head_dim] tensor, keys
and values interleaved).  The calls run on torch's current stream of the
cache's device.  Integer inputs may be of any integer type; values beyond 32 bits
are flagged as any other bad page or length.  They are forward operators: tensors
that require gradients are refused while autograd records.
"""

import functools
from collections import namedtuple

import torch

from . import _abi
from .api import _check

AttentionResult = namedtuple("AttentionResult", "out lse flags")
CompactResult = namedtuple("CompactResult", "context_len flags")
PagePool = namedtuple("PagePool", "page_table page_count ref_count free_list free_count")

_KV_DTYPES = {torch.float32: _abi.SPEC_F32, torch.bfloat16: _abi.SPEC_BF16,
              torch.float16: _abi.SPEC_F16}


_INT_MAX = 2 ** 31 - 1


def _c_int(x):
    """x for a C int: what lies beyond it would wrap, and is taken as its largest
    value or as -1."""
    return max(min(int(x), _INT_MAX), -1)


def _sizes(shape):
    if max(shape) > _INT_MAX:
        raise ValueError(f"sizes have to fit 32 bits, got {list(shape)}")


def _on(x, dev, name):
    if not isinstance(x, torch.Tensor) or x.device != dev:
        raise ValueError(f"{name} must be a tensor on {dev}")


def _forward_only(*tensors):
    for t in tensors:
        if t.requires_grad and torch.is_grad_enabled():
            raise ValueError(
                "the cache operators have no gradient: call them under torch.no_grad()")


def _int32(x):
    """x as int32.  What lies beyond that would wrap, and is taken as its largest
    or smallest value: no page, length, node or sequence is that large, so the
    operators flag it (and clamp num_new and position to their ranges)."""
    if x.dtype == torch.uint64:
        # as int64 the upper half is negative
        x = x.view(torch.int64)
        x = torch.where(x < 0, _INT_MAX, x)
    elif x.dtype == torch.uint32:
        x = x.to(torch.int64)
    if x.dtype == torch.int64:
        x = x.clamp(-_INT_MAX - 1, _INT_MAX)
    return x.to(torch.int32)


def _ints(x, shape, dev, name):
    """An int32 tensor of `shape` on dev, contiguous; another integer type is converted."""
    _on(x, dev, name)
    if x.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(x.shape)}")
    if x.dtype != torch.int32:
        if x.is_floating_point() or x.is_complex() or x.dtype == torch.bool:
            raise ValueError(f"{name} must hold integers")
        x = _int32(x)
    return x if x.is_contiguous() else x.contiguous()


def _inplace(x, shape, dev, name):
    """An int32 tensor that the call writes: no conversion, which would write a copy."""
    _on(x, dev, name)
    if x.dtype != torch.int32 or x.shape != shape or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor {list(shape)}")
    return x


def _cache(k, v, layers):
    """The spec_kv_cache of a pair of cache tensors.  layers: whether a layer
    dimension is allowed."""
    if not isinstance(k, torch.Tensor) or not k.is_cuda:
        raise ValueError("k_cache must be a CUDA tensor")
    _on(v, k.device, "v_cache")
    _forward_only(k, v)
    shape, code, ks, vs = k.shape, _KV_DTYPES.get(k.dtype), k.stride(), v.stride()
    if code is None or v.dtype != k.dtype:
        raise ValueError("k_cache and v_cache must both be float32, bfloat16 or float16")
    dims = len(shape)
    if v.shape != shape or dims != 4 and not (layers and dims == 5):
        raise ValueError("k_cache and v_cache must be [%snum_pages, page_size, num_heads, head_dim]"
                         % ("num_layers, " if layers else ""))
    _sizes(shape)
    if shape[-1] > 1 and (ks[-1] != 1 or vs[-1] != 1):
        raise ValueError("the last dimension of the caches must be contiguous")
    if dims == 4:
        return _abi.spec_kv_cache(k.data_ptr(), v.data_ptr(), 0, ks[0], ks[1], ks[2], 0, vs[0],
                                  vs[1], vs[2], code, 1, *shape)
    return _abi.spec_kv_cache(k.data_ptr(), v.data_ptr(), *ks[:4], *vs[:4], code, *shape)


def _table(page_table, B, dev):
    _on(page_table, dev, "page_table")
    shape = page_table.shape
    if len(shape) != 2 or shape[0] != B:
        raise ValueError(f"page_table must be [{B}, max_pages]")
    _sizes(shape)
    if page_table.dtype != torch.int32:
        page_table = _ints(page_table, tuple(shape), dev, "page_table")
    ld, step = page_table.stride()
    if step != 1 or ld < shape[1]:
        page_table = page_table.contiguous()
        ld = shape[1]
    return page_table, _abi.spec_page_table(page_table.data_ptr(), ld, shape[1])


# the current stream's handle, without a Stream object where torch offers that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


def _run(dev, fn, *args):
    """fn(*args, stream) on dev's current stream, with dev the current device."""
    index = dev.index
    if index == torch.cuda.current_device():
        code = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            code = fn(*args, _raw_stream(index))
    if code:
        _check(code)


def _ptr(x):
    return None if x is None else x.data_ptr()


def _rows(x):
    """x as rows that the kernels can read: 16-byte aligned and apart, the last
    dimension contiguous; a copy where they are not (slices at odd offsets,
    expanded dimensions, transposed heads)."""
    if x.is_contiguous() and x.data_ptr() % 16 == 0:
        return x
    shape, strides, size = x.shape, x.stride(), x.element_size()
    if x.data_ptr() % 16 == 0 and strides[-1] == 1 and all(
            n <= 1 or s >= shape[-1] and s * size % 16 == 0
            for n, s in zip(shape[:-1], strides[:-1])):
        return x
    return x.clone(memory_format=torch.contiguous_format)


@functools.lru_cache(maxsize=256)
def _attention_bytes(*sizes):
    return max(_abi.load().spec_paged_attention_workspace_size(*sizes), 32)


def paged_attention(q, k_cache, v_cache, page_table, context_len, scale=None, num_new=None,
                    tree_mask=None, position=None, window=0, sinks=0, return_lse=False,
                    return_flags=False, out=None):
    """Attention of N new tokens per sequence over the cache's pages (see
    spec_paged_attention); the pages already hold the new tokens (cache_append).

    q [B, N, num_q_heads, head_dim] with the cache's type; k_cache, v_cache
    [num_pages, page_size, num_heads, head_dim]; page_table [B, max_pages] and
    context_len [B] integer.  scale: 1/sqrt(head_dim) by default.  num_new [B]:
    new tokens of each sequence (N by default; outputs behind them are not
    written).  tree_mask: the words of tree_mask(), [B, N, ceil(N/64)] or one
    tree [N, ceil(N/64)] for all; without it new token n sees new tokens 0..n.
    window, sinks: a sliding window and the first tokens that stay visible;
    position [B, N] or [N]: the new tokens' depths, needed for windows over
    trees.  Returns AttentionResult with out [B, N, num_q_heads, head_dim], lse
    [B, N, num_q_heads] float32 or None, flags [B] int32 or None (asked for,
    they cost a launch).
    """
    cache = _cache(k_cache, v_cache, False)
    dev = k_cache.device
    _on(q, dev, "q")
    _forward_only(q)
    if q.dim() != 4 or q.shape[3] != k_cache.shape[3] or q.dtype != k_cache.dtype:
        raise ValueError("q must be [B, N, num_q_heads, head_dim] with the cache's type")
    B, N, Hq, D = shape = q.shape
    q = _rows(q)
    strides = q.stride()
    page_table, table = _table(page_table, B, dev)
    context_len = _ints(context_len, (B,), dev, "context_len")
    if num_new is not None:
        num_new = _ints(num_new, (B,), dev, "num_new")
    mask_stride = pos_stride = 0
    if tree_mask is not None:
        _on(tree_mask, dev, "tree_mask")
        words = (N + 63) // 64
        if tree_mask.dtype not in (torch.int64, torch.uint64) or \
                tuple(tree_mask.shape) not in ((B, N, words), (N, words)):
            raise ValueError(f"tree_mask must be int64 words [{B}, {N}, {words}] or [{N}, {words}]")
        tree_mask = tree_mask.contiguous()
        mask_stride = N * words if tree_mask.dim() == 3 else 0
    if position is not None:
        pos_stride = N if position.dim() == 2 else 0
        position = _ints(position, (B, N) if position.dim() == 2 else (N,), dev, "position")
    if out is None:
        out = torch.empty(shape, dtype=q.dtype, device=dev)
    else:
        _on(out, dev, "out")
        _forward_only(out)
        if out.shape != shape or out.dtype != q.dtype or not out.is_contiguous():
            raise ValueError("out must be a contiguous tensor like q")
    lse = torch.empty((B, N, Hq), dtype=torch.float32, device=dev) if return_lse else None
    flags = torch.empty(B, dtype=torch.int32, device=dev) if return_flags else None
    nbytes = _attention_bytes(B, N, Hq, cache.num_heads, D, cache.dtype)
    # of the caching allocator, ordered on this stream and kept by a graph that
    # captures the call: never shared with calls on other streams
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _run(dev, _abi.load().spec_paged_attention, q.data_ptr(), strides[0], strides[1], strides[2], Hq, cache,
         table, context_len.data_ptr(), _ptr(num_new), B, N, _ptr(tree_mask), mask_stride,
         _ptr(position), pos_stride, D ** -0.5 if scale is None else float(scale),
         _c_int(window), _c_int(sinks), out.data_ptr(), _ptr(lse), _ptr(flags), ws.data_ptr(), nbytes)
    return AttentionResult(out, lse, flags)


def cache_append(k_new, v_new, k_cache, v_cache, page_table, context_len, num_new=None,
                 return_flags=False):
    """Writes new tokens' keys and values into the pages (see spec_cache_append).

    k_new, v_new [B, N, num_heads, head_dim] for a cache of one layer, or
    [num_layers, B, N, num_heads, head_dim]; page_table, context_len, num_new as
    for paged_attention.  Returns flags [B] int32, or None (return_flags False;
    asked for, they cost a launch).
    """
    cache = _cache(k_cache, v_cache, True)
    dev = k_cache.device
    _on(k_new, dev, "k_new")
    _on(v_new, dev, "v_new")
    _forward_only(k_new, v_new)
    shape = k_new.shape
    if len(shape) != k_cache.dim() or shape[-2:] != k_cache.shape[-2:] or v_new.shape != shape or \
            (len(shape) == 5 and shape[0] != k_cache.shape[0]):
        raise ValueError("k_new and v_new must be [%sB, N, num_heads, head_dim] of the cache's sizes"
                         % ("num_layers, " if k_cache.dim() == 5 else ""))
    if k_new.dtype != k_cache.dtype or v_new.dtype != k_cache.dtype:
        raise ValueError("k_new and v_new must have the cache's type")
    B, N = shape[-4:-2]
    k_new, v_new = _rows(k_new), _rows(v_new)
    ks, vs = k_new.stride(), v_new.stride()
    if len(shape) == 4:
        ks, vs = (0, *ks), (0, *vs)
    page_table, table = _table(page_table, B, dev)
    context_len = _ints(context_len, (B,), dev, "context_len")
    if num_new is not None:
        num_new = _ints(num_new, (B,), dev, "num_new")
    flags = torch.empty(B, dtype=torch.int32, device=dev) if return_flags else None
    _run(dev, _abi.load().spec_cache_append, k_new.data_ptr(), *ks[:4], v_new.data_ptr(), *vs[:4],
         cache, table, context_len.data_ptr(), _ptr(num_new), B, N, _ptr(flags))
    return flags


def cache_compact(k_cache, v_cache, page_table, context_len, path, num_accepted):
    """Moves a verified tree's accepted path together behind the context, in
    every layer (see spec_cache_compact).

    path [B, width] and num_accepted [B]: verify_tree's results.  Returns
    CompactResult with context_len [B] int32 (the new lengths: context, root and
    accepted nodes) and flags [B] int32.
    """
    cache = _cache(k_cache, v_cache, True)
    dev = k_cache.device
    _on(path, dev, "path")
    if path.dim() != 2:
        raise ValueError("path must be [B, width]")
    B, width = path.shape
    path = _ints(path, (B, width), dev, "path")
    num_accepted = _ints(num_accepted, (B,), dev, "num_accepted")
    page_table, table = _table(page_table, B, dev)
    context_len = _ints(context_len, (B,), dev, "context_len")
    length = torch.empty(B, dtype=torch.int32, device=dev)
    flags = torch.empty(B, dtype=torch.int32, device=dev)
    _run(dev, _abi.load().spec_cache_compact, cache, table, context_len.data_ptr(),
         path.data_ptr(), width, num_accepted.data_ptr(), B, length.data_ptr(), flags.data_ptr())
    return CompactResult(length, flags)


def page_pool(num_seqs, max_pages, num_pages, device="cuda"):
    """A PagePool of empty sequences: every page is free, page 0 the next one."""
    ints = dict(dtype=torch.int32, device=device)
    return PagePool(torch.full((num_seqs, max_pages), -1, **ints), torch.zeros(num_seqs, **ints),
                    torch.zeros(num_pages, **ints), torch.arange(num_pages - 1, -1, -1, **ints),
                    torch.full((1,), num_pages, **ints))


def _pool(pool, page_size):
    table = pool.page_table
    if not isinstance(table, torch.Tensor) or not table.is_cuda or table.dim() != 2:
        raise ValueError("page_table must be a CUDA tensor [num_seqs, max_pages]")
    dev = table.device
    B, pages = table.shape[0], pool.ref_count.numel()
    if table.dtype != torch.int32 or table.stride(1) != 1 or \
            (B > 1 and table.stride(0) < table.shape[1]):
        raise ValueError("page_table must be int32 with contiguous rows")
    ld = table.stride(0) if B > 1 else table.shape[1]
    return _abi.spec_page_pool(
        table.data_ptr(), ld, table.shape[1],
        _inplace(pool.page_count, (B,), dev, "page_count").data_ptr(),
        _inplace(pool.ref_count, (pages,), dev, "ref_count").data_ptr(),
        _inplace(pool.free_list, (pages,), dev, "free_list").data_ptr(),
        _inplace(pool.free_count, (1,), dev, "free_count").data_ptr(), B, pages, page_size)


def cache_resize(pool, length, page_size):
    """Gives each sequence the pages of length[b] tokens, in place (see
    spec_cache_resize): pages behind them go back to the pool, missing ones are
    taken from it; length 0 frees a sequence.  Returns flags [num_seqs] int32.
    """
    p = _pool(pool, _c_int(page_size))
    dev = pool.page_table.device
    length = _ints(length, (p.num_seqs,), dev, "length")
    flags = torch.empty(p.num_seqs, dtype=torch.int32, device=dev)
    _run(dev, _abi.load().spec_cache_resize, p, length.data_ptr(), flags.data_ptr())
    return flags


def cache_fork(pool, k_cache, v_cache, context_len, src, dst):
    """Lets sequences dst[f] go on from the tokens of sequences src[f], in place
    (see spec_cache_fork): full pages are shared, a partly filled last page is
    copied in every layer, context_len[dst[f]] is set.  Returns flags [F] int32.
    """
    cache = _cache(k_cache, v_cache, True)
    p = _pool(pool, cache.page_size)
    dev = k_cache.device
    _on(pool.page_table, dev, "page_table")
    _inplace(context_len, (p.num_seqs,), dev, "context_len")
    _on(src, dev, "src")
    if src.dim() != 1:
        raise ValueError("src must be [F]")
    F = src.shape[0]
    src = _ints(src, (F,), dev, "src")
    dst = _ints(dst, (F,), dev, "dst")
    flags = torch.empty(F, dtype=torch.int32, device=dev)
    lib = _abi.load()
    ws = torch.empty(max(lib.spec_cache_fork_workspace_size(F), 16), dtype=torch.uint8, device=dev)
    _run(dev, lib.spec_cache_fork, p, cache, context_len.data_ptr(), src.data_ptr(),
         dst.data_ptr(), F, flags.data_ptr(), ws.data_ptr(), ws.numel())
    return flags
