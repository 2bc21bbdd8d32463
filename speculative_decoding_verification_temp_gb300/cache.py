"""Thin torch binding of the paged key-value cache operators: argument
marshalling only, as in ``api``.

A cache is a pair of tensors [num_pages, page_size, num_heads, head_dim] (one
layer) or [num_layers, num_pages, page_size, num_heads, head_dim]; any strides
whose last is 1 (a transposed [.., num_heads, page_size, head_dim] tensor, keys
and values interleaved).  A cache of 4-bit rows is a pair of uint8 tensors whose last
dimension is head_dim / 2 + 16 (cache_4bit makes one); every operator takes either.  The calls run on torch's current stream of the
cache's device.  Integer inputs may be of any integer type; values beyond 32 bits
are flagged as any other bad page or length.  They are forward operators: tensors
that require gradients are refused while autograd records.
"""

import functools
import math
from collections import namedtuple

import torch

from . import _abi
from .api import _check

AttentionResult = namedtuple("AttentionResult", "out lse flags")
RotaryAppendResult = namedtuple("RotaryAppendResult", "q flags")
ReadResult = namedtuple("ReadResult", "k v flags")
RotaryFrequency = namedtuple("RotaryFrequency", "frequency amplitude")
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


@functools.lru_cache(maxsize=512)
def _cache_layout(dtype, v_dtype, shape, v_shape, ks, vs, layers):
    """The spec_kv_cache of caches of these sizes and strides (2.7 us a call to check and
    fill it in, 1.4 to copy it)."""
    code = _KV_DTYPES.get(dtype)
    sizes = shape
    if dtype == torch.uint8:
        # 4-bit rows; their strides count bytes, and are never those of one element
        code, width = _abi.SPEC_Q4, shape[-1] if shape else 0
        if width not in (48, 80):
            raise ValueError("4-bit caches have rows of head_dim / 2 + 16 bytes, head_dim 64 or 128")
        sizes = (*shape[:-1], 2 * (width - 16))
    if code is None or v_dtype != dtype:
        raise ValueError("k_cache and v_cache must both be float32, bfloat16 or float16, or 4-bit rows "
                         "(uint8)")
    dims = len(shape)
    if v_shape != shape or dims != 4 and not (layers and dims == 5):
        raise ValueError("k_cache and v_cache must be [%snum_pages, page_size, num_heads, head_dim]"
                         % ("num_layers, " if layers else ""))
    _sizes(sizes)
    if sizes[-1] > 1 and (ks[-1] != 1 or vs[-1] != 1):
        raise ValueError("the last dimension of the caches must be contiguous")
    if dims == 4:
        return _abi.spec_kv_cache(None, None, 0, ks[0], ks[1], ks[2], 0, vs[0], vs[1], vs[2], code, 1, *sizes)
    return _abi.spec_kv_cache(None, None, *ks[:4], *vs[:4], code, *sizes)


def _cache(k, v, layers):
    """The spec_kv_cache of a pair of cache tensors.  layers: whether a layer
    dimension is allowed."""
    if not isinstance(k, torch.Tensor) or not k.is_cuda:
        raise ValueError("k_cache must be a CUDA tensor")
    _on(v, k.device, "v_cache")
    _forward_only(k, v)
    cache = _abi.spec_kv_cache.from_buffer_copy(
        _cache_layout(k.dtype, v.dtype, k.shape, v.shape, k.stride(), v.stride(), layers))
    cache.k, cache.v = k.data_ptr(), v.data_ptr()
    return cache


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
def _attention_bytes(four, *sizes):
    lib = _abi.load()
    size = lib.spec_paged_attention_q4_workspace_size if four else lib.spec_paged_attention_workspace_size
    return max(size(*sizes), 32)


def paged_attention(q, k_cache, v_cache, page_table, context_len, scale=None, num_new=None,
                    tree_mask=None, position=None, window=0, sinks=0, return_lse=False,
                    return_flags=False, out=None):
    """Attention of N new tokens per sequence over the cache's pages (see
    spec_paged_attention); the pages already hold the new tokens (cache_append).

    q [B, N, num_q_heads, head_dim] with the cache's type (bfloat16 or float16 over
    4-bit rows, see spec_paged_attention_q4); k_cache, v_cache
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
    four = cache.dtype == _abi.SPEC_Q4
    if q.dim() != 4 or q.shape[3] != cache.head_dim or \
            (q.dtype not in (torch.bfloat16, torch.float16) if four else q.dtype != k_cache.dtype):
        raise ValueError("q must be [B, N, num_q_heads, head_dim] with the cache's type (bfloat16 or "
                         "float16 over 4-bit rows)")
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
        _on(position, dev, "position")
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
    dtype = _KV_DTYPES[q.dtype]
    nbytes = _attention_bytes(four, B, N, Hq, cache.num_heads, D, dtype)
    # of the caching allocator, ordered on this stream and kept by a graph that
    # captures the call: never shared with calls on other streams
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    lib = _abi.load()
    fn, heads = (lib.spec_paged_attention_q4, (Hq, dtype)) if four else (lib.spec_paged_attention, (Hq,))
    _run(dev, fn, q.data_ptr(), strides[0], strides[1], strides[2], *heads, cache,
         table, context_len.data_ptr(), _ptr(num_new), B, N, _ptr(tree_mask), mask_stride,
         _ptr(position), pos_stride, D ** -0.5 if scale is None else float(scale),
         _c_int(window), _c_int(sinks), out.data_ptr(), _ptr(lse), _ptr(flags), ws.data_ptr(), nbytes)
    return AttentionResult(out, lse, flags)


def cache_append(k_new, v_new, k_cache, v_cache, page_table, context_len, num_new=None,
                 return_flags=False):
    """Writes new tokens' keys and values into the pages (see spec_cache_append).

    k_new, v_new [B, N, num_heads, head_dim] for a cache of one layer, or
    [num_layers, B, N, num_heads, head_dim]; page_table, context_len, num_new as
    for paged_attention.  A 4-bit cache takes float32, bfloat16 or float16 rows (see
    spec_cache_append_rotary).  Returns flags [B] int32, or None (return_flags False;
    asked for, they cost a launch).
    """
    if isinstance(k_cache, torch.Tensor) and k_cache.dtype == torch.uint8:
        return _append(k_new, v_new, k_cache, v_cache, page_table, context_len, num_new, None, return_flags)
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


def _row_view(x, shape):
    """The spec_rows of rows [(num_layers,) B, N, heads, head_dim] that _rows gave."""
    strides = x.stride()
    if len(shape) == 4:
        return _abi.spec_rows(x.data_ptr(), 0, strides[0], strides[1], strides[2])
    return _abi.spec_rows(x.data_ptr(), *strides[:4])


_NO_ROWS = _abi.spec_rows(None, 0, 0, 0, 0)
_NO_ROTATION = _abi.spec_rotation(None, 0, 0, 0, 1.0)


@functools.lru_cache(maxsize=256)
def _rotation_layout(dtype, shape, head_dim, interleaved, inverse, amplitude):
    """The spec_rotation of frequencies of this shape."""
    if dtype != torch.float64 or len(shape) != 1 or not 1 <= shape[0] <= min(256, head_dim // 2):
        raise ValueError("frequency must be float64 [dim / 2], dim at most head_dim and 512")
    return _abi.spec_rotation(None, 2 * shape[0], interleaved, inverse, amplitude)


def _rotation(frequency, head_dim, dev, interleaved, inverse, amplitude):
    _on(frequency, dev, "frequency")
    _forward_only(frequency)
    turn = _abi.spec_rotation.from_buffer_copy(_rotation_layout(
        frequency.dtype, frequency.shape, head_dim, bool(interleaved), bool(inverse), float(amplitude)))
    if not frequency.is_contiguous():
        frequency = frequency.contiguous()
    turn.frequency = frequency.data_ptr()
    return frequency, turn


def _append(k_new, v_new, k_cache, v_cache, page_table, context_len, num_new, rotation, return_flags,
            q=None, out=None, position=None):
    """spec_cache_append_rotary; rotation: (frequency, interleaved, amplitude) or None."""
    cache = _cache(k_cache, v_cache, True)
    dev = k_cache.device
    _on(k_new, dev, "k_new")
    _on(v_new, dev, "v_new")
    _forward_only(k_new, v_new)
    shape, D, dtype = k_new.shape, cache.head_dim, k_new.dtype
    if len(shape) != k_cache.dim() or shape[-1] != D or shape[-2] != cache.num_heads or \
            v_new.shape != shape or (len(shape) == 5 and shape[0] != cache.num_layers):
        raise ValueError("k_new and v_new must be [%sB, N, num_heads, head_dim] of the cache's sizes"
                         % ("num_layers, " if k_cache.dim() == 5 else ""))
    if v_new.dtype != dtype or dtype not in _KV_DTYPES or \
            (cache.dtype != _abi.SPEC_Q4 and dtype != k_cache.dtype):
        raise ValueError("k_new and v_new must have the cache's type (float32, bfloat16 or float16 for "
                         "4-bit rows)")
    B, N = shape[-4:-2]
    k_new, v_new = _rows(k_new), _rows(v_new)
    q_rows = out_rows = _NO_ROWS
    heads = 0
    if q is not None:
        _on(q, dev, "q")
        _forward_only(q)
        if q.dtype != dtype or q.dim() != len(shape) or q.shape[:-2] != shape[:-2] or q.shape[-1] != D:
            raise ValueError("q must be [.., B, N, num_q_heads, head_dim] with the type of k_new")
        q = _rows(q)
        if out is None:
            out = torch.empty(q.shape, dtype=dtype, device=dev)
        else:
            _on(out, dev, "out")
            _forward_only(out)
            if out.shape != q.shape or out.dtype != dtype or _rows(out) is not out:
                raise ValueError("out must be like q, with rows on 16 bytes")
        heads = q.shape[-2]
        if heads:
            q_rows, out_rows = _row_view(q, shape), _row_view(out, shape)
    elif out is not None:
        raise ValueError("out is for the rotated q")
    frequency, turn = None, _NO_ROTATION
    if rotation is not None:
        frequency, turn = _rotation(rotation[0], D, dev, rotation[1], False, rotation[2])
    pos_stride = 0
    if position is not None:
        _on(position, dev, "position")
        pos_stride = N if position.dim() == 2 else 0
        position = _ints(position, (B, N) if position.dim() == 2 else (N,), dev, "position")
    page_table, table = _table(page_table, B, dev)
    context_len = _ints(context_len, (B,), dev, "context_len")
    if num_new is not None:
        num_new = _ints(num_new, (B,), dev, "num_new")
    flags = torch.empty(B, dtype=torch.int32, device=dev) if return_flags else None
    _run(dev, _abi.load().spec_cache_append_rotary, q_rows, out_rows, heads, _row_view(k_new, shape),
         _row_view(v_new, shape), _KV_DTYPES[dtype], cache, table, context_len.data_ptr(),
         _ptr(num_new), _ptr(position), pos_stride, B, N, turn, _ptr(flags))
    return flags if q is None else RotaryAppendResult(out, flags)


def cache_append_rotary(k_new, v_new, k_cache, v_cache, page_table, context_len, frequency, q=None,
                        out=None, position=None, num_new=None, interleaved=False, amplitude=1.0,
                        return_flags=False):
    """cache_append with the position rotation on the way (see
    spec_cache_append_rotary): k_new is rotated and written, v_new written, and q, if
    given, rotated.

    The rotation is rotary()'s, by position context_len[b] + position[b, n]; position
    [B, N] or [N], for trees tree_mask()'s position, is 0, 1, .. by default.  q [..,
    B, N, num_q_heads, head_dim] like k_new but for its heads; out: where the rotated
    q goes (q itself: in place).  The cache has the type of k_new, or 4-bit rows.
    Returns RotaryAppendResult with q (None without one) and flags [B] int32 or None.
    """
    result = _append(k_new, v_new, k_cache, v_cache, page_table, context_len, num_new,
                     (frequency, interleaved, amplitude), return_flags, q, out, position)
    return RotaryAppendResult(None, result) if q is None else result


def cache_read(k_cache, v_cache, page_table, start, N, num=None, dtype=None, return_flags=False):
    """Tokens start[b] .. start[b] + N - 1 of each sequence as rows: the inverse of
    cache_append (see spec_cache_read).

    num [B]: only the first num[b] of them; rows that are not there are zeros.  dtype: of
    the rows of a 4-bit cache, bfloat16 by default.  Returns ReadResult with k and v
    [(num_layers,) B, N, num_heads, head_dim] and flags [B] int32 or None.
    """
    cache = _cache(k_cache, v_cache, True)
    dev = k_cache.device
    if cache.dtype == _abi.SPEC_Q4:
        dtype = torch.bfloat16 if dtype is None else dtype
    if dtype is None:
        dtype = k_cache.dtype
    if dtype not in _KV_DTYPES or (cache.dtype != _abi.SPEC_Q4 and dtype != k_cache.dtype):
        raise ValueError("dtype must be the cache's type (float32, bfloat16 or float16 for 4-bit rows)")
    _on(start, dev, "start")
    if start.dim() != 1:
        raise ValueError("start must be [B]")
    B, N = start.shape[0], int(N)
    if not 0 <= N <= 4096:
        raise ValueError("N must be 0..4096")
    start = _ints(start, (B,), dev, "start")
    page_table, table = _table(page_table, B, dev)
    if num is not None:
        num = _ints(num, (B,), dev, "num")
    shape = (B, N, cache.num_heads, cache.head_dim)
    if k_cache.dim() == 5:
        shape = (cache.num_layers, *shape)
    k, v = (torch.empty(shape, dtype=dtype, device=dev) for _ in "kv")
    flags = torch.empty(B, dtype=torch.int32, device=dev) if return_flags else None
    _run(dev, _abi.load().spec_cache_read, cache, table, start.data_ptr(), _ptr(num), B, N,
         _KV_DTYPES[dtype], _row_view(k, shape), _row_view(v, shape), _ptr(flags))
    return ReadResult(k, v, flags)


def cache_4bit(num_pages, page_size, num_heads, head_dim, num_layers=None, device="cuda"):
    """An empty cache of 4-bit rows: k and v, uint8 [(num_layers,) num_pages, page_size,
    num_heads, head_dim / 2 + 16], with a head's tokens of a page one behind another: with
    pages of a power of two tokens, the layout that attention reads fastest."""
    if head_dim not in (64, 128):
        raise ValueError("4-bit caches have head_dim 64 or 128")
    lead = (num_pages,) if num_layers is None else (num_layers, num_pages)
    shape = (*lead, num_heads, page_size, head_dim // 2 + 16)
    return tuple(torch.zeros(shape, dtype=torch.uint8, device=device).transpose(-3, -2) for _ in "kv")


def rotary_frequency(dim, base=10000.0, scaling=None, factor=1.0, context=4096, low=1.0, high=32.0,
                     device="cuda"):
    """Frequencies of a rotation of dim values: RotaryFrequency with frequency float64
    [dim / 2], base^(-2i/dim) radians per token, and the amplitude that goes with it.

    scaling, for contexts `factor` times longer than the `context` tokens that a model
    was trained on:
      None       as they are
      "linear"   divided by factor
      "base"     base times factor^(dim / (dim - 2)): the longest wave is factor times
                 longer, the shortest stays
      "turns"    pairs that turn less than `low` times over the context are divided by
                 factor, those that turn more than `high` times kept, the others mixed
                 in proportion to their turns
      "index"    the same, mixed in proportion to the pairs' index, with amplitude
                 0.1 ln(factor) + 1
    """
    dim = int(dim)
    if dim < 2 or dim % 2 or not base > 1.0 or not factor >= 1.0:
        raise ValueError("dim must be even, base above 1, factor at least 1")
    if scaling in ("turns", "index") and not (context > 0 and 0 < low < high):
        raise ValueError("context and 0 < low < high are needed")
    if scaling == "base" and dim > 2:
        base = base * factor ** (dim / (dim - 2))
    i = torch.arange(0, dim, 2, dtype=torch.float64)
    f = torch.tensor(float(base), dtype=torch.float64) ** (-i / dim)
    amplitude = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "turns":
        turns = f * (context / (2 * math.pi))
        keep = ((turns - low) / (high - low)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
    elif scaling == "index":
        # the index of a pair with so many turns over the context
        at = [dim * math.log(context / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (high, low)]
        first, last = max(math.floor(at[0]), 0), min(math.ceil(at[1]), dim - 1)
        keep = 1 - ((i / 2 - first) / max(last - first, 1e-3)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
        amplitude = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "base"):
        raise ValueError("scaling must be None, 'linear', 'base', 'turns' or 'index'")
    return RotaryFrequency(f.to(device), amplitude)


@functools.lru_cache(maxsize=512)
def _rotary_rows(dtype, shape, strides):
    """Of heads to rotate, their type's code, B, N, heads, head_dim and the spec_rows of
    tensors with these strides; None where rows are not apart, or their last dimension is
    not contiguous."""
    code, dims = _KV_DTYPES.get(dtype), len(shape)
    if code is None or not 2 <= dims <= 4:
        raise ValueError("x must be [B, N, heads, D], [N, heads, D] or [heads, D], float32, bfloat16 or "
                         "float16")
    _sizes(shape)
    lead = 4 - dims
    rows = None
    if strides[-1] == 1 and all(n <= 1 or s >= shape[-1] for n, s in zip(shape[:-1], strides[:-1])):
        rows = _abi.spec_rows(None, 0, *(0,) * lead, *strides[:-1])
    return code, ((1,) * lead + tuple(shape)), rows


def rotary(x, position, frequency, interleaved=False, amplitude=1.0, inverse=False, out=None):
    """Rotates heads by their tokens' positions (see spec_rotary).

    x [B, N, heads, D], [N, heads, D] or [heads, D], float32, bfloat16 or float16;
    position: integers of x's shape without its last two dimensions, or [N] for all
    sequences (beyond 32 bits: as their largest or smallest).  frequency float64 [dim / 2], radians per token (rotary_frequency); the
    values of a head behind the first dim are copied.  Pairs are (i, i + dim / 2), or
    interleaved (2i, 2i + 1).  amplitude: a factor of the rotated values.  inverse:
    turns back (with amplitude 1 the inverse, and the gradient).  out: where the
    result goes (x itself: in place).  Returns the rotated rows.
    """
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    _forward_only(x)
    dev, shape = x.device, x.shape
    code, sizes, rows = _rotary_rows(x.dtype, shape, x.stride())
    frequency, turn = _rotation(frequency, sizes[3], dev, interleaved, inverse, amplitude)
    _on(position, dev, "position")
    pos_stride = 0
    if len(shape) == 4 and position.dim() == 1:
        position = _ints(position, shape[1:2], dev, "position")
    else:
        position = _ints(position, shape[:-2], dev, "position")
        if len(shape) == 4:
            pos_stride = sizes[1]
    if rows is None:
        x = x.clone(memory_format=torch.contiguous_format)
        rows = _rotary_rows(x.dtype, shape, x.stride())[2]
    if out is None:
        out = torch.empty(shape, dtype=x.dtype, device=dev)
        out_rows = _rotary_rows(x.dtype, shape, out.stride())[2]
    else:
        _on(out, dev, "out")
        _forward_only(out)
        out_rows = None
        if out.shape == shape and out.dtype == x.dtype:
            out_rows = _rotary_rows(x.dtype, shape, out.stride())[2]
        if out_rows is None:
            raise ValueError("out must be like x, its last dimension contiguous")
    if x.numel():
        x_view, out_view = (_abi.spec_rows.from_buffer_copy(r) for r in (rows, out_rows))
        x_view.data, out_view.data = x.data_ptr(), out.data_ptr()
        _run(dev, _abi.load().spec_rotary, x_view, out_view, code, *sizes, position.data_ptr(), pos_stride, turn)
    return out


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
