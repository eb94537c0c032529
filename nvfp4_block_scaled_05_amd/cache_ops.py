"""A key/value cache held in NVFP4: Python face of the kv_cache_* entry points of
include/nvfp4.h, with the argument checks of the package.

A cache is four uint8 tensors and the static amax of its keys and values.  Its pages
may be handed out by a table, [batch, pages of an entry] int32 in order, so entries of
unequal lengths share one pool; without a table entry b is page b.  Calls are enqueued
on the current stream; everything is forward only.
"""

import math
import struct
from collections import namedtuple

from . import _NO_WORKSPACE, _opt, _ptr, _tensor, _torch
from ._binding import Nvfp4Error, load
from .block_ops import _VIEW, _heads, _new_heads, _out_heads, _place, _stream_at

#: codes uint8 [pages, kv_heads, page_size, dim / 2] and E4M3 scales uint8
#: [pages, kv_heads, page_size, dim / 16] of keys and of values; amax float32 [2]
KvCache = namedtuple("KvCache", ["k_codes", "k_scales", "v_codes", "v_scales", "amax"])

#: the kv_cache of the C ABI, as bytes
_CACHE = struct.Struct("@5P4qPq").pack

#: the amax with which a tensor's scale is 1: block scales alone cover 2^-9 to 448
UNIT_AMAX = 2688.0


def kv_cache(pages, page_size, kv_heads, dim, k_amax=UNIT_AMAX, v_amax=UNIT_AMAX, device="cuda"):
    """A zeroed cache of ``pages`` pages of ``page_size`` tokens (a multiple of 16; a
    power of two where a table names the pages); dim: a multiple of 16 up to 128.

    k_amax, v_amax: the static amax of keys and values, from calibration (or a bound:
    a key norm's); larger elements saturate.  They are kept on the device, in
    ``cache.amax``, and may be set there (to a producer's amax) before the first write.
    """
    torch = _torch()
    if pages <= 0 or kv_heads <= 0 or page_size <= 0 or page_size % 16:
        raise ValueError("pages and kv_heads must be positive, page_size a positive multiple of 16; "
                         f"got {pages}, {kv_heads}, {page_size}")
    if dim <= 0 or dim % 16 or dim > 128:
        raise ValueError(f"dim must be a positive multiple of 16 up to 128, got {dim}")
    for name, v in (("k_amax", k_amax), ("v_amax", v_amax)):
        if not (2.0 ** -96 <= v <= 2.0 ** 96):
            raise ValueError(f"{name} must be in [2^-96, 2^96], got {v}")

    def zeros(n):
        return torch.zeros((pages, kv_heads, page_size, n), dtype=torch.uint8, device=device)

    return KvCache(zeros(dim // 2), zeros(dim // 16), zeros(dim // 2), zeros(dim // 16),
                   torch.tensor([k_amax, v_amax], dtype=torch.float32, device=device))


def _check_cache(cache):
    """Raises ValueError for what is not a cache."""
    torch = _torch()
    if not isinstance(cache, KvCache):
        raise ValueError("cache: expected a KvCache (kv_cache)")
    codes = cache.k_codes
    if not isinstance(codes, torch.Tensor) or codes.dim() != 4:
        raise ValueError("cache.k_codes: expected a 4-D torch.Tensor")
    pages, kv_heads, page_size, half = shape = codes.shape
    dim = 2 * half
    if pages <= 0 or kv_heads <= 0 or page_size <= 0 or page_size % 16 or dim <= 0 or dim % 16 or dim > 128:
        raise ValueError(f"cache.k_codes: shape {tuple(shape)} is not that of a cache (kv_cache)")
    scales = (pages, kv_heads, page_size, dim // 16)
    for name, t, want in (("k_codes", codes, shape), ("k_scales", cache.k_scales, scales),
                          ("v_codes", cache.v_codes, shape), ("v_scales", cache.v_scales, scales)):
        _tensor(t, f"cache.{name}", torch.uint8, want)
    _tensor(cache.amax, "cache.amax", torch.float32, (2,))


def _cache(cache, table, batch):
    """(batch, kv_heads, dim, capacity) and the C view of a cache whose table serves
    ``batch`` entries (None: as many as it has)."""
    torch = _torch()
    u8 = torch.uint8
    # what is common takes one look, as in block_ops
    try:
        kc, ks, vc, vs, amax = cache
        shape = kc.shape
        pages, kv_heads, page_size, half = shape
        dim = 2 * half
        good = (type(cache) is KvCache and kc.dtype is u8 and ks.dtype is u8 and vc.dtype is u8 and vs.dtype is u8
                and amax.dtype is torch.float32 and kc.is_contiguous() and ks.is_contiguous()
                and vc.is_contiguous() and vs.is_contiguous() and amax.is_contiguous() and vc.shape == shape
                and ks.shape == vs.shape == (pages, kv_heads, page_size, half >> 3) and amax.shape == (2,)
                and kc.numel() > 0 and not (page_size | dim) & 15 and dim <= 128)
    except (AttributeError, TypeError, ValueError):
        good = False
    if not good:
        _check_cache(cache)
    if table is None:
        if batch is None:
            batch = pages
        if batch > pages:
            raise ValueError(f"{batch} entries, but the cache has {pages} pages (no table is given)")
        per, at, capacity = 0, 0, page_size
    else:
        if not isinstance(table, torch.Tensor) or table.dim() != 2:
            raise ValueError("table: expected a 2-D torch.Tensor")
        rows, per = table.shape
        if batch is None:
            batch = rows
        if table.dtype is not torch.int32 or rows != batch or not table.is_contiguous():
            _tensor(table, "table", torch.int32, (batch, per), 0)
        if page_size & (page_size - 1):
            raise ValueError(f"a table needs a page size that is a power of two, got {page_size}")
        if per == 0:
            raise ValueError("table: needs a page for each entry at least")
        at, capacity = table.data_ptr(), per * page_size
    return batch, kv_heads, dim, capacity, _CACHE(kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(),
                                                  amax.data_ptr(), pages, page_size, kv_heads, dim, at, per)


def _entries(t, name, batch, optional=True):
    if t is None and optional:
        return
    torch = _torch()
    if (not isinstance(t, torch.Tensor) or t.dtype is not torch.int32 or t.dim() != 1 or t.shape[0] != batch
            or not t.is_contiguous()):
        _tensor(t, name, torch.int32, (batch,), 0)


def cache_write(cache, k, v, starts, counts=None, table=None, dev_status=None):
    """Quantize new tokens into the cache: token t of entry b becomes its position
    starts[b] + t, for t < counts[b].  The bytes are those of ``quantize`` on that
    head's row with the cache's amax.

    k, v: bf16 [tokens, kv_heads, dim] or [batch, tokens, kv_heads, dim]; views of a
    fused projection are taken as they are.  starts, counts: int32 [batch] (counts
    None: all tokens).  table: int32 [batch, pages of an entry], or None.  Positions
    past the entry's pages, below 0 or on no page of the cache are dropped; what else
    the cache holds is left as it is.  No two tokens of a call may have one place.

    A block that holds an infinity or NaN reads back as NaN; dev_status: optional
    one-element int32 device tensor, set to 0, or to the status of non-finite input.
    """
    torch = _torch()
    (batch, tokens, heads, dim), kv = _heads(k, "k")
    v_shape, vv = _heads(v, "v")
    if v.dim() != k.dim() or v_shape != (batch, tokens, heads, dim):
        raise ValueError(f"k, v: shapes {tuple(k.shape)}, {tuple(v.shape)} do not go together")
    _, kv_heads, cache_dim, _, view = _cache(cache, table, batch)
    if (heads, dim) != (kv_heads, cache_dim):
        raise ValueError(f"k: {heads} heads of {dim}, the cache has {kv_heads} of {cache_dim}")
    _entries(starts, "starts", batch, optional=False)
    _entries(counts, "counts", batch)
    _opt(dev_status, "dev_status", torch.int32)
    at = _place((k, v, cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales, cache.amax, starts,
                 counts, table, dev_status),
                "k v cache.k_codes cache.k_scales cache.v_codes cache.v_scales cache.amax starts counts "
                "table dev_status")
    status = load().kv_cache_write(view, kv, vv, batch, tokens, _ptr(starts), _ptr(counts),
                                   _ptr(dev_status), _stream_at(at))
    if status:
        raise Nvfp4Error(status, "kv_cache_write")


def cache_read(cache, tokens, starts=None, counts=None, table=None, out=None):
    """The keys and values of positions starts[b] + t, t < tokens, as bf16 tensors
    [batch, tokens, kv_heads, dim]: what ``dequantize`` gives.  Zeros from counts[b] on,
    and for positions past the entry's pages, below 0 or on no page of the cache.

    starts, counts: int32 [batch] or None (0; all tokens).  out: optional (k, v) to
    write into, all of it.  Returns (k, v).
    """
    torch = _torch()
    batch = None
    for t in (starts, counts):
        if isinstance(t, torch.Tensor) and t.dim() == 1:
            batch = t.shape[0]
    batch, kv_heads, dim, _, view = _cache(cache, table, batch)
    if tokens < 0:
        raise ValueError(f"tokens must not be negative, got {tokens}")
    _entries(starts, "starts", batch)
    _entries(counts, "counts", batch)
    shape = (batch, tokens, kv_heads, dim)
    if out is not None:
        if not isinstance(out, (tuple, list)) or len(out) != 2:
            raise ValueError("out: expected a tuple of 2 tensors")
        views = []
        for t, name in zip(out, ("out k", "out v")):
            got, one = _heads(t, name, out=True)
            if t.dim() != 4 or got != shape:
                raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape}")
            views.append(one)
        if out[0].data_ptr() == out[1].data_ptr() and out[0].numel():
            raise ValueError("out k and out v are the same buffer")
        k, v = out
        kv, vv = views
    else:
        k = v = None
    at = _place((cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales, cache.amax, starts, counts,
                 table, k, v),
                "cache.k_codes cache.k_scales cache.v_codes cache.v_scales cache.amax starts counts table "
                "out_k out_v")
    if out is None:
        k = cache.amax.new_empty(shape, dtype=torch.bfloat16)
        v, vv = _new_heads(k, shape)
        kv = _VIEW(k.data_ptr(), tokens * kv_heads * dim, kv_heads * dim, dim)
    status = load().kv_cache_read(view, kv, vv, batch, tokens, _ptr(starts), _ptr(counts), _stream_at(at))
    if status:
        raise Nvfp4Error(status, "kv_cache_read")
    return k, v


def cache_attention_workspace(batch, queries, heads, kv_heads, dim, capacity, device="cuda"):
    """A workspace for ``cache_attention`` on these sizes (capacity: the positions of an
    entry, its pages times their size), or None if it would not split the keys."""
    nbytes = load().kv_cache_attention_workspace_bytes(batch, queries, heads, kv_heads, dim, capacity)
    if nbytes == 0:
        return None
    return _torch().empty(nbytes, dtype=_torch().uint8, device=device)


def cache_attention(q, cache, lengths, starts=None, table=None, scale=None, out=None,
                    workspace=_NO_WORKSPACE):
    """softmax(scale q k^T) v over what the cache holds.

    q: bf16 [queries, heads, dim] or [batch, queries, heads, dim]; the cache's heads
    divide q's (query heads share key heads in order).  lengths: int32 [batch], the
    positions that each entry holds.  starts: int32 [batch] or None: the position of
    each entry's first query; query t then sees positions up to starts[b] + t, its own,
    else all of them.  table: as for ``cache_write``.  A query that sees no key, or
    whose scores are all -infinity, gets zeros; what lies out of sight does not count,
    whatever it holds.  scale: dim ** -0.5 by default.  out: overlaps no input.

    ``workspace``: a uint8 device tensor from ``cache_attention_workspace`` (reused
    across calls on one stream), None not to split any entry's keys, or left out to
    have one taken from torch's caching allocator for this call.
    """
    torch = _torch()
    (batch, queries, heads, dim), qv = _heads(q, "q")
    _, kv_heads, cache_dim, capacity, view = _cache(cache, table, batch)
    if dim != cache_dim:
        raise ValueError(f"q: head size {dim}, the cache has {cache_dim}")
    if heads <= 0 or heads % kv_heads:
        raise ValueError(f"q has {heads} heads, not a positive multiple of the cache's {kv_heads}")
    if scale is None:
        scale = dim ** -0.5
    if not (scale > 0 and math.isfinite(scale)):
        raise ValueError(f"scale must be positive, got {scale}")
    _entries(lengths, "lengths", batch, optional=False)
    _entries(starts, "starts", batch)
    ov = _out_heads(out, q, "out")
    ws = None if workspace is _NO_WORKSPACE else _opt(workspace, "workspace", torch.uint8)
    at = _place((q, cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales, cache.amax, lengths, starts,
                 table, out, ws),
                "q cache.k_codes cache.k_scales cache.v_codes cache.v_scales cache.amax lengths starts table "
                "out workspace")
    if out is None:
        out, ov = _new_heads(q, (batch, queries, heads, dim))
    lib = load()
    ws_bytes = 0
    if workspace is _NO_WORKSPACE:
        ws_bytes = lib.kv_cache_attention_workspace_bytes(batch, queries, heads, kv_heads, dim, capacity)
        if ws_bytes:
            ws = q.new_empty((ws_bytes,), dtype=torch.uint8)
    elif ws is not None:
        ws_bytes = ws.numel()
    status = lib.kv_cache_attention(view, qv, _ptr(lengths), _ptr(starts), batch, queries, heads, scale,
                                    ov, _ptr(ws), ws_bytes, _stream_at(at))
    if status:
        raise Nvfp4Error(status, "kv_cache_attention")
    return out
