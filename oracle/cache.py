"""A key/value cache held in NVFP4, from its definition.

What a cache holds is kept here as plain arrays per position; pages are looked up one
position at a time.  Attention is in binary64, one row at a time.  Shares no code with
the library.
"""

import numpy as np

from .quant import dequantize, quantize
from .formats import e2m1_value, e4m3_value

_E2M1 = np.array([float(e2m1_value(c)) for c in range(16)])
_E4M3 = np.append(np.array([float(e4m3_value(b)) for b in range(127)]), np.nan)


def quantized_rows(bits, amax):
    """bf16 bit patterns [..., dim] -> (codes [..., dim/2], scales [..., dim/16],
    tensor scale) under a static amax; a 16-block with a non-finite element has the
    scale byte 0x7F and zero codes."""
    dim = bits.shape[-1]
    blocks = np.ascontiguousarray(bits).reshape(-1, 16).copy()
    bad = ((blocks & 0x7FFF) >= 0x7F80).any(1)
    blocks[bad] = 0
    q = quantize(blocks, amax=np.float32(amax))
    scales = np.where(bad, 0x7F, q.scales[:, 0]).astype(np.uint8)
    return (q.codes.reshape(*bits.shape[:-1], dim // 2), scales.reshape(*bits.shape[:-1], dim // 16),
            q.tensor_scale)


def held(codes, scales, tensor_scale):
    """The numbers that codes and scales stand for, in binary64."""
    v = np.stack([_E2M1[codes & 15], _E2M1[codes >> 4]], -1).reshape(*codes.shape[:-1], -1)
    return v * np.repeat(_E4M3[scales], 16, -1) * float(tensor_scale)


def read_bits(codes, scales, tensor_scale):
    """The bf16 bit patterns that a row reads as (finite scales)."""
    dim = 2 * codes.shape[-1]
    return dequantize(codes.reshape(-1, dim // 2), scales.reshape(-1, dim // 16), tensor_scale, dim).reshape(
        *codes.shape[:-1], dim)


def place(table, page_size, pages, entry, position):
    """(page, place in it) of an entry's position, None if it has none."""
    if position < 0:
        return None
    if table is None:
        return (entry, position) if position < page_size else None
    if position // page_size >= table.shape[1]:
        return None
    page = int(table[entry, position // page_size])
    return (page, position % page_size) if 0 <= page < pages else None


def attention(q, k, v, visible, scale):
    """q [queries, heads, dim]; k, v [keys, kv_heads, dim]; visible [queries, keys].
    Returns the output and the same sum over |v|; zeros where nothing is visible."""
    out, size = np.zeros(q.shape), np.zeros(q.shape)
    group = q.shape[1] // k.shape[1]
    for t in range(q.shape[0]):
        seen = np.flatnonzero(visible[t])
        if seen.size == 0:
            continue
        for h in range(q.shape[1]):
            s = scale * (k[seen, h // group] @ q[t, h])
            w = np.exp(s - s.max())
            w /= w.sum()
            out[t, h] = w @ v[seen, h // group]
            size[t, h] = w @ np.abs(v[seen, h // group])
    return out, size
