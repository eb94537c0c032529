"""Helpers of the tests of the NVFP4 key/value cache: caches filled by hand, their
numbers in binary64, and the bound of attention over them."""

import numpy as np
import torch

import nvfp4_block_scaled_05_amd as nv
import oracle.cache as oc
from tests.block_util import U32, UBF, f64
from tests.gpu_util import bits_of

UH = 2.0 ** -11            # half a step of fp16, relative

K_AMAX, V_AMAX = 9.0, 5.0


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def filled(rng, pages, page_size, kv_heads, dim, std=1.0, k_amax=K_AMAX, v_amax=V_AMAX):
    """A cache whose every place holds quantized normal numbers, and the numbers
    [pages, page_size, kv_heads, dim] of keys and values."""
    cache = nv.kv_cache(pages, page_size, kv_heads, dim, k_amax, v_amax)
    numbers = []
    for codes, scales, amax in ((cache.k_codes, cache.k_scales, k_amax), (cache.v_codes, cache.v_scales, v_amax)):
        x = torch.from_numpy(rng.standard_normal((pages, kv_heads, page_size, dim)) * std).to(torch.bfloat16)
        c, s, ts = oc.quantized_rows(x.view(torch.int16).numpy().view(np.uint16), amax)
        codes.copy_(torch.from_numpy(c))
        scales.copy_(torch.from_numpy(s))
        numbers.append(oc.held(c, s, ts).transpose(0, 2, 1, 3))
    return cache, numbers[0], numbers[1]


def numbers_of(cache):
    """The numbers [pages, page_size, kv_heads, dim] that a cache holds now."""
    out = []
    for i, (codes, scales) in enumerate(((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales))):
        ts = np.float32(1.0) / (np.float32(2688.0) / np.float32(cache.amax[i].item()))
        out.append(oc.held(codes.cpu().numpy(), scales.cpu().numpy(), ts).transpose(0, 2, 1, 3))
    return out


def shuffled_table(rng, batch, per, pages):
    return rng.permutation(pages)[:batch * per].reshape(batch, per).astype(np.int32)


def rows_of(numbers, table, entry, n):
    """[n, kv_heads, dim]: an entry's first n positions; NaN where it has no page."""
    pages, page_size = numbers.shape[:2]
    out = np.full((n, *numbers.shape[2:]), np.nan)
    for j in range(n):
        at = oc.place(table, page_size, pages, entry, j)
        if at is not None:
            out[j] = numbers[at]
    return out


def expected(q, k, v, lengths, starts=None, table=None, scale=None):
    """(want, bound) of cache_attention; q float64 [batch, queries, heads, dim], k, v
    the numbers of the pages.

    Bounds, relative to W = sum_j w_j |v_j|: each weight is rounded to fp16 (UH, or
    2^-32 of the row's largest where that is less); a score is a binary32 sum of dim
    exact products and a few more roundings, off by d = (dim + 8) U32 scale sum |q k|,
    which changes a weight by at most 2 d relative; the weights' and outputs' binary32
    sums and the exponentials add (keys + 64) U32.  The output rounding is UBF of the
    value."""
    batch, queries, heads, dim = q.shape
    scale = scale or dim ** -0.5
    want, bound = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(batch):
        n = int(lengths[b])
        kk, vv = rows_of(k, table, b, n), rows_of(v, table, b, n)
        on_page = ~np.isnan(kk).all((1, 2))
        visible = np.broadcast_to(on_page, (queries, n)).copy()
        if starts is not None:
            visible &= np.arange(n) <= int(starts[b]) + np.arange(queries)[:, None]
        want[b], size = oc.attention(q[b], kk, vv, visible, scale)
        if not on_page.any():
            continue
        most = np.abs(q[b]).sum(-1).max() * np.abs(kk[on_page]).max()
        d = (dim + 8) * U32 * scale * most
        bound[b] = (UBF * np.abs(want[b]) + (UH + 2 * d + (n + 64) * U32) * size
                    + n * 2.0 ** -32 * np.abs(vv[on_page]).max() * visible.any(1)[:, None, None])
    return want, bound


def check(got, q, k, v, lengths, starts=None, table=None, scale=None):
    want, bound = expected(f64(q), k, v, lengths, starts, table, scale)
    g = f64(got)
    assert g.shape == want.shape
    assert np.isfinite(g).all(), f"{np.count_nonzero(~np.isfinite(g))} non-finite"
    off = np.abs(g - want) - bound
    if g.size and off.max() > 0:
        i = np.unravel_index(off.argmax(), off.shape)
        raise AssertionError(f"at {i}: got {g[i]!r}, want {want[i]!r}, bound {bound[i]:.3e}; "
                             f"{np.count_nonzero(off > 0)} of {g.size} outside")


def raw(t):
    return bits_of(t)
