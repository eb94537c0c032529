"""The operators between a block's linears, from their definitions in binary64.

Inputs are float64 arrays holding whatever values the GPU tensors hold; nothing
is rounded here.  Shares no code with the library.
"""

import numpy as np


def normalise(v, kind, eps):
    """Layer or RMS norm over the last axis; kind "none" returns v."""
    if kind == "none":
        return v
    c = v - v.mean(-1, keepdims=True) if kind == "layer" else v
    return c / np.sqrt((c * c).mean(-1, keepdims=True) + eps)


def gated_norm(x, y=None, gate=None, scale=None, shift=None, norm="layer", weight=None, bias=None,
               post_norm="none", post_weight=None, residual_scale=1.0, eps=1e-6):
    """x, y [batch, tokens, channels]; gate, scale, shift [batch, channels].  Returns (r, h)."""
    r = x
    if y is not None:
        z = normalise(y, post_norm, eps)
        if post_weight is not None:
            z = z * post_weight
        if gate is not None:
            z = z * gate[:, None, :]
        r = residual_scale * x + z
    h = normalise(r, norm, eps)
    if weight is not None:
        h = h * weight
    if bias is not None:
        h = h + bias
    if scale is not None:
        h = h * (1.0 + scale[:, None, :])
    if shift is not None:
        h = h + shift[:, None, :]
    return r, h


def rotary(v, positions, radians, axis, rotary_dim, layout="interleaved", magnitude=1.0,
           weight=None, eps=1e-6):
    """v [batch, tokens, heads, dim]; positions [batch, tokens, axes] integers;
    radians / axis per pair.  One complex product per pair."""
    z = v if weight is None else normalise(v, "rms", eps) * weight
    out = z.copy()
    for j, (f, ax) in enumerate(zip(radians, axis)):
        turn = magnitude * np.exp(1j * (positions[:, :, ax].astype(np.float64) * f))[:, :, None]
        a, b = (2 * j, 2 * j + 1) if layout == "interleaved" else (j, j + rotary_dim // 2)
        w = (z[..., a] + 1j * z[..., b]) * turn
        out[..., a], out[..., b] = w.real, w.imag
    return out


def attention(q, k, v, visible, scale):
    """q [batch, queries, heads, dim]; k, v [batch, keys, kv_heads, dim]; visible
    [batch, keys] booleans.  Keys out of sight are left out of every sum (they
    may hold anything); a query with none left gets zeros.  Returns the output
    and the same sum over |v|."""
    out, size = np.zeros(q.shape), np.zeros(q.shape)
    group = q.shape[2] // k.shape[2]
    for b in range(q.shape[0]):
        at = np.flatnonzero(visible[b])
        if not at.size:
            continue
        for h in range(q.shape[2]):
            s = (q[b, :, h] @ k[b, at, h // group].T) * scale
            w = np.exp(s - s.max(1, keepdims=True))
            w /= w.sum(1, keepdims=True)
            out[b, :, h] = w @ v[b, at, h // group]
            size[b, :, h] = w @ np.abs(v[b, at, h // group])
    return out, size


def lora_add(y, x, down, up, ids, scales=None):
    """y + s_a up_a (down_a x) per row, a = ids[row] (rows with an id outside the
    adapters: y).  Returns the sum and, per element, sum_j |up| s |down| |x|
    taken over both products (the size of its terms)."""
    out, size = y.copy(), np.zeros(y.shape)
    for a in range(down.shape[0]):
        m = ids == a
        s = 1.0 if scales is None else scales[a]
        out[m] += s * (x[m] @ down[a].T) @ up[a].T
        size[m] = abs(s) * (np.abs(x[m]) @ np.abs(down[a]).T) @ np.abs(up[a]).T
    return out, size


def lora_rank_size(x, down, up, ids, scales=None):
    """Per element sum_j |up_j| |s t_j|: the size of the second product's terms."""
    size = np.zeros((x.shape[0], up.shape[1]))
    for a in range(down.shape[0]):
        m = ids == a
        s = 1.0 if scales is None else scales[a]
        size[m] = np.abs(s * (x[m] @ down[a].T)) @ np.abs(up[a]).T
    return size
