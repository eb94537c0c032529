"""The operators between a block's linears: Python face of the dit_* entry
points of include/nvfp4.h, with the argument checks of the package.

Tensors are bf16 on the current HIP device unless said otherwise, calls are
enqueued on the current stream, and outputs that are not passed in are
allocated with torch.  Everything is forward only: no output carries a
gradient.
"""

import math
import struct
from collections import namedtuple

from . import _NO_WORKSPACE, _device, _epilogue, _matrix, _opt, _ptr, _stream, _tensor, _torch
from ._binding import Nvfp4Error, load

NORMS = {"none": 0, "layer": 1, "rms": 2}
ROTARY_LAYOUTS = {"interleaved": 0, "half": 1}
ROTARY_SCALINGS = ("none", "linear", "ntk", "yarn")


# These calls take a few microseconds on the GPU when they are small, and their
# checks have to cost no more than that: what is common (everything given is right
# and on the current device) is a comparison or two a tensor, and names and
# messages are put together only for an error.

_CURRENT_DEVICE = None
_RAW_STREAM = None


def _place(tensors, names):
    """_device on some tensors (None skipped, the first given).  Returns the
    index of their device, which is the current one."""
    global _CURRENT_DEVICE
    at = tensors[0].get_device()
    good = at >= 0
    for t in tensors:
        if t is not None and t.get_device() != at:
            good = False
    if good:
        if _CURRENT_DEVICE is None:
            torch = _torch()
            torch.cuda.current_device()                      # initialises the device API
            _CURRENT_DEVICE = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        good = _CURRENT_DEVICE() == at
    if not good:
        _device(**dict(zip(names.split(), tensors)))         # raises, with the name
    return at


def _stream_at(at):
    """The current stream of device ``at``, the current one."""
    global _RAW_STREAM
    if _RAW_STREAM is None:
        _RAW_STREAM = getattr(_torch()._C, "_cuda_getCurrentRawStream", False)
    return _RAW_STREAM(at) if _RAW_STREAM else _stream()


def _like(t, name, dtype, shape):
    """_tensor for a torch.Size that is at hand; an error takes the long way."""
    if (not isinstance(t, _torch().Tensor) or t.dtype != dtype or t.shape != shape
            or not t.is_contiguous()):
        _tensor(t, name, dtype, shape, 0)


def _choice(value, choices, name):
    if value not in choices:
        raise ValueError(f"{name} must be one of {sorted(choices)}, got {value!r}")
    return choices[value]


def _rows3(t, name):
    """(batch, tokens, channels) of a [tokens, channels] or [batch, tokens, channels] tensor."""
    if not isinstance(t, _torch().Tensor) or t.dim() not in (2, 3):
        raise ValueError(f"{name}: expected a 2-D or 3-D torch.Tensor")
    return t.shape if t.dim() == 3 else (1, *t.shape)


def _vector(t, name, shape, dtype):
    """The stride of a [batch, channels] tensor whose rows are dense (a chunk of
    a wider one), after its checks."""
    if not isinstance(t, _torch().Tensor) or t.shape != shape:
        raise ValueError(f"{name}: expected a torch.Tensor of shape {shape}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    row, dense = t.stride()
    if dense != 1 and shape[1] > 1:
        raise ValueError(f"{name}: the last dimension must be dense (got strides {(row, dense)})")
    return row if shape[0] > 1 else 0


def gated_norm(x, y=None, gate=None, scale=None, shift=None, norm="layer", weight=None, bias=None,
               post_norm="none", post_weight=None, residual_scale=1.0, eps=1e-6, amax=None,
               out=None, residual_out=None):
    """The gate and residual after a linear and the norm before the next, in one pass:

        r = residual_scale * x + gate * z,  z = y or post_norm(y) * post_weight
        h = (norm(r) * weight + bias) * (1 + scale) + shift

    x: [tokens, channels] or [batch, tokens, channels], bf16 or float32 (the
    residual stream); y: bf16 of the same shape, or None (r is x).  gate, scale,
    shift: [batch, channels] (batch 1 for a 2-D x), all bf16 or all float32, dense
    rows of any stride that is a multiple of 8, so chunks of the modulation
    linear's output are taken as they are.  weight, bias, post_weight: float32
    [channels].  norm, post_norm: "none", "layer" or "rms"; norm None: only r
    is wanted (the last residual of a model), h is None.  amax: optional
    one-element float32 device tensor, set to max |h| for ``quantize``.

    Returns (r, h): r in x's type (x itself when there is no y), h in bf16.
    ``residual_out`` may be x, ``out`` may be y, no other overlap; channels: a multiple of 8, at
    most 16384.
    """
    torch = _torch()
    batch, tokens, channels = _rows3(x, "x")
    fp32 = x.dtype == torch.float32
    _tensor(x, "x", torch.float32 if fp32 else torch.bfloat16, min_numel=0)
    if channels <= 0 or channels % 8 or channels > 16384:
        raise ValueError(f"x: channels must be a positive multiple of 8 up to 16384, got {channels}")
    norm_id = NORMS["none"] if norm is None else _choice(norm, NORMS, "norm")
    post_id = _choice(post_norm, NORMS, "post_norm")
    if y is None:
        for name, v in (("gate", gate), ("post_weight", post_weight), ("residual_out", residual_out)):
            if v is not None:
                raise ValueError(f"{name} needs y")
        if post_id or residual_scale != 1.0:
            raise ValueError("post_norm and residual_scale need y")
    if norm is None:
        for name, v in (("scale", scale), ("shift", shift), ("weight", weight), ("bias", bias),
                        ("amax", amax), ("out", out)):
            if v is not None:
                raise ValueError(f"{name} needs a norm")
        if y is None:
            raise ValueError("norm None needs y")
    if not (eps > 0 and math.isfinite(eps) and math.isfinite(residual_scale)):
        raise ValueError(f"eps must be positive, residual_scale finite; got {eps}, {residual_scale}")
    shape = x.shape
    if y is not None:
        _like(y, "y", torch.bfloat16, shape)
    mod = None                                # the type of the first vector; all have it
    g_stride = sc_stride = sh_stride = 0
    for v in (gate, scale, shift):
        if v is not None:
            mod = getattr(v, "dtype", None)
            if mod not in (torch.bfloat16, torch.float32):
                raise ValueError(f"gate, scale, shift: dtype {mod}, expected bfloat16 or float32")
            break
    if gate is not None:
        g_stride = _vector(gate, "gate", (batch, channels), mod)
    if scale is not None:
        sc_stride = _vector(scale, "scale", (batch, channels), mod)
    if shift is not None:
        sh_stride = _vector(shift, "shift", (batch, channels), mod)
    for v, name in ((weight, "weight"), (bias, "bias"), (post_weight, "post_weight")):
        if v is not None:
            _tensor(v, name, torch.float32, (channels,))
    if amax is not None:
        _tensor(amax, "amax", torch.float32)
    if out is not None:
        _like(out, "out", torch.bfloat16, shape)
    if residual_out is not None:
        _like(residual_out, "residual_out", x.dtype, shape)
        if out is not None and out.data_ptr() == residual_out.data_ptr() and x.numel():
            raise ValueError("out and residual_out are the same buffer")
    at = _place((x, y, gate, scale, shift, weight, bias, post_weight, amax, out, residual_out),
                "x y gate scale shift weight bias post_weight amax out residual_out")
    if out is None and norm is not None:
        out = torch.empty_like(x, dtype=torch.bfloat16) if fp32 else torch.empty_like(x)
    if residual_out is None and y is not None:
        residual_out = torch.empty_like(x)
    status = load().dit_gated_norm(
        x.data_ptr(), fp32, _ptr(y), _ptr(gate), g_stride, _ptr(scale), sc_stride, _ptr(shift),
        sh_stride, mod is torch.float32, _ptr(weight), _ptr(bias), _ptr(post_weight), batch, tokens,
        channels, norm_id, post_id, residual_scale, eps, _ptr(residual_out), _ptr(out),
        _ptr(amax), _stream_at(at))
    if status:
        raise Nvfp4Error(status, "dit_gated_norm")
    return (x if y is None else residual_out), out


#: turns per position (float64) and position axis (int32) of each rotary pair,
#: the rotated elements per head, the number of axes, and the factor on rotated values
RotaryPlan = namedtuple("RotaryPlan", ["turns", "axis", "rotary_dim", "axes", "magnitude"])


def _yarn_blend(pairs, dim, base, original_length, beta_fast, beta_slow):
    """How far each pair's frequency is interpolated (0: kept, 1: divided by the
    factor): none for pairs with more than beta_fast turns over the trained
    length, fully below beta_slow turns, linear in the pair index between, from
    whole pair to whole pair."""
    def index_of(turns):
        return dim * math.log(original_length / (2 * math.pi * turns)) / (2 * math.log(base))
    fast, slow = index_of(beta_fast), index_of(beta_slow)
    # no pair between the two: the ramp's ends, clamped to the pairs, would change places
    if fast >= pairs - 1:
        return [0.0] * pairs
    if slow <= 0:
        return [1.0] * pairs
    low = max(math.floor(fast), 0)
    high = min(math.ceil(slow), dim - 1)
    width = high - low if high != low else 0.001
    return [min(max((j - low) / width, 0.0), 1.0) for j in range(pairs)]


def rotary_plan(rotary_dim, base=10000.0, axes=None, scaling="none", factor=1.0,
                original_length=0, beta_fast=32.0, beta_slow=1.0, device="cuda"):
    """The frequencies of ``rotary``, made once per model: pair j of an axis of d
    elements turns by base ** (-2 j / d) radians a position.

    axes: elements of each position axis (they sum to rotary_dim; text index,
    image row and image column of a DiT), None for one axis.  scaling, for
    positions past the trained length by ``factor``:
      "linear"  every frequency divided by the factor;
      "ntk"     the base raised to base * factor ** (d / (d - 2));
      "yarn"    by parts ("YaRN: Efficient Context Window Extension of Large
                Language Models"): frequencies below beta_slow turns over
                original_length divided, above beta_fast kept, blended between;
                rotated values scaled by 0.1 ln(factor) + 1.  The blend is linear
                in the pair index between whole pairs, the form that released
                checkpoints are trained and run with; the paper's section 3
                states it linear in the turns.
    """
    torch = _torch()
    if rotary_dim <= 0 or rotary_dim % 16 or rotary_dim > 256:
        raise ValueError(f"rotary_dim must be a positive multiple of 16 up to 256, got {rotary_dim}")
    dims = [rotary_dim] if axes is None else list(axes)
    if not 1 <= len(dims) <= 16 or any(d <= 0 or d % 2 for d in dims) or sum(dims) != rotary_dim:
        raise ValueError(f"axes must be up to 16 positive even sizes that sum to {rotary_dim}, got {dims}")
    if scaling not in ROTARY_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROTARY_SCALINGS)}, got {scaling!r}")
    if not (base > 1 and math.isfinite(base) and factor >= 1 and math.isfinite(factor)):
        raise ValueError(f"base must be above 1 and factor at least 1, got {base}, {factor}")
    if scaling == "none" and factor != 1.0:
        raise ValueError(f"factor {factor} needs a scaling")
    if scaling == "yarn" and not (original_length > 0 and beta_fast > beta_slow > 0):
        raise ValueError("yarn needs original_length > 0 and beta_fast > beta_slow > 0")
    turns, axis = [], []
    for a, d in enumerate(dims):
        b = base * factor ** (d / (d - 2)) if scaling == "ntk" and d > 2 else base
        radians = [b ** (-2 * j / d) for j in range(d // 2)]
        if scaling == "linear":
            radians = [f / factor for f in radians]
        if scaling == "yarn":
            blend = _yarn_blend(d // 2, d, base, original_length, beta_fast, beta_slow)
            radians = [f * (1 - m) + f / factor * m for f, m in zip(radians, blend)]
        turns += [f / (2 * math.pi) for f in radians]
        axis += [a] * (d // 2)
    return RotaryPlan(torch.tensor(turns, dtype=torch.float64, device=device),
                      torch.tensor(axis, dtype=torch.int32, device=device), rotary_dim, len(dims),
                      0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0)


#: the dit_heads of the C ABI, as bytes: data, then the batch, token and head strides
_VIEW = struct.Struct("@Pqqq").pack


def _heads(t, name, out=False):
    """(batch, tokens, heads, dim) and the C view of bf16 heads [tokens, heads,
    dim] or [batch, tokens, heads, dim]: dim dense, other strides multiples of
    8.  ``out``: no element may lie twice."""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.dim() not in (3, 4):
        raise ValueError(f"{name}: expected a 3-D or 4-D torch.Tensor")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {torch.bfloat16}")
    if t.dim() == 4:
        (b, n, h, d), (sb, sn, sh, sd) = t.shape, t.stride()
    else:
        (n, h, d), (sn, sh, sd) = t.shape, t.stride()
        b, sb = 1, 0
    if sd != 1 and d > 1:
        raise ValueError(f"{name}: the last dimension must be dense (got strides {tuple(t.stride())})")
    # the stride of a dimension that is never stepped along means nothing
    if b <= 1:
        sb = 0
    if n <= 1:
        sn = 0
    if h <= 1:
        sh = 0
    if (sb | sn | sh) & 7:
        raise ValueError(f"{name}: strides must be multiples of 8 (got {tuple(t.stride())})")
    if out:
        reach = d
        for s, size in sorted((s, size) for s, size in ((sb, b), (sn, n), (sh, h)) if size > 1):
            if s < reach:
                raise ValueError(f"{name}: elements overlap (strides {tuple(t.stride())})")
            reach = s * size
    return (b, n, h, d), _VIEW(t.data_ptr(), sb, sn, sh)


def _new_heads(like, shape4):
    """A new dense output like ``like`` (``shape4`` its shape with a batch) and its C view."""
    torch = _torch()
    t = torch.empty_like(like, memory_format=torch.contiguous_format)
    _, n, h, d = shape4
    return t, _VIEW(t.data_ptr(), n * h * d, h * d, d)


def _out_heads(out, like, name):
    """The C view of an output like ``like``, None when it is not given."""
    if out is None:
        return None
    _, view = _heads(out, name, out=True)
    if out.shape != like.shape:
        raise ValueError(f"{name}: shape {tuple(out.shape)}, expected {tuple(like.shape)}")
    return view


def rotary(q, positions, plan, k=None, layout="interleaved", q_weight=None, k_weight=None,
           eps=1e-6, out=None, k_out=None):
    """Rotary positions on the query heads and, in the same launch, the key
    heads; with ``q_weight`` / ``k_weight`` (float32 [dim]) each head is first
    RMS-normalised (the query/key norm).

    q: [tokens, heads, dim] or [batch, tokens, heads, dim], k the same with its
    own head count; views of a fused projection are taken as they are.
    positions: int32 [tokens] or [batch, tokens], with a last dimension of
    plan.axes when the plan has several axes.  layout: "interleaved" (pairs of
    neighbours) or "half" (j with j + rotary_dim / 2).  Elements from
    plan.rotary_dim on are not rotated.  ``out`` / ``k_out`` may be q / k; no
    other overlap.
    Returns out, or (out, k_out) when k is given.
    """
    torch = _torch()
    shape, qv = _heads(q, "q")
    batch, tokens, heads, dim = shape
    if not isinstance(plan, RotaryPlan):
        raise ValueError("plan: expected a RotaryPlan (rotary_plan)")
    if dim % 8 or not plan.rotary_dim <= dim <= 256:
        raise ValueError(f"q: head size must be a multiple of 8 in [{plan.rotary_dim}, 256], got {dim}")
    layout_id = _choice(layout, ROTARY_LAYOUTS, "layout")
    if not (eps > 0 and math.isfinite(eps)):
        raise ValueError(f"eps must be positive, got {eps}")
    if not isinstance(positions, torch.Tensor):
        raise ValueError("positions: expected a torch.Tensor")
    tail = (plan.axes,) if plan.axes > 1 or positions.dim() == q.dim() - 1 else ()
    _tensor(positions, "positions", torch.int32, (*q.shape[:-2], *tail), 0)
    _tensor(plan.turns, "plan.turns", torch.float64, (plan.rotary_dim // 2,))
    _tensor(plan.axis, "plan.axis", torch.int32, (plan.rotary_dim // 2,))
    kv_heads, kv = 0, None
    if k is not None:
        k_shape, kv = _heads(k, "k")
        kv_heads = k_shape[2]
        if k.dim() != q.dim() or (k_shape[:2], k_shape[3]) != (shape[:2], dim):
            raise ValueError(f"k: shape {tuple(k.shape)} does not go with q's {tuple(q.shape)}")
    elif k_weight is not None or k_out is not None:
        raise ValueError("k_weight and k_out need k")
    _opt(q_weight, "q_weight", torch.float32, (dim,))
    _opt(k_weight, "k_weight", torch.float32, (dim,))
    qo = _out_heads(out, q, "out")
    ko = None if k is None else _out_heads(k_out, k, "k_out")
    if k is not None and (out is not None or k_out is not None) and q.numel() and k.numel():
        # in place is each tensor in its own place; q and k in one would race
        here = None if out is None else out.data_ptr()
        there = None if k_out is None else k_out.data_ptr()
        if here == k.data_ptr() or there == q.data_ptr() or (here is not None and here == there):
            raise ValueError("out may be q itself and k_out k itself, but not the other's")
    at = _place((q, k, positions, plan.turns, plan.axis, q_weight, k_weight, out, k_out),
                "q k positions turns axis q_weight k_weight out k_out")
    if out is None:
        out, qo = _new_heads(q, shape)
    if k is not None and k_out is None:
        k_out, ko = _new_heads(k, k_shape)
    status = load().dit_rotary(
        qv, qo, heads, kv, ko, kv_heads, positions.data_ptr(), plan.axes, plan.turns.data_ptr(),
        plan.axis.data_ptr(), plan.magnitude, _ptr(q_weight), _ptr(k_weight), eps, batch, tokens,
        dim, plan.rotary_dim, layout_id, _stream_at(at))
    if status:
        raise Nvfp4Error(status, "dit_rotary")
    return out if k is None else (out, k_out)


def cross_attention_workspace(batch, queries, keys, heads, kv_heads, dim, device="cuda"):
    """A workspace for ``cross_attention`` on these sizes, or None if it would not split."""
    nbytes = load().dit_cross_attention_workspace_bytes(batch, queries, keys, heads, kv_heads, dim)
    if nbytes == 0:
        return None
    return _torch().empty(nbytes, dtype=_torch().uint8, device=device)


def cross_attention(q, k, v, kv_lengths=None, key_mask=None, scale=None, out=None,
                    workspace=_NO_WORKSPACE):
    """softmax(scale q k^T) v over an encoder's states (no causal order).

    q: [queries, heads, dim] or [batch, queries, heads, dim]; k, v the same with
    a length and a head count of their own, which divides q's (query heads share
    key heads in order).  Views of fused projections are taken as they are.
    dim: a multiple of 8 up to 128.  kv_lengths: int32 [batch], the keys each
    entry sees; key_mask: bool or uint8 [batch, keys], the keys to see (both:
    their intersection).  What lies out of sight does not count, whatever it
    holds; a query that sees no key, or whose scores are all -infinity, gets
    zeros.  scale: dim ** -0.5 by default.

    ``workspace``: a uint8 device tensor from ``cross_attention_workspace``
    (reused across calls on one stream), None not to split the keys, or left
    out to have one taken from torch's caching allocator for this call.
    """
    torch = _torch()
    (batch, queries, heads, dim), qv = _heads(q, "q")
    k_shape, kv = _heads(k, "k")
    v_shape, vv = _heads(v, "v")
    if not k.dim() == v.dim() == q.dim() or k_shape != v_shape:
        raise ValueError(f"k, v: shapes {tuple(k.shape)}, {tuple(v.shape)} do not go together")
    if k_shape[0] != batch or k_shape[3] != dim:
        raise ValueError(f"k: shape {tuple(k.shape)} does not go with q's {tuple(q.shape)}")
    keys, kv_heads = k_shape[1], k_shape[2]
    if kv_heads <= 0 or heads <= 0 or heads % kv_heads:
        raise ValueError(f"q has {heads} heads, not a positive multiple of k's {kv_heads}")
    if dim <= 0 or dim % 8 or dim > 128:
        raise ValueError(f"q: head size must be a multiple of 8 up to 128, got {dim}")
    if scale is None:
        scale = dim ** -0.5
    if not (scale > 0 and math.isfinite(scale)):
        raise ValueError(f"scale must be positive, got {scale}")
    _opt(kv_lengths, "kv_lengths", torch.int32, (batch,))
    mask_stride = 0
    if key_mask is not None:
        if not isinstance(key_mask, torch.Tensor) or tuple(key_mask.shape) != (batch, keys):
            raise ValueError(f"key_mask: expected a torch.Tensor of shape {(batch, keys)}")
        if key_mask.dtype not in (torch.bool, torch.uint8):
            raise ValueError(f"key_mask: dtype {key_mask.dtype}, expected bool or uint8")
        if keys > 1 and key_mask.stride(1) != 1:
            raise ValueError(f"key_mask: the last dimension must be dense (got strides {key_mask.stride()})")
        mask_stride = key_mask.stride(0) if batch > 1 else 0
    ov = _out_heads(out, q, "out")
    ws = None if workspace is _NO_WORKSPACE else _opt(workspace, "workspace", torch.uint8)
    at = _place((q, k, v, kv_lengths, key_mask, out, ws), "q k v kv_lengths key_mask out workspace")
    if out is None:
        out, ov = _new_heads(q, (batch, queries, heads, dim))
    lib = load()
    ws_bytes = 0
    if workspace is _NO_WORKSPACE:
        ws_bytes = lib.dit_cross_attention_workspace_bytes(batch, queries, keys, heads, kv_heads, dim)
        if ws_bytes:
            ws = q.new_empty((ws_bytes,), dtype=torch.uint8)
    elif ws is not None:
        ws_bytes = ws.numel()
    status = lib.dit_cross_attention(
        qv, kv, vv, _ptr(kv_lengths), _ptr(key_mask), mask_stride, batch, queries, keys, heads,
        kv_heads, dim, scale, ov, _ptr(ws), ws_bytes, _stream_at(at))
    if status:
        raise Nvfp4Error(status, "dit_cross_attention")
    return out


def lora_workspace(rows, inner, rank, device="cuda"):
    """A workspace for ``lora_add`` on these sizes."""
    nbytes = load().dit_lora_workspace_bytes(rows, inner, rank)
    return _torch().empty(nbytes, dtype=_torch().uint8, device=device)


def lora_add(y, x, down, up, ids, scales=None, epilogue="none", y_amax=None, out=None,
             workspace=_NO_WORKSPACE):
    """Low-rank adapters of many requests beside a projection they share:

        out[m] = epi(y[m] + scales[a] * up[a] @ (down[a] @ x[m])),  a = ids[m]

    y: [rows, outer], the shared projection's output (``gemm`` without an
    epilogue); x: [rows, inner], its input before quantization; down:
    [adapters, rank, inner], up: [adapters, outer, rank], lower ranks padded
    with zeros; ids: int32 [rows], -1 for a row without an adapter (any value
    outside [0, adapters) is); scales: optional float32 [adapters].  epilogue:
    "none" or "gelu", applied to every row after the sum; y_amax: optional
    one-element float32 device tensor, set to max |out| for ``quantize``.
    inner and outer are multiples of 8, rank a multiple of 8 up to 128.

    Returns out: y itself, updated in place, unless ``out`` is given.
    ``workspace``: from ``lora_workspace`` (reused across calls on one stream),
    or left out to have one taken from torch's caching allocator for this call.
    """
    torch = _torch()
    rows, outer = _matrix(y, "y", torch.bfloat16)
    x_rows, inner = _matrix(x, "x", torch.bfloat16)
    if x_rows != rows:
        raise ValueError(f"x: {x_rows} rows, y has {rows}")
    if not isinstance(down, torch.Tensor) or down.dim() != 3:
        raise ValueError("down: expected a 3-D torch.Tensor")
    adapters, rank, _ = down.shape
    if adapters <= 0 or rank <= 0 or rank % 8 or rank > 128:
        raise ValueError(f"down: needs adapters and a rank that is a multiple of 8 up to 128, got {tuple(down.shape)}")
    if inner <= 0 or inner % 8 or outer % 8:
        raise ValueError(f"inner and outer must be multiples of 8, got {inner} and {outer}")
    _tensor(down, "down", torch.bfloat16, (adapters, rank, inner))
    _tensor(up, "up", torch.bfloat16, (adapters, outer, rank))
    _tensor(ids, "ids", torch.int32, (rows,))
    _opt(scales, "scales", torch.float32, (adapters,))
    epi = _epilogue(epilogue)
    _opt(y_amax, "y_amax", torch.float32)
    _opt(out, "out", torch.bfloat16, (rows, outer))
    ws = None if workspace is _NO_WORKSPACE else _tensor(workspace, "workspace", torch.uint8, min_numel=0)
    at = _place((y, x, down, up, ids, scales, y_amax, out, ws),
                "y x down up ids scales y_amax out workspace")
    if out is None:
        out = y
    lib = load()
    if ws is None:
        ws = y.new_empty((lib.dit_lora_workspace_bytes(rows, inner, rank),), dtype=torch.uint8)
    status = lib.dit_lora_add(y.data_ptr(), x.data_ptr(), down.data_ptr(), up.data_ptr(),
                              ids.data_ptr(), _ptr(scales), rows, inner, outer, rank, adapters, epi,
                              out.data_ptr(), _ptr(y_amax), ws.data_ptr(), ws.numel(), _stream_at(at))
    if status:
        raise Nvfp4Error(status, "dit_lora_add")
    return out
