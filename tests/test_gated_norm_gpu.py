"""gated_norm against its definition in binary64, element by element.

Bounds, fixed before the first run.  One output rounding: UBF (bf16) or U32
relative to the value.  Before it, binary32 arithmetic: a thread sums 8 or 16
values, then at most 6 + 15 partial sums follow, so a mean is off by at most
(16 + 21) U32 of the mean magnitude of its terms; with the few roundings of the
products around it, 64 U32 of the row's largest term, scaled as the output
is, covers mean, variance (half its relative error reaches the result) and
products."""

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_05_amd as nv
import oracle.block as ob
from nvfp4_block_scaled_05_amd.graph import capture
from tests.block_util import U32, UBF, assert_within, f64, normal

pytestmark = pytest.mark.gpu


def make(seed, batch, tokens, channels, stream="bf16", mod=torch.bfloat16, use="ygsh", offset=0.0,
         weights=False, post="none"):
    rng = np.random.default_rng(seed)
    dt = torch.float32 if stream == "f32" else torch.bfloat16
    d = dict(x=normal(rng, (batch, tokens, channels), 2.0, offset, dt),
             y=normal(rng, (batch, tokens, channels)) if "y" in use else None)
    chunks = normal(rng, (batch, 6 * channels), 0.5, dtype=mod)
    for i, (name, letter) in enumerate((("gate", "g"), ("scale", "s"), ("shift", "h"))):
        d[name] = chunks[:, i * channels:(i + 1) * channels] if letter in use else None
    d["weight"] = normal(rng, (channels,), 0.2, 1.0, torch.float32) if weights else None
    d["bias"] = normal(rng, (channels,), 0.2, dtype=torch.float32) if weights else None
    d["post_weight"] = normal(rng, (channels,), 0.2, 1.0, torch.float32) if weights and post != "none" else None
    return d


def check(d, r, h, **kw):
    a = {k: f64(v) for k, v in d.items()}
    eps = kw.get("eps", 1e-6)
    want_r, want_h = ob.gated_norm(**a, **kw)

    def amp(v, kind):            # the norm's factor on a row and its largest term
        c = v - v.mean(-1, keepdims=True) if kind == "layer" else v
        f = 1.0 if kind == "none" else 1 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
        return f * np.abs(v).max(-1, keepdims=True)

    one = np.ones(1)
    gate = np.abs(a["gate"])[:, None] if a["gate"] is not None else one
    r_err = 0.0
    if a["y"] is not None:
        kind = kw.get("post_norm", "none")
        pw = np.abs(a["post_weight"]) if a["post_weight"] is not None else one
        z = np.abs(ob.normalise(a["y"], kind, eps)) if kind == "none" else amp(a["y"], kind)
        r_err = U32 * (64 * gate * pw * z + 4 * np.abs(kw.get("residual_scale", 1.0) * a["x"]))
    if r is not None and r is not d["x"]:
        assert_within(r, want_r, r_err + (U32 if r.dtype == torch.float32 else UBF) * np.abs(want_r), "r")
    kind = kw.get("norm", "layer")
    w = np.abs(a["weight"]) if a["weight"] is not None else one
    s = np.abs(1 + a["scale"])[:, None] if a["scale"] is not None else one
    f = amp(want_r, kind) / np.maximum(np.abs(want_r).max(-1, keepdims=True), 1e-300)
    bias = np.abs(a["bias"]) if a["bias"] is not None else 0.0
    shift = np.abs(a["shift"])[:, None] if a["shift"] is not None else 0.0
    # an error of r moves the mean and the variance too: 3 times its largest
    err = s * (w * (64 * U32 * amp(want_r, kind) + 3 * f * np.max(r_err + 0 * want_r, -1, keepdims=True))
               + 4 * U32 * bias) + 4 * U32 * shift
    assert_within(h, want_h, (err + UBF * np.abs(want_h)) * 1.001, "h")


SHAPES = [(1, 1, 8), (1, 7, 64), (2, 3, 520), (3, 5, 512), (2, 33, 1024), (1, 19, 3072), (2, 2, 8192),
          (1, 3, 16384), (1, 2, 8200)]


@pytest.mark.parametrize("stream", ["bf16", "f32"])
@pytest.mark.parametrize("norm", ["layer", "rms", "none"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_shapes(shape, norm, stream):
    d = make(sum(shape), *shape, stream=stream)
    r, h = nv.gated_norm(**d, norm=norm)
    check(d, r, h, norm=norm)


@pytest.mark.parametrize("use", ["", "s", "h", "y", "yg", "sh", "ygs", "ygsh"])
@pytest.mark.parametrize("weights", [False, True])
def test_optional_parts(use, weights):
    d = make(7, 2, 9, 264, use=use, weights=weights)
    r, h = nv.gated_norm(**d)
    assert (r is d["x"]) == (d["y"] is None)
    check(d, r, h)


@pytest.mark.parametrize("post", ["layer", "rms"])
@pytest.mark.parametrize("stream", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(2, 5, 72), (1, 11, 3072), (2, 3, 5000)], ids=str)
def test_post_norm(shape, stream, post):
    d = make(3, *shape, stream=stream, weights=True, post=post, mod=torch.float32)
    kw = dict(norm="rms", post_norm=post, residual_scale=0.5, eps=1e-5)
    r, h = nv.gated_norm(**d, **kw)
    check(d, r, h, **kw)


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("mod", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(5, 977, 1024), (70, 61, 520), (3, 6000, 72), (900, 3, 264)], ids=str)
def test_modulation_follows_the_batch_entry(shape, mod, weights):
    # workgroups take several rows, of several entries
    d = make(5, *shape, mod=mod, weights=weights)
    r, h = nv.gated_norm(**d)
    check(d, r, h)


def test_common_offset_loses_nothing():
    # mean 1000, deviation 2: a variance as a difference of squares would be
    # off by 1000^2 / 2^2 * U32 = 1.5 % here
    d = make(5, 1, 6, 3072, stream="f32", offset=1000.0)
    r, h = nv.gated_norm(**d)
    check(d, r, h)


def test_constant_rows():
    # no variance: h is the bias and shift alone, whatever eps
    x = torch.full((4, 256), 3.0, dtype=torch.bfloat16, device="cuda")
    _, h = nv.gated_norm(x)
    assert torch.equal(h, torch.zeros_like(h))
    x[1] = 0
    _, h = nv.gated_norm(x, norm="rms")
    assert torch.equal(h[1], torch.zeros_like(h[1]))


@pytest.mark.parametrize("tokens", [1, 5000])
def test_many_rows_and_amax(tokens):
    d = make(11, 2, tokens, 320)
    amax = torch.full((1,), 77.0, device="cuda")
    r, h = nv.gated_norm(**d, amax=amax)
    check(d, r, h)
    assert amax.item() == h.abs().max().item()
    # the quantizer takes it: the same bytes as with its own
    a, b = nv.quantize(h.view(-1, 320), amax=amax), nv.quantize(h.view(-1, 320))
    assert all(torch.equal(u, v) for u, v in zip(a[:3], b[:3]))


def test_nan_reaches_its_row_and_the_amax():
    d = make(12, 1, 9, 264)
    d["y"][0, 4, 17] = float("nan")
    amax = torch.zeros(1, device="cuda")
    r, h = nv.gated_norm(**d, amax=amax)
    assert torch.isnan(h[0, 4]).all() and not torch.isfinite(amax).any()
    keep = [i for i in range(9) if i != 4]
    assert torch.isfinite(h[0, keep]).all() and torch.isfinite(r[0, keep]).all()
    # an infinity: its row has no norm, the others are untouched
    d["y"][0, 4, 17] = float("inf")
    _, g = nv.gated_norm(**d)
    assert torch.equal(g[0, keep], h[0, keep])


def test_in_place_and_two_dimensions():
    d = make(13, 1, 300, 1032)
    want_r, want_h = nv.gated_norm(**d)
    flat = {k: v.view(-1, v.shape[-1]).clone() if k in "xy" else v for k, v in d.items() if v is not None}
    r, h = nv.gated_norm(**flat, residual_out=flat["x"], out=flat["y"])
    assert r is flat["x"] and h is flat["y"]
    assert torch.equal(r, want_r[0]) and torch.equal(h, want_h[0])


def test_empty_call():
    amax = torch.full((1,), 5.0, device="cuda")
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    r, h = nv.gated_norm(x, x, amax=amax)
    assert h.shape == (0, 64) and amax.item() == 0


def test_captured_and_on_two_streams():
    d = make(14, 2, 70, 512)
    out, res = torch.empty_like(d["y"]), torch.empty_like(d["x"])
    amax = torch.zeros(1, device="cuda")
    fn = lambda: nv.gated_norm(**d, amax=amax, out=out, residual_out=res)
    g = capture(fn)
    for i in range(3):
        d["x"].copy_(make(20 + i, 2, 70, 512)["x"])
        want_r, want_h = nv.gated_norm(**d)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want_h) and torch.equal(res, want_r)
        assert amax.item() == want_h.abs().max().item()
    others = [make(30 + i, 2, 700, 512) for i in range(2)]
    want = [nv.gated_norm(**o)[1] for o in others]
    torch.cuda.synchronize()
    got = [None, None]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            got[i] = nv.gated_norm(**others[i])[1]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def held_rows(channels):
    """More rows than the launch takes in two rounds of 24 waves a compute unit (256 a packed
    workgroup's lanes, or one workgroup each), from where on modulations are held."""
    chunks = channels // 8
    lanes = next((n for n in (8, 16, 32, 64) if chunks <= n), 0)
    waves = 4 if lanes else -(-chunks // 64)
    units = torch.cuda.get_device_properties(0).multi_processor_count
    return int(2.3 * units * (24 // waves)) * (256 // lanes if lanes else 1)


@pytest.mark.parametrize("stream,mod", [("bf16", torch.bfloat16), ("bf16", torch.float32),
                                        ("f32", torch.bfloat16), ("f32", torch.float32)])
@pytest.mark.parametrize("entries", [3, 211])     # several rows of a workgroup in an entry; one at most
@pytest.mark.parametrize("channels", [64, 120, 200, 264, 520, 1032, 3000, 6008, 8192])
def test_held_modulations_follow_the_batch_entry(channels, entries, stream, mod):
    tokens = held_rows(channels) // entries + 1
    weights, use = channels % 16 == 8, "ygsh" if channels != 1032 else "ysh"
    d = make(channels + entries, entries, tokens, channels, stream=stream, mod=mod, weights=weights, use=use,
             post="rms" if weights else "none")
    kw = dict(norm="layer" if channels % 3 else "rms", post_norm="rms" if weights else "none")
    amax = torch.zeros(1, device="cuda")
    r, h = nv.gated_norm(**d, **kw, amax=amax)
    check(d, r, h, **kw)
    assert amax.item() == h.abs().max().item()
    # in place, entry after entry in calls that are too small to hold anything: the same bits
    i = entries // 2
    one = {k: v if v is None or v.dim() == 1 else v[i:i + 1, :300] if v.dim() == 3 else v[i:i + 1]
           for k, v in d.items()}
    one["x"], one["y"] = one["x"].contiguous(), one["y"].contiguous()
    r1, h1 = nv.gated_norm(**one, **kw)
    assert torch.equal(r1, r[i:i + 1, :300]) and torch.equal(h1, h[i:i + 1, :300])
    r2, h2 = nv.gated_norm(**d, **kw, residual_out=d["x"], out=d["y"])
    assert torch.equal(r2, r) and torch.equal(h2, h)


@pytest.mark.parametrize("tokens", [5, 2600])
def test_one_modulation_for_all_entries(tokens):
    d = make(21, 3, tokens, 1032)
    for name in ("gate", "scale", "shift"):
        d[name] = d[name][1:2].expand(3, -1)
    r, h = nv.gated_norm(**d)
    check(d, r, h)
