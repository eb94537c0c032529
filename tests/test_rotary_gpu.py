"""rotary against its definition in binary64, element by element.

Bounds, fixed before the first run: the output rounding is UBF of the value.
An angle is a binary64 product reduced to a fraction of a turn, rounded to
binary32 (at most pi U32 rad off) before a sine and cosine good to a few U32,
and the two products and their sum add three more roundings: 16 U32 of
magnitude * (|a| + |b|).  The norm adds its factor's error, 16 + 8 terms in a
sum of squares of which half the relative error counts: 32 U32."""

import math

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_05_amd as nv
import oracle.block as ob
from nvfp4_block_scaled_05_amd.graph import capture
from tests.block_util import U32, UBF, assert_within, f64, normal

pytestmark = pytest.mark.gpu


def radians_of(plan):
    return f64(plan.turns) * 2 * np.pi


def check(got, v, positions, plan, layout, weight=None):
    p = positions.cpu().numpy().reshape(*v.shape[:2], plan.axes)
    want = ob.rotary(f64(v), p, radians_of(plan), plan.axis.cpu().numpy(), plan.rotary_dim, layout,
                     plan.magnitude, f64(weight))
    z = f64(v)
    if weight is not None:
        z = ob.normalise(z, "rms", 1e-6) * f64(weight)
    # 2 U32 pi |position| covers the 64-bit turns' rounding at any position here
    m = plan.magnitude * 2 * np.abs(z).max(-1, keepdims=True)
    exact_tail = weight is None and plan.rotary_dim < v.shape[-1]
    assert_within(got, want, UBF * np.abs(want) + (16 + (32 if weight is not None else 0)) * U32 * m, layout)
    if exact_tail:
        assert torch.equal(got[..., plan.rotary_dim:], v[..., plan.rotary_dim:])


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("batch,tokens,heads,kv,dim,rot", [
    (1, 1, 1, 1, 16, 16), (2, 5, 3, 1, 32, 16), (1, 7, 4, 2, 40, 32), (2, 9, 2, 2, 64, 64),
    (1, 33, 6, 2, 80, 32), (1, 13, 5, 5, 96, 96), (3, 17, 24, 8, 128, 128), (1, 6, 4, 4, 128, 48),
    (1, 11, 2, 1, 256, 256), (2, 3, 3, 2, 200, 112), (1, 2100, 2, 2, 64, 32)])
def test_shapes(batch, tokens, heads, kv, dim, rot, norm, layout):
    rng = np.random.default_rng(dim + tokens)
    q, k = normal(rng, (batch, tokens, heads, dim)), normal(rng, (batch, tokens, kv, dim))
    pos = torch.from_numpy(rng.integers(-50, 5000, (batch, tokens))).int().cuda()
    qw = normal(rng, (dim,), 0.2, 1.0, torch.float32) if norm else None
    kw = normal(rng, (dim,), 0.2, 1.0, torch.float32) if norm else None
    plan = nv.rotary_plan(rot)
    qo, ko = nv.rotary(q, pos, plan, k=k, layout=layout, q_weight=qw, k_weight=kw)
    check(qo, q, pos, plan, layout, qw)
    check(ko, k, pos, plan, layout, kw)
    # alone, and with a norm on one tensor only: the same numbers
    assert torch.equal(nv.rotary(q, pos, plan, layout=layout, q_weight=qw), qo)
    k2 = nv.rotary(q, pos, plan, k=k, layout=layout, k_weight=kw)[1]
    assert torch.equal(k2, ko)


def test_three_axes_of_a_fused_projection():
    rng = np.random.default_rng(1)
    b, t, h, d = 2, 75, 6, 128
    qkv = normal(rng, (b, t, 3, h, d))
    pos = torch.from_numpy(rng.integers(0, 200, (b, t, 3))).int().cuda()
    plan = nv.rotary_plan(d, axes=(16, 56, 56))
    w = normal(rng, (d,), 0.2, 1.0, torch.float32)
    q, k, v = qkv.unbind(2)
    before = v.clone()
    want = nv.rotary(q.contiguous(), pos, plan, k=k.contiguous(), q_weight=w, k_weight=w)
    check(want[0], q, pos, plan, "interleaved", w)
    check(want[1], k, pos, plan, "interleaved", w)
    got = nv.rotary(q, pos, plan, k=k, q_weight=w, k_weight=w, out=q, k_out=k)      # in place
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(v, before)


@pytest.mark.parametrize("scaling,factor,original", [("linear", 8.0, 0), ("ntk", 8.0, 0),
                                                     ("yarn", 32.0, 4096), ("yarn", 1.0, 4096)])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_far_positions(scaling, factor, original, layout):
    rng = np.random.default_rng(2)
    q = normal(rng, (1, 64, 2, 128))
    pos = torch.from_numpy(rng.integers(2 ** 30, 2 ** 31 - 1, (1, 64))).int().cuda()
    pos[0, :40] = torch.arange(131072 - 40, 131072)
    plan = nv.rotary_plan(64, scaling=scaling, factor=factor, original_length=original)
    # binary64 turns at 2^31 positions: 2^31 * 2^-53 turns, below U32
    check(nv.rotary(q, pos, plan, layout=layout), q, pos, plan, layout)


def test_position_zero_and_whole_turns():
    rng = np.random.default_rng(3)
    q = normal(rng, (1, 4, 2, 32))
    plan = nv.rotary_plan(32)
    zero = torch.zeros((1, 4), dtype=torch.int32, device="cuda")
    assert torch.equal(nv.rotary(q, zero, plan), q)
    # a quarter turn a position: positions of a multiple of 4 leave q as it is
    plan = plan._replace(turns=torch.full_like(plan.turns, 0.25))
    pos = torch.tensor([[0, 4, 1 << 30, -8]], dtype=torch.int32, device="cuda")
    assert torch.equal(nv.rotary(q, pos, plan), q)
    got = nv.rotary(q, pos + 2, plan, layout="half")
    assert torch.equal(got, -q)


def test_norm_of_zero_and_nan_heads():
    rng = np.random.default_rng(4)
    q = normal(rng, (1, 3, 4, 64))
    q[0, 1, 2] = 0
    q[0, 2, 0, 5] = float("nan")
    plan, w = nv.rotary_plan(64), torch.ones(64, device="cuda")
    pos = torch.arange(3, dtype=torch.int32, device="cuda")[None]
    got = nv.rotary(q, pos, plan, q_weight=w)
    assert torch.equal(got[0, 1, 2], torch.zeros_like(got[0, 1, 2]))
    assert torch.isnan(got[0, 2, 0]).all()
    assert torch.isfinite(got[0, :2]).all() and torch.isfinite(got[0, 2, 1:]).all()


def test_strided_output_leaves_the_rest():
    rng = np.random.default_rng(5)
    q = normal(rng, (2, 9, 3, 48))
    pos = torch.arange(18, dtype=torch.int32, device="cuda").view(2, 9)
    plan = nv.rotary_plan(48)
    wide = torch.full((2, 12, 5, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, 2:11, 1:4, 8:56]
    nv.rotary(q, pos, plan, out=out)
    assert torch.equal(out, nv.rotary(q, pos, plan))
    out.fill_(7.0)
    assert torch.equal(wide, torch.full_like(wide, 7.0))
    # a 3-D call, and an expanded input
    assert torch.equal(nv.rotary(q[0], pos[0], plan), nv.rotary(q, pos, plan)[0])
    e = q[:1].expand(2, -1, -1, -1)
    assert torch.equal(nv.rotary(e, pos, plan), nv.rotary(e.contiguous(), pos, plan))


def test_empty_and_captured():
    plan = nv.rotary_plan(32)
    e = torch.empty((0, 2, 32), dtype=torch.bfloat16, device="cuda")
    assert nv.rotary(e, torch.empty(0, dtype=torch.int32, device="cuda"), plan).shape == e.shape
    rng = np.random.default_rng(6)
    q, k = normal(rng, (1, 40, 4, 32)), normal(rng, (1, 40, 2, 32))
    pos = torch.arange(40, dtype=torch.int32, device="cuda")[None].contiguous()
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    g = capture(lambda: nv.rotary(q, pos, plan, k=k, out=qo, k_out=ko))
    for i in range(3):
        pos.add_(i + 1)
        want = nv.rotary(q, pos, plan, k=k)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("heads,kv,dim,rot", [(3, 2, 32, 32), (4, 1, 40, 32), (9, 3, 128, 96), (2, 1, 200, 112)])
def test_tensors_past_the_last_level_cache(heads, kv, dim, rot, norm, layout):
    # more than 256 MiB read and written: accesses that pass the caches by, here in place
    # on views of a fused projection
    rng = np.random.default_rng(dim)
    tokens = (256 << 20) // (4 * dim * (heads + kv)) + 77
    g = torch.Generator(device="cuda").manual_seed(dim)
    qkv = torch.randn((tokens, heads + 2 * kv, dim), generator=g, device="cuda").bfloat16()
    q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
    pos = torch.randint(-100, 70000, (tokens, 2), generator=g, device="cuda", dtype=torch.int32)
    qw = normal(rng, (dim,), 0.2, 1.0, torch.float32) if norm else None
    kw = normal(rng, (dim,), 0.2, 1.0, torch.float32) if norm else None
    plan = nv.rotary_plan(rot, axes=(16, rot - 16))
    args = dict(layout=layout, q_weight=qw, k_weight=kw)
    before = v.clone()
    # parts of it, which the cache holds: the kernel of the tests above
    parts = [nv.rotary(a.contiguous(), p.contiguous(), plan, k=b.contiguous(), **args)
             for a, b, p in zip(q.split(tokens // 3), k.split(tokens // 3), pos.split(tokens // 3))]
    at = torch.cat([torch.arange(100), torch.arange(tokens - 100, tokens),
                    torch.from_numpy(rng.integers(0, tokens, 300))]).cuda()
    q0, k0 = q[at].unsqueeze(0), k[at].unsqueeze(0)
    qo, ko = nv.rotary(q, pos, plan, k=k, out=q, k_out=k, **args)
    check(qo[at].unsqueeze(0), q0, pos[at], plan, layout, qw)
    check(ko[at].unsqueeze(0), k0, pos[at], plan, layout, kw)
    assert torch.equal(qo, torch.cat([p[0] for p in parts])) and torch.equal(ko, torch.cat([p[1] for p in parts]))
    assert torch.equal(v, before)
