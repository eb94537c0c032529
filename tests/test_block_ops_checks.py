"""Argument checks of the operators between the linears that need no GPU: the
Python layer raises ValueError before any pointer reaches the library, and the C
entry points report errors before touching a device (their pointers are fake and
never dereferenced: every call fails a check first, the device check at the
latest).  The rotary plan's frequencies are checked against their formulas."""

import math

import pytest
import torch

import nvfp4_block_scaled_05_amd as nv
from nvfp4_block_scaled_05_amd import _binding
from nvfp4_block_scaled_05_amd.block_ops import _VIEW

OK, NULL, SHAPE, ALIGN, WORKSPACE, DEVICE, ARG = 0, -1, -2, -3, -4, -5, -6
A = 1 << 20


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def f32(*shape):
    return torch.zeros(shape)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def raises(match, fn, *args, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*args, **kw)


def test_gated_norm_rejects():
    g, x = nv.gated_norm, bf16(2, 3, 64)
    raises("GPU tensor", g, x)
    raises("GPU tensor", g, f32(3, 64))
    raises("2-D or 3-D", g, bf16(64))
    raises("dtype", g, x.half())
    raises("contiguous", g, bf16(64, 4).t())
    raises("multiple of 8", g, bf16(3, 60))
    raises("up to 16384", g, bf16(1, 16392))
    raises("norm must be", g, x, norm="batch")
    raises("post_norm must be", g, x, x, post_norm="batch")
    raises("gate needs y", g, x, gate=bf16(2, 64))
    raises("post_weight needs y", g, x, post_weight=f32(64))
    raises("residual_out needs y", g, x, residual_out=x)
    raises("need y", g, x, residual_scale=0.5)
    raises("need y", g, x, post_norm="rms")
    raises("eps", g, x, eps=0.0)
    raises("eps", g, x, eps=float("nan"))
    raises("residual_scale finite", g, x, x, residual_scale=float("inf"))
    raises("y: shape", g, x, bf16(2, 3, 72))
    raises("y: dtype", g, x, f32(2, 3, 64))
    raises("gate: expected", g, x, x, gate=bf16(1, 64))
    raises("scale: dtype", g, x, x, gate=bf16(2, 64), scale=f32(2, 64))
    raises("shift: the last dimension", g, x, shift=bf16(64, 2).t())
    raises("expected bfloat16 or float32", g, x, scale=torch.zeros(2, 64, dtype=torch.float16))
    raises("weight: dtype", g, x, weight=bf16(64))
    raises("bias: shape", g, x, bias=f32(65))
    raises("amax: needs", g, x, amax=f32(0))
    raises("out: shape", g, x, out=bf16(6, 64))
    raises("residual_out: dtype", g, x, x, residual_out=f32(2, 3, 64))


def test_rotary_plan_rejects_and_formulas():
    p = nv.rotary_plan
    raises("rotary_dim", p, 24, device="cpu")
    raises("rotary_dim", p, 272, device="cpu")
    raises("axes", p, 64, axes=(16, 32), device="cpu")
    raises("axes", p, 64, axes=(63, 1), device="cpu")
    raises("scaling must be", p, 64, scaling="dynamic", device="cpu")
    raises("needs a scaling", p, 64, factor=2.0, device="cpu")
    raises("at least 1", p, 64, scaling="linear", factor=0.5, device="cpu")
    raises("base", p, 64, base=1.0, device="cpu")
    raises("yarn needs", p, 64, scaling="yarn", factor=2.0, device="cpu")

    def radians(*a, **k):
        return (p(*a, device="cpu", **k).turns * 2 * math.pi).tolist()
    plain = radians(64)
    assert plain == pytest.approx([10000.0 ** (-j / 32) for j in range(32)], rel=1e-14)
    assert radians(64, scaling="linear", factor=4.0) == pytest.approx([f / 4 for f in plain], rel=1e-14)
    ntk = radians(64, scaling="ntk", factor=4.0)
    # the fastest pair keeps its frequency, the slowest is divided by the factor
    assert ntk[0] == pytest.approx(1.0) and ntk[-1] == pytest.approx(plain[-1] / 4, rel=1e-12)
    y = p(64, scaling="yarn", factor=32.0, original_length=4096, device="cpu")
    yr = (y.turns * 2 * math.pi).tolist()
    for f, g in zip(plain, yr):
        turns = f * 4096 / (2 * math.pi)
        assert f / 32 * (1 - 1e-12) <= g <= f * (1 + 1e-12)
        if turns > 64:
            assert g == pytest.approx(f, rel=1e-12)
        if turns < 0.5:
            assert g == pytest.approx(f / 32, rel=1e-12)
    assert y.magnitude == pytest.approx(0.1 * math.log(32) + 1)
    three = p(128, axes=(16, 56, 56), device="cpu")
    assert three.axes == 3 and three.axis.tolist() == [0] * 8 + [1] * 28 + [2] * 28
    assert three.turns[8:36].tolist() == three.turns[36:].tolist()


def test_rotary_rejects():
    plan = nv.rotary_plan(32, device="cpu")
    r, q, pos = nv.rotary, bf16(2, 5, 3, 64), i32(2, 5)
    raises("GPU tensor", r, q, pos, plan)
    raises("3-D or 4-D", r, bf16(5, 64), pos, plan)
    raises("q: dtype", r, f32(2, 5, 3, 64), pos, plan)
    raises("last dimension must be dense", r, bf16(2, 5, 64, 3).transpose(2, 3), pos, plan)
    raises("multiples of 8", r, bf16(2, 5, 3, 68)[..., :64], pos, plan)
    raises("head size", r, bf16(2, 5, 3, 24), pos, plan)
    raises("head size", r, bf16(2, 5, 3, 264), pos, plan)
    raises("RotaryPlan", r, q, pos, (plan.turns, plan.axis))
    raises("layout must be", r, q, pos, plan, layout="pairs")
    raises("positions: dtype", r, q, pos.long(), plan)
    raises("positions: shape", r, q, i32(2, 6), plan)
    raises("positions: shape", r, q, i32(2, 5, 2), plan)
    raises("positions: shape", r, q, pos, nv.rotary_plan(32, axes=(16, 16), device="cpu"))
    raises("k: shape", r, q, pos, plan, k=bf16(2, 6, 3, 64))
    raises("k: shape", r, q, pos, plan, k=bf16(2, 5, 3, 72))
    raises("need k", r, q, pos, plan, k_weight=f32(64))
    raises("q_weight: shape", r, q, pos, plan, q_weight=f32(32))
    raises("out: shape", r, q, pos, plan, out=bf16(2, 5, 4, 64))
    raises("out: elements overlap", r, q, pos, plan, out=bf16(1, 5, 3, 64).expand(2, -1, -1, -1))
    raises("out: elements overlap", r, q, pos, plan, out=bf16(9000).as_strided((2, 5, 3, 64), (960, 192, 56, 1)))
    raises("eps", r, q, pos, plan, eps=-1.0)


def test_cross_attention_rejects():
    c = nv.cross_attention
    q, k = bf16(2, 5, 4, 64), bf16(2, 9, 2, 64)
    raises("GPU tensor", c, q, k, k)
    raises("do not go together", c, q, k, bf16(2, 8, 2, 64))
    raises("do not go together", c, q[0], k, k)
    raises("does not go with", c, q, bf16(1, 9, 2, 64), bf16(1, 9, 2, 64))
    raises("does not go with", c, q, bf16(2, 9, 2, 72), bf16(2, 9, 2, 72))
    raises("positive multiple", c, q, bf16(2, 9, 3, 64), bf16(2, 9, 3, 64))
    raises("positive multiple", c, q, bf16(2, 9, 0, 64), bf16(2, 9, 0, 64))
    raises("head size", c, bf16(2, 5, 4, 136), bf16(2, 9, 2, 136), bf16(2, 9, 2, 136))
    raises("scale", c, q, k, k, scale=0.0)
    raises("scale", c, q, k, k, scale=float("inf"))
    raises("kv_lengths: dtype", c, q, k, k, kv_lengths=torch.zeros(2, dtype=torch.int64))
    raises("kv_lengths: shape", c, q, k, k, kv_lengths=i32(3))
    raises("key_mask: dtype", c, q, k, k, key_mask=f32(2, 9))
    raises("key_mask: expected", c, q, k, k, key_mask=torch.zeros(2, 8, dtype=torch.bool))
    raises("key_mask: the last", c, q, k, k, key_mask=torch.zeros(9, 2, dtype=torch.bool).t())
    raises("out: dtype", c, q, k, k, out=f32(2, 5, 4, 64))
    raises("workspace: dtype", c, q, k, k, workspace=f32(8))


def test_lora_rejects():
    f = nv.lora_add
    y, x, d, u, ids = bf16(6, 32), bf16(6, 64), bf16(3, 16, 64), bf16(3, 32, 16), i32(6)
    raises("GPU tensor", f, y, x, d, u, ids)
    raises("rows", f, y, bf16(7, 64), d, u, ids)
    raises("3-D", f, y, x, bf16(16, 64), u, ids)
    raises("rank", f, y, x, bf16(3, 12, 64), bf16(3, 32, 12), ids)
    raises("rank", f, y, x, bf16(3, 136, 64), bf16(3, 32, 136), ids)
    raises("rank", f, y, x, bf16(0, 16, 64), bf16(0, 32, 16), ids)
    raises("multiples of 8", f, bf16(6, 30), x, d, bf16(3, 30, 16), ids)
    raises("down: shape", f, y, x, bf16(3, 16, 72), u, ids)
    raises("up: shape", f, y, x, d, bf16(3, 16, 32), ids)
    raises("up: shape", f, y, x, d, bf16(2, 32, 16), ids)
    raises("ids: dtype", f, y, x, d, u, ids.long())
    raises("ids: shape", f, y, x, d, u, i32(5))
    raises("scales: shape", f, y, x, d, u, ids, scales=f32(2))
    raises("epilogue", f, y, x, d, u, ids, epilogue="relu")
    raises("contiguous", f, bf16(32, 6).t(), x, d, u, ids)
    raises("out: shape", f, y, x, d, u, ids, out=bf16(5, 32))
    raises("workspace: expected", f, y, x, d, u, ids, workspace=None)


# ---------------------------------------------------------------- C entry points

@pytest.fixture(scope="module")
def lib():
    return _binding.load()


def test_declared_and_exported(lib):
    import re
    from tests.test_abi import HEADER
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(dit_\w+)\s*\(", text)))
    assert names == sorted(["dit_gated_norm", "dit_rotary", "dit_cross_attention",
                            "dit_cross_attention_workspace_bytes", "dit_lora_add",
                            "dit_lora_workspace_bytes"])
    for n in names:
        assert n in _binding.SIGNATURES and hasattr(lib, n)


def gpu():
    return torch.cuda.is_available()


def test_gated_norm_c(lib):
    def f(x=A, y=A, gate=None, gs=0, batch=2, tokens=3, c=64, norm=1, post=0, rs=1.0, eps=1e-6, r=A, h=A,
          amax=None, w=None):
        return lib.dit_gated_norm(x, 0, y, gate, gs, None, 0, None, 0, 0, w, None, None, batch, tokens,
                                  c, norm, post, rs, eps, r, h, amax, None)
    assert f(x=None) == NULL
    assert f(r=None, h=None) == NULL
    assert f(h=None, amax=A) == NULL
    for kw in (dict(batch=-1), dict(tokens=1 << 31), dict(c=0), dict(c=60), dict(c=16392),
               dict(batch=1 << 20, tokens=1 << 20), dict(gate=A, gs=4), dict(gate=A, gs=-8)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(x=A + 8), dict(y=A + 2), dict(gate=A + 8), dict(r=A + 8), dict(h=A + 8), dict(amax=A + 2),
               dict(w=A + 4)):
        assert f(**kw) == ALIGN, kw
    for kw in (dict(norm=3), dict(post=-1), dict(eps=0.0), dict(eps=float("nan")), dict(rs=float("inf")),
               dict(y=None), dict(y=None, r=None, rs=0.5), dict(y=None, r=None, post=1),
               dict(y=None, r=None, gate=A)):
        assert f(**kw) == ARG, kw
    if not gpu():
        assert f() == DEVICE
        assert f(batch=0, x=None, y=None, r=None, h=None) == DEVICE


def heads(data=A, b=8192, t=1024, h=64):
    return _VIEW(data or 0, b, t, h)


def test_rotary_c(lib):
    def f(q=heads(), qo=heads(), nh=4, k=None, ko=None, nk=0, pos=A, axes=1, turns=A, axis=None, mag=1.0,
          qw=None, eps=1e-6, batch=2, tokens=3, dim=64, rot=32, layout=0):
        return lib.dit_rotary(q, qo, nh, k, ko, nk, pos, axes, turns, axis, mag, qw, None, eps, batch, tokens,
                              dim, rot, layout, None)
    for kw in (dict(q=None), dict(qo=None), dict(nk=2), dict(nk=2, k=heads()), dict(pos=None), dict(turns=None),
               dict(axes=2), dict(q=heads(None)), dict(nk=2, k=heads(None), ko=heads())):
        assert f(**kw) == NULL, kw
    for kw in (dict(nh=0), dict(nh=-1), dict(nh=1 << 17), dict(dim=60), dict(dim=264), dict(rot=24), dict(rot=80),
               dict(rot=0), dict(axes=0), dict(axes=17, axis=A), dict(q=heads(t=100)), dict(qo=heads(h=-64)),
               dict(nk=2, k=heads(b=4), ko=heads()), dict(tokens=-1)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(q=heads(A + 8)), dict(qo=heads(A + 2)), dict(pos=A + 2), dict(turns=A + 4), dict(qw=A + 2),
               dict(nk=2, k=heads(), ko=heads(A + 8))):
        assert f(**kw) == ALIGN, kw
    for kw in (dict(layout=2), dict(eps=0.0), dict(mag=0.0), dict(mag=float("inf"))):
        assert f(**kw) == ARG, kw
    if not gpu():
        assert f() == DEVICE
        assert f(nk=2, k=heads(), ko=heads()) == DEVICE


def test_cross_attention_c(lib):
    def f(q=heads(), k=heads(), v=heads(), out=heads(), lengths=None, mask=None, ms=0, b=2, lq=5, lk=9, h=4, hk=2,
          dim=64, scale=0.1, ws=None, wsb=0):
        return lib.dit_cross_attention(q, k, v, lengths, mask, ms, b, lq, lk, h, hk, dim, scale, out, ws, wsb, None)
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(q=heads(None)), dict(v=heads(None)),
               dict(out=heads(None))):
        assert f(**kw) == NULL, kw
    for kw in (dict(b=-1), dict(lk=(1 << 31) - 1), dict(h=5), dict(hk=0), dict(h=0), dict(dim=60), dict(dim=136),
               dict(k=heads(t=1 << 23)), dict(v=heads(t=12)), dict(out=heads(b=-8)), dict(mask=A, ms=-1),
               dict(b=1 << 16, lq=1 << 16, h=4)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(q=heads(A + 8)), dict(out=heads(A + 8)), dict(lengths=A + 2), dict(ws=A + 16, wsb=1 << 20)):
        assert f(**kw) == ALIGN, kw
    for kw in (dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan"))):
        assert f(**kw) == ARG, kw
    wb = lib.dit_cross_attention_workspace_bytes
    assert wb(0, 5, 9, 4, 2, 64) == wb(1, 1, 9, 4, 3, 64) == wb(1, 1, 9, 4, 2, 60) == wb(1, 1, -1, 4, 2, 64) == 0
    assert wb(1, 16384, 512, 24, 24, 128) == 0          # rows enough to fill the chip
    assert wb(1, 1, 8192, 8, 8, 128) > 0
    if not gpu():
        assert f() == DEVICE
        assert f(lk=0, k=heads(None), v=heads(None)) == DEVICE


def test_lora_c(lib):
    def f(y=A, x=A, d=A, u=A, ids=A, s=None, rows=6, k=64, n=32, r=16, ad=3, epi=0, out=A, amax=None, ws=A,
          wsb=1 << 20):
        return lib.dit_lora_add(y, x, d, u, ids, s, rows, k, n, r, ad, epi, out, amax, ws, wsb, None)
    for kw in (dict(y=None), dict(x=None), dict(d=None), dict(u=None), dict(ids=None), dict(out=None), dict(ws=None)):
        assert f(**kw) == NULL, kw
    for kw in (dict(rows=-1), dict(k=0), dict(k=60), dict(n=30), dict(r=12), dict(r=0), dict(r=136), dict(ad=0)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(y=A + 8), dict(x=A + 8), dict(d=A + 8), dict(u=A + 8), dict(out=A + 8), dict(ids=A + 2),
               dict(s=A + 2), dict(amax=A + 2), dict(ws=A + 16)):
        assert f(**kw) == ALIGN, kw
    assert f(epi=2) == ARG
    need = lib.dit_lora_workspace_bytes(6, 64, 16)
    assert need == 6 * 16 * 4
    assert f(wsb=need - 1) == WORKSPACE
    assert lib.dit_lora_workspace_bytes(0, 64, 16) == lib.dit_lora_workspace_bytes(6, 60, 16) == 0
    if not gpu():
        assert f(wsb=need) == DEVICE
        assert f(rows=0, y=None, x=None, d=None, u=None, ids=None, out=None, ws=None, wsb=0) == DEVICE


def test_norm_none_rejects():
    x = bf16(2, 3, 64)
    raises("needs a norm", nv.gated_norm, x, x, norm=None, scale=bf16(2, 64))
    raises("needs a norm", nv.gated_norm, x, x, norm=None, amax=f32(1))
    raises("needs y", nv.gated_norm, x, norm=None)


def test_gated_norm_refuses_one_place_for_two():
    x, y = bf16(2, 3, 64), bf16(2, 3, 64)
    raises("same buffer", nv.gated_norm, x, y, out=y, residual_out=y)
    raises("same buffer", nv.gated_norm, x, y, out=x, residual_out=x)
    raises("GPU tensor", nv.gated_norm, x, y, out=y, residual_out=x)
    empty = bf16(2, 0, 64)
    raises("GPU tensor", nv.gated_norm, empty, empty, out=empty, residual_out=empty)


def test_rotary_refuses_one_place_for_two():
    plan = nv.rotary_plan(32, device="cpu")
    q, k, pos = bf16(2, 5, 3, 64), bf16(2, 5, 3, 64), i32(2, 5)
    raises("not the other's", nv.rotary, q, pos, plan, k=q, out=q, k_out=q)
    raises("not the other's", nv.rotary, q, pos, plan, k=k, out=k)
    raises("not the other's", nv.rotary, q, pos, plan, k=k, k_out=q)
    raises("not the other's", nv.rotary, q, pos, plan, k=k, out=(o := bf16(2, 5, 3, 64)), k_out=o)
    raises("GPU tensor", nv.rotary, q, pos, plan, k=k, out=q, k_out=k)      # each in its own place


def test_subnormal_eps_is_refused(lib):
    sub = 1e-40
    assert lib.dit_gated_norm(A, 0, A, None, 0, None, 0, None, 0, 0, None, None, None, 1, 1, 64, 1, 0, 1.0, sub,
                              A, A, None, None) == ARG
    assert lib.dit_rotary(heads(), heads(), 4, None, None, 0, A, 1, A, None, 1.0, A, None, sub, 1, 1, 64, 32, 0,
                          None) == ARG


def test_sizes_past_the_grid_are_refused(lib):
    assert lib.dit_lora_add(A, A, A, A, A, None, 1 << 26, 64, 32, 16, 1, 0, A, None, A, 1 << 40, None) == SHAPE
    assert lib.dit_cross_attention(heads(), heads(), heads(), None, None, 0, 1 << 12, 33, 9, 1 << 13, 1 << 13, 64,
                                   0.1, heads(), None, 0, None) == SHAPE


def yarn_radians(dim, length, factor=32.0, **kw):
    return (nv.rotary_plan(dim, scaling="yarn", factor=factor, original_length=length, device="cpu", **kw).turns
            * 2 * math.pi).tolist()


def test_yarn_blend_between_the_ends():
    # 32 turns over 4096 positions fall to pair 64 ln(4096 / 64 pi) / (2 ln 10000) = 10.47, one turn
    # to pair 22.5: kept up to 10, divided from 23 on, in between linear in the pair index
    for j, f in enumerate(yarn_radians(64, 4096)):
        plain, slow = 10000.0 ** (-j / 32), min(max((j - 10) / 13, 0.0), 1.0)
        assert f == pytest.approx(plain * (1 - slow) + plain / 32 * slow, rel=1e-12), j


@pytest.mark.parametrize("kw,length", [(dict(base=2.0), 4096), (dict(base=1.01), 300), ({}, 1 << 50),
                                       (dict(axes=(16, 48)), 1 << 50)])
def test_yarn_keeps_pairs_that_all_turn_often(kw, length):
    # every pair turns more than 32 times over the trained length: none is divided
    want = (nv.rotary_plan(64, device="cpu", **kw).turns * 2 * math.pi).tolist()
    assert min(want) * length / (2 * math.pi) > 32
    assert yarn_radians(64, length, **kw) == pytest.approx(want, rel=1e-12)


@pytest.mark.parametrize("length", [1, 3, 6])
def test_yarn_divides_pairs_that_all_turn_less_than_once(length):
    want = (nv.rotary_plan(64, device="cpu").turns * 2 * math.pi / 32).tolist()
    assert yarn_radians(64, length) == pytest.approx(want, rel=1e-12)


def test_lora_takes_the_workspace_of_no_rows():
    # what lora_workspace makes for no rows has no bytes; the call is a no-op, not an error
    ws = nv.lora_workspace(0, 64, 16, device="cpu")
    assert ws.numel() == 0
    raises("GPU tensor", nv.lora_add, bf16(0, 32), bf16(0, 64), bf16(3, 16, 64), bf16(3, 32, 16), i32(0),
           workspace=ws)
    # for rows it is refused all the same, by its size
    raises("GPU tensor", nv.lora_add, bf16(6, 32), bf16(6, 64), bf16(3, 16, 64), bf16(3, 32, 16), i32(6),
           workspace=ws)
