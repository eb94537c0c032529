"""DitCrossBlock: the operators between the linears run together with the
quantized linears, stage by stage against binary64 on the GPU's own inputs of
each stage (so a code flipped at a rounding tie cannot propagate), captured in a
HIP graph, and equal to the same calls made one by one."""

import math

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_05_amd as nv
import oracle.block as ob
from nvfp4_block_scaled_05_amd.dit_block import CROSS_LAYERS, DitCrossBlock
from nvfp4_block_scaled_05_amd.graph import capture
from tests.block_util import U32, UBF, assert_within, f64, normal

pytestmark = pytest.mark.gpu

B, T, L, HID, HEADS, KV, DIM, MLP, ENC = 2, 70, 33, 256, 4, 2, 64, 512, 128
MOD, Q, KVP, OUT, UP, DOWN = CROSS_LAYERS


def make(with_lora=True):
    rng = np.random.default_rng(0)
    w = {"w_mod": (6 * HID, HID), "w_q": (HEADS * DIM, HID), "w_kv": (2 * KV * DIM, ENC), "w_o": (HID, HEADS * DIM),
         "w_up": (MLP, HID), "w_down": (HID, MLP)}
    weights = {k: normal(rng, s, 0.05) for k, s in w.items()}
    lora = None
    if with_lora:
        lora = {}
        for name in (Q, UP, DOWN):
            n, k = weights[CROSS_LAYERS[name][0]].shape
            lora[name] = (normal(rng, (3, 8, k), 0.05), normal(rng, (3, n, 8), 0.3),
                          torch.tensor([1.0, 0.5, 2.0], device="cuda"))
    qn = normal(rng, (DIM,), 0.1, 1.0, torch.float32)
    kn = normal(rng, (DIM,), 0.1, 1.0, torch.float32)
    block = DitCrossBlock(weights, B, T, L, HEADS, KV, qn, kn, nv.rotary_plan(DIM, axes=(16, 24, 24)), lora)
    states = normal(rng, (B, L, ENC))
    states[1, 5:] = 0                                 # padding
    lengths = torch.tensor([L, 5], dtype=torch.int32, device="cuda")
    pos = torch.from_numpy(rng.integers(0, 64, (B, T, 3))).int().cuda()
    ids = torch.from_numpy(np.repeat([0, 2, -1, 1], [50, 40, 20, 30])).int().cuda()
    return block, (normal(rng, (B, HID)), normal(rng, (B, T, HID)), pos, ids), states, lengths


def test_unencoded_and_unknown_layer():
    block, (temb, x, pos, ids), _, _ = make(False)
    with pytest.raises(ValueError, match="encode"):
        block(temb, x, pos)
    with pytest.raises(ValueError, match="not layers"):
        DitCrossBlock({"w_q": temb}, B, T, L, HEADS, KV, None, None, None, {MOD: None})


def linear64(block, name, ids=None, x=None):
    """The layer in binary64 on the values its NVFP4 operands stand for, and the
    size of its terms; adapters from the bf16 input x."""
    codes, scales, ts = block.qbuf[name]
    w = block.weights[name]
    a = nv.Nvfp4Tensor(codes, scales, ts, w.cols)
    a, ww = values(a), values(w)
    y, size = a @ ww.T, np.abs(a) @ np.abs(ww).T
    if ids is not None and name in block.lora:
        down, up, s = (f64(t) for t in block.lora[name])
        i = ids.cpu().numpy()
        y, more = ob.lora_add(y, f64(x), down, up, i, s)
        size = size * (1 + UBF) + UBF * np.abs(y) + more
    return y, size


def values(q):
    """What an Nvfp4Tensor stands for, in binary64."""
    from oracle.formats import e2m1_value, e4m3_value
    e2m1 = np.array([float(e2m1_value(c)) for c in range(16)])
    e4m3 = np.array([float(e4m3_value(b)) for b in range(127)])
    codes = q.codes.cpu().numpy()
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1)
    s = e4m3[q.scales.cpu().numpy()]
    return e2m1[nib] * np.repeat(s, 16, 1) * q.tensor_scale.double().item()


def test_stage_by_stage():
    block, (temb, x, pos, ids), states, lengths = make()
    block.encode(states, lengths)
    result = block(temb, x, pos, ids)
    torch.cuda.synchronize()
    mod = [f64(m) for m in block.out[MOD].chunk(6, 1)]
    want_mod = f64(temb) @ f64(block.weights[MOD]).T
    size = np.abs(f64(temb)) @ np.abs(f64(block.weights[MOD])).T
    assert_within(block.out[MOD], want_mod, UBF * np.abs(want_mod) + (HID + 8) * U32 * size, "modulation")

    # the query projection, adapters, norm and rotation: the projection's bf16
    # output is rounded twice (gemm, adapters) before the norm and once after
    _, h = ob.gated_norm(f64(x), scale=mod[1], shift=mod[0])
    h_bf = torch.from_numpy(h).bfloat16().cuda()
    y, size = linear64(block, Q, ids, h_bf.view(-1, HID))
    y, size = y.reshape(B, T, HEADS, DIM), size.reshape(B, T, HEADS, DIM)
    qn = f64(block.q_norm)
    f = qn / np.sqrt((y * y).mean(-1, keepdims=True) + 1e-6)
    pre = np.max((3 * UBF * size) * np.abs(f), -1, keepdims=True)
    rad = f64(block.plan.turns) * 2 * np.pi
    want = ob.rotary(y, pos.cpu().numpy(), rad, block.plan.axis.cpu().numpy(), DIM, weight=qn)
    assert_within(block.out[Q].view(B, T, HEADS, DIM), want, UBF * np.abs(want) + 4 * pre, "queries")

    # attention over the encoder's states
    vis = np.arange(L) < lengths.cpu().numpy()[:, None]
    q, k, v = f64(block.out[Q].view(B, T, HEADS, DIM)), f64(block.k), f64(block.v)
    want, size = ob.attention(q, k, v, vis, DIM ** -0.5)
    d = (DIM + 8) * U32 * DIM ** -0.5 * np.abs(q).sum(-1).max() * np.abs(k).max()
    assert_within(block.attended, want, UBF * np.abs(want) + (UBF + 2 * d + (L + 64) * U32) * size, "attention")

    # output projection, gate and residual
    y, size = linear64(block, OUT)
    assert_within(block.out[OUT], y, UBF * np.abs(y) + (HID + 8) * U32 * size, "to_out")
    o = f64(block.out[OUT]).reshape(B, T, HID)
    r, h = ob.gated_norm(f64(x), o, mod[2], mod[4], mod[3])
    assert_within(block.r, r, UBF * np.abs(r) + 4 * U32 * (np.abs(f64(x)) + np.abs(mod[2][:, None] * o)), "residual")
    f = 1 / np.sqrt(((r - r.mean(-1, keepdims=True)) ** 2).mean(-1, keepdims=True) + 1e-6)
    amp = np.abs(1 + mod[4])[:, None] * f * np.abs(r).max(-1, keepdims=True) + np.abs(mod[3])[:, None]
    assert_within(block.h, h, UBF * np.abs(h) + 128 * U32 * amp, "second norm")

    # the last residual
    dn = f64(block.out[DOWN]).reshape(B, T, HID)
    r1 = f64(block.r)
    want = r1 + mod[5][:, None] * dn
    assert_within(result, want, UBF * np.abs(want) + 4 * U32 * (np.abs(r1) + np.abs(mod[5][:, None] * dn)), "result")
    y, size = linear64(block, DOWN, ids, block.out[UP])
    assert_within(block.out[DOWN], y, 2 * UBF * size + (MLP + 8) * U32 * size, "down")


@pytest.mark.parametrize("adapters", [False, True])
def test_equal_to_the_calls_one_by_one(adapters):
    block, (temb, x, pos, ids), states, lengths = make(adapters)
    ids = ids if adapters else None
    block.encode(states, lengths)
    got = block(temb, x, pos, ids).clone()

    def lin(name, z, amax=None):
        lo = block.lora.get(name)
        epi = CROSS_LAYERS[name][1]
        if amax is None and lo is not None and ids is not None:
            return nv.linear(z, block.weights[name], name, epilogue=epi, lora=(lo[0], lo[1], ids, lo[2]))
        return nv.linear(z, block.weights[name], name, epilogue=epi)
    m = nv.gemm_bf16(temb, block.weights[MOD]).chunk(6, 1)
    _, h = nv.gated_norm(x, scale=m[1], shift=m[0])
    q = lin(Q, h.view(-1, HID)).view(B, T, HEADS, DIM)
    q = nv.rotary(q, pos, block.plan, q_weight=block.q_norm)
    kv = nv.linear(states.view(-1, ENC), block.weights[KVP], KVP).view(B, L, 2, KV, DIM)
    k = nv.rotary(kv[:, :, 0], block.no_positions, block.plan, q_weight=block.k_norm)
    a = nv.cross_attention(q, k, kv[:, :, 1], kv_lengths=lengths)
    o = lin(OUT, a.view(B * T, -1)) if OUT not in block.lora else None
    r, h = nv.gated_norm(x, o.view(B, T, HID), gate=m[2], scale=m[4], shift=m[3])
    d = lin(DOWN, lin(UP, h.view(-1, HID)))
    want, none = nv.gated_norm(r, d.view(B, T, HID), gate=m[5], norm=None)
    assert none is None and torch.equal(got, want)


def test_graph_replays_equal_eager_and_follow_the_inputs():
    block, (temb, x, pos, ids), states, lengths = make()
    block.encode(states, lengths)
    g = capture(lambda: block(temb, x, pos, ids))
    for i in range(4):
        x.mul_(0.9)
        lengths[0] = 33 - 7 * i
        want = block(temb, x, pos, ids).clone()
        torch.cuda.synchronize()
        got = g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


@pytest.mark.parametrize("first", ["lengths", "none"])
def test_replay_follows_another_prompt(first):
    # captured under one prompt, replayed under others, whose lengths are tensors of their own
    block, (temb, x, pos, ids), states, lengths = make()
    rng = np.random.default_rng(9)
    block.encode(states, lengths if first == "lengths" else None)
    g = capture(lambda: block(temb, x, pos, ids))
    prompts = [(normal(rng, (B, L, ENC)), n if n is None else torch.tensor(n, dtype=torch.int32, device="cuda"))
               for n in ([3, L], None, [L, 1], [0, 20])]
    seen = []
    for s, n in prompts + [(states, lengths)]:
        block.encode(s, n)
        for _ in range(2):
            want = block(temb, x, pos, ids).clone()
            torch.cuda.synchronize()
            block.result.fill_(7.0)
            got = g.replay()
            torch.cuda.synchronize()
            assert torch.equal(got, want)
        seen.append(want)
        # as with a block that never saw another prompt
        fresh = make()[0]
        fresh.encode(s, n)
        assert torch.equal(fresh(temb, x, pos, ids), want)
    assert all(not torch.equal(a, b) for i, a in enumerate(seen) for b in seen[:i])


def test_lengths_are_the_prompts():
    block, (temb, x, pos, ids), states, lengths = make(False)
    block.encode(states, lengths)
    want = block(temb, x, pos).clone()
    lengths.zero_()                                   # the caller's again after encode
    assert torch.equal(block(temb, x, pos), want)
    for bad in (lengths.long(), lengths[:1], lengths.cpu(), [L, 5]):
        with pytest.raises(ValueError, match="lengths"):
            block.encode(states, bad)
    assert torch.equal(block(temb, x, pos), want)     # a refused call left the prompt alone


def test_captured_encode_follows_states_and_lengths():
    block, (temb, x, pos, ids), states, lengths = make()
    g = capture(lambda: (block.encode(states, lengths), block(temb, x, pos, ids))[1])
    rng = np.random.default_rng(10)
    other = make()[0]
    for n in ([1, 2], [L, 0], [17, L]):
        states.copy_(normal(rng, (B, L, ENC)))
        lengths.copy_(torch.tensor(n, dtype=torch.int32))
        other.encode(states, lengths)
        want = other(temb, x, pos, ids).clone()
        torch.cuda.synchronize()
        got = g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_text_keys_carry_no_rotary_factor(monkeypatch):
    # a YaRN plan over half of each head: its factor belongs to rotated elements,
    # and the text keys are not rotated
    plan = nv.rotary_plan(32, scaling="yarn", factor=32.0, original_length=4096)
    assert plan.magnitude > 1.3
    monkeypatch.setattr(nv, "rotary_plan", lambda *a, **k: plan)
    block, _, states, lengths = make(False)
    block.encode(states, lengths)
    kv = nv.linear(states.view(-1, ENC), block.weights[KVP], KVP).view(B, L, 2, KV, DIM)
    assert torch.equal(block.v, kv[:, :, 1])
    # bounds as in the norm's own tests: 64 U32 of the row's largest term, and one rounding
    want = ob.normalise(f64(kv[:, :, 0]), "rms", 1e-6) * f64(block.k_norm)
    assert_within(block.k, want, UBF * np.abs(want) + 64 * U32 * np.abs(want).max(-1, keepdims=True), "keys")


def adapted64(block, name, ids, x):
    """A layer with adapters in binary64 on its NVFP4 operands and bf16 input, and the bound on
    what precedes its epilogue: the product's output is rounded once, then the adapters are added
    (their rank values rounded once more)."""
    y, size = linear64(block, name)
    depth = x.shape[1]
    off = UBF * np.abs(y) + (depth + 8) * U32 * size
    down, up, s = (f64(t) for t in block.lora[name])
    i = ids.cpu().numpy()
    full, more = ob.lora_add(y, f64(x), down, up, i, s)
    rank = ob.lora_rank_size(f64(x), down, up, i, s)
    off = (1 + UBF) * off + (UBF * rank + (depth + down.shape[1] + 32) * U32 * more) * 1.01
    return full, off + 2 * U32 * np.abs(full)


def test_mlp_with_adapters():
    block, (temb, x, pos, ids), states, lengths = make()
    block.encode(states, lengths)
    block(temb, x, pos, ids)
    h, u, d = block.h.view(-1, HID), block.out[UP], block.out[DOWN]
    # both inputs are quantized with their producers' amax: the codes of their own
    for name, z in ((UP, h), (DOWN, u)):
        q = nv.quantize(z)
        assert all(torch.equal(a, b) for a, b in zip(block.qbuf[name], q[:3]))
    z, off = adapted64(block, UP, ids, h)
    want = 0.5 * z * np.vectorize(math.erfc)(-z / math.sqrt(2))
    off = 1.13 * off + 2e-5 * np.abs(want)            # GELU's slope and its approximation
    assert_within(u, want, off + UBF * (np.abs(want) + off), "up")
    y, off = adapted64(block, DOWN, ids, u)
    assert_within(d, y, off + UBF * (np.abs(y) + off), "down")
