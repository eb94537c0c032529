"""The block operators' oracle (oracle/block.py) pinned to closed forms and to
independent torch computations in binary64 (CPU)."""

import math

import numpy as np
import torch

import oracle.block as ob


def rng(seed=0):
    return np.random.default_rng(seed)


def test_norms_against_torch():
    v = rng().standard_normal((3, 5, 24)) * 3 + 1
    t = torch.from_numpy(v)
    want = torch.nn.functional.layer_norm(t, (24,), eps=1e-5).numpy()
    assert np.abs(ob.normalise(v, "layer", 1e-5) - want).max() < 1e-13
    want = torch.nn.functional.rms_norm(t, (24,), eps=1e-5).numpy()
    assert np.abs(ob.normalise(v, "rms", 1e-5) - want).max() < 1e-13
    assert ob.normalise(v, "none", 1e-5) is v


def test_gated_norm_by_hand():
    # one row (1, 3): mean 2, deviation 1; eps 0 gives (-1, 1)
    x, y = np.array([[[0.0, 1.0]]]), np.array([[[0.5, 1.0]]])
    gate, scale, shift = np.array([[2.0, 2.0]]), np.array([[1.0, 0.0]]), np.array([[10.0, 20.0]])
    r, h = ob.gated_norm(x, y, gate, scale, shift, eps=0.0)
    assert np.array_equal(r, [[[1.0, 3.0]]])
    assert np.allclose(h, [[[-1 * 2 + 10, 1 + 20]]], atol=1e-15)
    r, h = ob.gated_norm(x, y, None, None, None, norm="none", post_norm="rms",
                         post_weight=np.array([1.0, 4.0]), residual_scale=0.5, eps=0.0)
    rms = math.sqrt((0.25 + 1) / 2)
    assert np.allclose(r, [[[0.5 / rms, 0.5 + 4 / rms]]]) and h is r


def test_rotary_by_hand_and_its_group_property():
    v = np.zeros((1, 1, 1, 6))
    v[..., :] = [1, 2, 3, 4, 5, 6]
    pos = np.array([[[3]]])
    f = [math.pi / 6, math.pi / 3]          # 3 steps: a quarter and a half turn
    out = ob.rotary(v, pos, f, [0, 0], 4, "interleaved")
    assert np.allclose(out[0, 0, 0], [-2, 1, -3, -4, 5, 6])
    out = ob.rotary(v, pos, f, [0, 0], 4, "half")
    assert np.allclose(out[0, 0, 0], [-3, -2, 1, -4, 5, 6])
    # two axes, and a magnitude
    out = ob.rotary(v, np.array([[[3, 1]]]), [math.pi / 6, math.pi], [0, 1], 4, magnitude=2.0)
    assert np.allclose(out[0, 0, 0], [-4, 2, -6, -8, 5, 6])
    # scores depend on the difference of positions alone
    q, k = rng(1).standard_normal((2, 1, 1, 1, 8))
    f = [0.7, 0.2, 0.05, 0.01]
    s = [np.sum(ob.rotary(q, np.array([[[a]]]), f, [0] * 4, 8) * ob.rotary(k, np.array([[[b]]]), f, [0] * 4, 8))
         for a, b in ((5, 2), (105, 102))]
    assert abs(s[0] - s[1]) < 1e-12


def test_attention_against_torch_and_closed_forms():
    g = rng(2)
    q, k, v = g.standard_normal((2, 5, 4, 8)), g.standard_normal((2, 7, 2, 8)), g.standard_normal((2, 7, 2, 8))
    vis = g.random((2, 7)) < 0.6
    vis[:, 0] = True
    out, size = ob.attention(q, k, v, vis, 0.3)
    t = lambda a: torch.from_numpy(a).transpose(1, 2)
    want = torch.nn.functional.scaled_dot_product_attention(
        t(q), t(k).repeat_interleave(2, 1), t(v).repeat_interleave(2, 1),
        attn_mask=torch.from_numpy(vis)[:, None, None], scale=0.3).transpose(1, 2).numpy()
    assert np.abs(out - want).max() < 1e-13
    assert (size >= np.abs(out) - 1e-15).all()
    # equal scores: the mean of the visible values; none visible: zeros
    vis[1] = False
    out, _ = ob.attention(q * 0, k, np.where(vis[:, :, None, None], v, np.nan), vis, 1.0)
    assert np.allclose(out[0, 3, 1], v[0, vis[0], 0].mean(0)) and not out[1].any()


def test_lora_as_one_dense_weight():
    g = rng(3)
    y, x = g.standard_normal((6, 5)), g.standard_normal((6, 4))
    down, up = g.standard_normal((2, 3, 4)), g.standard_normal((2, 5, 3))
    ids, s = np.array([0, 1, -1, 1, 2, 0]), np.array([0.5, 2.0])
    out, size = ob.lora_add(y, x, down, up, ids, s)
    for m, a in enumerate(ids):
        want = y[m] + (s[a] * up[a] @ down[a] @ x[m] if 0 <= a < 2 else 0)
        assert np.allclose(out[m], want)
    assert (size >= np.abs(out - y) - 1e-12).all()
    assert (ob.lora_rank_size(x, down, up, ids, s) <= size + 1e-12).all()
