"""cross_attention against its definition in binary64, element by element.

Bounds, fixed before the first run, relative to W = sum_j w_j |v_j| (what the
output would be without cancellation): each weight is rounded to bf16 (UBF);
a score is a binary32 sum of dim exact products and a few more roundings, off
by d = (dim + 8) U32 scale max_j sum |q k|, which changes a weight by at most
2 d relative (its own and the sum's); the weights' and outputs' binary32 sums
and the exponentials add (keys + 64) U32.  The output rounding is UBF of the
value."""

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_05_amd as nv
import oracle.block as ob
from nvfp4_block_scaled_05_amd.graph import capture
from tests.block_util import U32, UBF, assert_within, f64, normal

pytestmark = pytest.mark.gpu


def visible_of(batch, keys, lengths=None, mask=None):
    v = np.ones((batch, keys), bool)
    if lengths is not None:
        v &= np.arange(keys) < np.asarray(lengths.cpu())[:, None]
    if mask is not None:
        v &= mask.cpu().numpy().astype(bool)
    return v


def check(got, q, k, v, lengths=None, mask=None, scale=None):
    dim, keys = q.shape[3], k.shape[1]
    scale = scale or dim ** -0.5
    vis = visible_of(q.shape[0], keys, lengths, mask)
    kk, vv = f64(k), f64(v)
    kk[~vis] = 0
    want, size = ob.attention(f64(q), kk, f64(v), vis, scale)
    most = np.abs(f64(q)).sum(-1).max() * (np.abs(kk).max() if kk.size else 0)
    d = (dim + 8) * U32 * scale * most
    assert_within(got, want, UBF * np.abs(want) + (UBF + 2 * d + (keys + 64) * U32) * size)


def make(seed, batch, queries, keys, heads, kv, dim, std=1.0):
    rng = np.random.default_rng(seed)
    return (normal(rng, (batch, queries, heads, dim), std), normal(rng, (batch, keys, kv, dim), std),
            normal(rng, (batch, keys, kv, dim)))


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("batch,queries,keys,heads,kv,dim", [
    (1, 1, 1, 1, 1, 8), (1, 1, 1, 1, 1, 128), (1, 32, 64, 1, 1, 64), (1, 32, 64, 1, 1, 128),
    (2, 33, 65, 2, 2, 64), (1, 128, 128, 2, 1, 128), (1, 129, 63, 3, 3, 72), (2, 31, 200, 4, 2, 80),
    (1, 257, 130, 6, 2, 96), (3, 5, 77, 24, 8, 128), (1, 1, 5000, 8, 2, 128), (2, 1, 4097, 6, 6, 64),
    (1, 7, 3001, 4, 1, 40), (1, 700, 513, 2, 2, 128), (1, 1, 70, 3, 1, 16), (4, 2, 1000, 2, 1, 120)])
def test_shapes(batch, queries, keys, heads, kv, dim):
    q, k, v = make(keys + dim, batch, queries, keys, heads, kv, dim)
    check(nv.cross_attention(q, k, v), q, k, v)
    check(nv.cross_attention(q, k, v, workspace=None), q, k, v)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("queries", [1, 40])
def test_lengths(dim, queries):
    b, keys = 7, 2100
    q, k, v = make(dim, b, queries, keys, 4, 2, dim)
    lengths = ints(0, 1, 63, 64, 65, 2099, 2100)
    for i, n in enumerate(lengths.tolist()):
        k[i, n:] = float("nan")
        v[i, n:] = float("inf")
    for ws in ({}, {"workspace": None}):
        got = nv.cross_attention(q, k, v, kv_lengths=lengths, **ws)
        check(got, q, k, v, lengths)
        assert torch.equal(got[0], torch.zeros_like(got[0]))
    # lengths outside [0, keys] are taken as the nearest end
    far = ints(-5, 1, 63, 64, 65, 2099, 1 << 30)
    assert torch.equal(nv.cross_attention(q, k, v, kv_lengths=far, workspace=None), got)


@pytest.mark.parametrize("dim", [64, 80, 128])
@pytest.mark.parametrize("queries", [1, 70])
@pytest.mark.parametrize("dtype", [torch.bool, torch.uint8])
def test_key_mask(dim, queries, dtype):
    rng = np.random.default_rng(dim + queries)
    b, keys = 6, 1301
    q, k, v = make(dim, b, queries, keys, 4, 1, dim)
    m = rng.random((b, keys)) < 0.7
    m[1] = False                        # nothing left
    m[2, :1200] = False                 # whole tiles out of sight, then some keys
    m[3] = False
    m[3, 700] = True                    # one key
    m[4] = True
    mask = torch.from_numpy(m).to(dtype).cuda()
    if dtype == torch.uint8:
        mask *= 200                     # any nonzero byte counts
    hidden = torch.from_numpy(~m).cuda()
    k[hidden] = float("nan")
    v[hidden] = float("nan")
    v[hidden.roll(1, 0) & hidden] = torch.finfo(torch.bfloat16).min
    lengths = ints(1301, 1301, 1301, 1301, 900, 100)
    for kw in ({"mask": mask}, {"mask": mask, "lengths": lengths}):
        for ws in ({}, {"workspace": None}):
            got = nv.cross_attention(q, k, v, key_mask=mask, kv_lengths=kw.get("lengths"), **ws)
            check(got, q, k, v, **kw)
            assert torch.equal(got[1], torch.zeros_like(got[1]))
            if kw.get("lengths") is None:
                want = v[3, 700].unsqueeze(1).expand(1, 4, dim)
                assert torch.equal(got[3], want.expand(queries, 4, dim))


def test_views_of_fused_projections():
    rng = np.random.default_rng(3)
    qkv = normal(rng, (2, 50, 12, 64))
    kv = normal(rng, (2, 90, 2, 4, 64))
    q, k, v = qkv[:, :, 2:10], kv[:, :, 0], kv[:, :, 1]
    want = nv.cross_attention(q.contiguous(), k.contiguous(), v.contiguous())
    check(want, q, k, v)
    assert torch.equal(nv.cross_attention(q, k, v), want)
    # into a strided output, whose other parts stay
    wide = torch.full((2, 50, 10, 72), 3.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, :, 1:9, :64]
    nv.cross_attention(q, k, v, out=out)
    assert torch.equal(out, want)
    out.fill_(3.0)
    assert torch.equal(wide, torch.full_like(wide, 3.0))
    # heads before tokens in memory; one encoding for the whole batch; 3-D
    qt = q.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(nv.cross_attention(qt, k, v), want)
    e, f = k[:1].expand(2, -1, -1, -1), v[:1].expand(2, -1, -1, -1)
    assert torch.equal(nv.cross_attention(q, e, f), nv.cross_attention(q, e.contiguous(), f.contiguous()))
    assert torch.equal(nv.cross_attention(q[1], k[1], v[1]), want[1])


@pytest.mark.parametrize("queries", [3, 200])
def test_large_scores_and_scale(queries):
    # scores to a few hundred: the running maximum moves, weights underflow
    q, k, v = make(9, 1, queries, 900, 2, 2, 128, std=4.0)
    check(nv.cross_attention(q, k, v, scale=0.3), q, k, v, scale=0.3)
    # ascending scores: the maximum moves in every tile
    k2 = k * torch.linspace(0.01, 3, 900, device="cuda").bfloat16()[None, :, None, None]
    q2 = q.abs()
    k2 = k2.abs()
    check(nv.cross_attention(q2, k2, v), q2, k2, v)
    # descending: weights of later tiles vanish
    k3 = k2.flip(1).contiguous()
    check(nv.cross_attention(q2, k3, v), q2, k3, v)
    # all scores far below zero: the softmax does not see a common offset
    check(nv.cross_attention(-q2, k2, v), -q2, k2, v)


@pytest.mark.parametrize("queries", [3, 200])
@pytest.mark.parametrize("hidden", [slice(0, 330), slice(128, 700), slice(0, 900)])
def test_scores_of_minus_infinity_weigh_nothing(queries, hidden):
    q, k, v = make(14, 1, queries, 900, 2, 1, 128)
    q = q.abs() + 0.1
    k[:, hidden] = float("-inf")
    mask = torch.ones(1, 900, dtype=torch.bool, device="cuda")
    mask[:, hidden] = False
    for ws in ({}, {"workspace": None}):
        got = nv.cross_attention(q, k, v, **ws)
        check(got, q, k, v, mask=mask)
        assert torch.equal(got, nv.cross_attention(q, k, v, key_mask=mask, **ws))


def test_nan_stays_in_its_query_and_head():
    q, k, v = make(10, 1, 70, 200, 4, 2, 64)
    want = nv.cross_attention(q, k, v)
    q[0, 9, 2, 5] = float("nan")
    got = nv.cross_attention(q, k, v)
    assert torch.isnan(got[0, 9, 2]).all()
    got[0, 9, 2] = want[0, 9, 2]
    assert torch.equal(got, want)
    v[0, 3, 0, 7] = float("inf")             # seen: its column of heads 0 and 1
    got = nv.cross_attention(q, k, v)
    assert torch.isinf(got[0, :, :2, 7]).all()
    assert torch.equal(got[0, :, 3], want[0, :, 3])


def test_long_key_offsets():
    # keys whose elements lie past 2^31 elements from the first
    token = (1 << 23) - 8
    keys = 300
    pool = torch.zeros(token * keys + 256, dtype=torch.bfloat16, device="cuda")
    k = pool.as_strided((1, keys, 1, 64), (0, token, 64, 1))
    v = pool.as_strided((1, keys, 1, 64), (0, token, 64, 1), 64)
    q, k0, v0 = make(11, 1, 3, keys, 2, 1, 64)
    k.copy_(k0)
    v.copy_(v0)
    assert torch.equal(nv.cross_attention(q, k, v), nv.cross_attention(q, k0, v0))


def test_empty_calls():
    q, k, v = make(12, 2, 5, 9, 2, 1, 64)
    assert nv.cross_attention(q[:, :0], k, v).shape == (2, 0, 2, 64)
    assert torch.equal(nv.cross_attention(q, k[:, :0], v[:, :0]), torch.zeros_like(q))


def test_same_bits_every_time_and_workspace_reuse():
    q, k, v = make(13, 2, 1, 6000, 8, 4, 128)
    ws = nv.cross_attention_workspace(2, 1, 6000, 8, 4, 128)
    assert ws is not None
    ws.fill_(255)                            # contents on entry do not matter
    a = nv.cross_attention(q, k, v, workspace=ws)
    for _ in range(3):
        assert torch.equal(nv.cross_attention(q, k, v, workspace=ws), a)
    assert torch.equal(nv.cross_attention(q, k, v), a)
    small = ws[:256]                         # too small: no split, still right
    check(nv.cross_attention(q, k, v, workspace=small), q, k, v)


@pytest.mark.parametrize("dim", [40, 64, 96, 128])
@pytest.mark.parametrize("queries,heads,kv", [(1, 3, 1), (11, 3, 1), (45, 3, 1), (150, 2, 2)])
def test_many_splits(queries, heads, kv, dim):
    # splits that see all, some and none of their keys; a workspace of NaNs
    keys = 4100
    q, k, v = make(dim + queries, 3, queries, keys, heads, kv, dim)
    lengths = ints(keys, 1900, 70)
    mask = torch.ones(3, keys, dtype=torch.bool, device="cuda")
    mask[0, 512:2700] = False
    mask[1, :1700] = False
    ws = nv.cross_attention_workspace(3, queries, keys, heads, kv, dim)
    assert ws is not None
    for kw in ({}, {"kv_lengths": lengths}, {"kv_lengths": lengths, "key_mask": mask}):
        ws.fill_(255)
        got = nv.cross_attention(q, k, v, workspace=ws, **kw)
        check(got, q, k, v, lengths=kw.get("kv_lengths"), mask=kw.get("key_mask"))


def test_captured_and_on_two_streams():
    q, k, v = make(14, 2, 3, 2000, 4, 2, 64)
    lengths = ints(2000, 17)
    out = torch.empty_like(q)
    ws = nv.cross_attention_workspace(2, 3, 2000, 4, 2, 64)
    g = capture(lambda: nv.cross_attention(q, k, v, kv_lengths=lengths, out=out, workspace=ws))
    for n in (3, 1999, 640):
        lengths[1] = n
        q.mul_(-1)
        want = nv.cross_attention(q, k, v, kv_lengths=lengths)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    sets = [make(40 + i, 1, 2, 3000, 4, 4, 128) for i in range(2)]
    want = [nv.cross_attention(*s) for s in sets]
    torch.cuda.synchronize()
    got = [None, None]
    for i in range(2):
        with torch.cuda.stream(torch.cuda.Stream()):
            got[i] = nv.cross_attention(*sets[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("queries", [1, 40])
@pytest.mark.parametrize("what", ["key", "value", "infinity"])
def test_nan_in_a_split_of_its_own_is_not_lost(what, queries):
    # one visible key among 2000 hidden ones, so some split sees that key alone
    q, k, v = make(15, 1, queries, 4100, 2, 1, 64)
    q = q.abs() + 0.5
    mask = torch.ones(1, 4100, dtype=torch.bool, device="cuda")
    mask[0, 1000:3000] = False
    mask[0, 2000] = True
    ws = nv.cross_attention_workspace(1, queries, 4100, 2, 1, 64)
    assert ws is not None
    if what == "key":                        # a score that is no number: no weight is one
        k[0, 2000] = float("nan")
    else:                                    # a weight of 2^-1000 or less is 0, and 0 times these is NaN
        k[0, 2000] = -500.0
        v[0, 2000, 0, 7] = float("nan" if what == "value" else "inf")
    for w in (ws, None):
        got = nv.cross_attention(q, k, v, key_mask=mask, workspace=w)
        gone = torch.isnan(got)
        if what == "key":
            assert gone.all()
        else:
            assert gone[..., 7].all()
            gone[..., 7] = False
            assert not gone.any()


@pytest.mark.parametrize("queries", [3, 200])
def test_rows_of_minus_infinity_are_zeros_whatever_the_values(queries):
    q, k, v = make(16, 1, queries, 900, 2, 1, 64)
    q = q.abs() + 0.1
    k[:] = float("-inf")
    v[..., 5] = float("nan")
    v[..., 6] = float("inf")
    for ws in ({}, {"workspace": None}):
        got = nv.cross_attention(q, k, v, **ws)
        assert torch.equal(got, torch.zeros_like(got))


@pytest.mark.parametrize("dim", [64, 80, 128])
@pytest.mark.parametrize("batch,queries,keys,heads,kv", [
    (1, 300, 333, 11, 11), (3, 150, 333, 8, 4), (2, 129, 70, 27, 9),
    (2, 1500, 130, 24, 24), (5, 601, 200, 12, 6)])         # and more units than workgroups run at once
def test_heads_side_by_side_over_several_row_tiles(batch, queries, keys, heads, kv, dim):
    # at least eight kv heads (one a chiplet, and some left over) with several row tiles each
    rng = np.random.default_rng(dim + keys)
    q, k, v = make(dim + queries, batch, queries, keys, heads, kv, dim)
    lengths = torch.from_numpy(rng.integers(keys // 3, keys + 1, batch)).int().cuda()
    lengths[0] = keys
    mask = torch.from_numpy(rng.random((batch, keys)) < 0.8).cuda()
    for kw in ({}, {"kv_lengths": lengths, "key_mask": mask}):
        want = nv.cross_attention(q, k, v, workspace=None, **kw)
        check(want, q, k, v, lengths=kw.get("kv_lengths"), mask=kw.get("key_mask"))
        check(nv.cross_attention(q, k, v, **kw), q, k, v, lengths=kw.get("kv_lengths"), mask=kw.get("key_mask"))
        # a head alone, where nothing lies side by side: the same bits
        for b, h in ((0, 0), (batch - 1, heads - 1), (batch // 2, heads // 2)):
            g = h // (heads // kv)
            one = nv.cross_attention(q[b:b + 1, :, h:h + 1], k[b:b + 1, :, g:g + 1], v[b:b + 1, :, g:g + 1],
                                     workspace=None, **{n: t[b:b + 1].contiguous() for n, t in kw.items()})
            assert torch.equal(one, want[b:b + 1, :, h:h + 1])


@pytest.mark.parametrize("queries,heads,kv,dim", [(1, 40, 1, 64), (3, 40, 1, 128), (20, 7, 1, 128), (9, 66, 2, 40),
                                                  (33, 13, 1, 64)])
def test_many_heads_share_a_key_head(queries, heads, kv, dim):
    # a group that is longer than a load's rows, shorter, and no divisor of them
    q, k, v = make(heads, 2, queries, 300, heads, kv, dim)
    wide = torch.from_numpy(np.random.default_rng(1).random((2, 390)) < 0.7).cuda()
    for mask in (wide[:, 50:350], wide[:1, 7:307].expand(2, -1)):       # a part of a wider mask; one for all
        check(nv.cross_attention(q, k, v, key_mask=mask), q, k, v, mask=mask)
