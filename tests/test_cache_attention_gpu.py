"""cache_attention against its definition in binary64 on the numbers that the cache
holds, element by element (bounds in cache_util)."""

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_05_amd as nv
from nvfp4_block_scaled_05_amd.graph import capture
from tests.block_util import normal
from tests.cache_util import check, filled, ints, numbers_of, shuffled_table
from tests.gpu_util import bits_of

pytestmark = pytest.mark.gpu


def run(rng, batch, queries, heads, kv, dim, page, per, lengths, causal=False, std=1.0, workspace="own", paged=True):
    pages = batch * per + 1 if paged else batch
    table = shuffled_table(rng, batch, per, pages) if paged else None
    dev_table = None if table is None else torch.from_numpy(table).cuda()
    cache, k, v = filled(rng, pages, page, kv, dim, std)
    q = normal(rng, (batch, queries, heads, dim), std)
    starts = [max(n - queries, 0) for n in lengths] if causal else None
    kw = {} if workspace == "own" else {"workspace": None}
    got = nv.cache_attention(q, cache, ints(*lengths), starts=None if starts is None else ints(*starts),
                             table=dev_table, **kw)
    check(got, q, k, v, lengths, starts, table)
    return got, (q, cache, dev_table)


@pytest.mark.parametrize("workspace", ["own", "none"])
@pytest.mark.parametrize("batch,queries,heads,kv,dim,page,per,lengths", [
    (1, 1, 1, 1, 16, 16, 1, [1]), (1, 1, 1, 1, 128, 16, 1, [16]), (2, 1, 8, 2, 128, 64, 3, [192, 65]),
    (3, 1, 5, 1, 64, 16, 5, [80, 17, 0]), (2, 1, 16, 2, 96, 32, 4, [31, 128]), (4, 1, 8, 8, 112, 128, 2, [129, 256, 1, 0]),
    (2, 3, 12, 4, 128, 16, 8, [127, 33]), (1, 16, 1, 1, 128, 64, 2, [100]), (1, 17, 1, 1, 128, 64, 2, [128]),
    (2, 8, 4, 1, 64, 16, 9, [144, 130]), (1, 33, 1, 1, 80, 32, 3, [96]), (1, 16, 4, 1, 128, 64, 4, [250]),
    (2, 21, 3, 1, 48, 16, 6, [96, 70]), (1, 65, 1, 1, 128, 16, 9, [144]), (2, 33, 4, 2, 64, 64, 3, [190, 64]),
    (1, 130, 2, 2, 128, 256, 1, [256]), (2, 100, 6, 3, 96, 32, 5, [160, 3]), (1, 257, 2, 1, 32, 16, 12, [191])])
def test_shapes(batch, queries, heads, kv, dim, page, per, lengths, workspace):
    run(np.random.default_rng(dim + queries), batch, queries, heads, kv, dim, page, per, lengths, workspace=workspace)


@pytest.mark.parametrize("workspace", ["own", "none"])
@pytest.mark.parametrize("batch,queries,heads,kv,dim,page,per,lengths", [
    (1, 1, 4, 4, 64, 16, 2, [32]), (2, 5, 2, 1, 128, 16, 4, [64, 9]), (2, 16, 4, 4, 128, 32, 3, [96, 16]),
    (3, 7, 6, 2, 80, 16, 3, [48, 7, 3]), (1, 60, 1, 1, 128, 64, 2, [127]), (2, 40, 4, 2, 64, 16, 9, [144, 41]),
    (1, 140, 2, 2, 128, 64, 4, [256]), (2, 131, 3, 1, 96, 32, 6, [192, 131]), (2, 90, 2, 1, 128, 16, 10, [150, 20])])
def test_causal(batch, queries, heads, kv, dim, page, per, lengths, workspace):
    run(np.random.default_rng(dim + queries), batch, queries, heads, kv, dim, page, per, lengths, causal=True,
        workspace=workspace)


@pytest.mark.parametrize("queries", [1, 20, 150])
def test_without_a_table(queries):
    run(np.random.default_rng(3), 3, queries, 4, 2, 128, 208, 1, [208, 77, 1], paged=False)
    run(np.random.default_rng(4), 2, queries, 4, 2, 64, 48, 1, [48, 33], causal=True, paged=False)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("batch,queries,heads,kv,page,per,lengths,causal", [
    (1, 1, 8, 2, 64, 80, [5100], False), (5, 1, 4, 1, 256, 12, [3000, 1, 0, 700, 2049], False),
    (1, 90, 1, 1, 64, 30, [1900], False), (3, 25, 3, 1, 64, 30, [1900, 5, 1200], True),
    (2, 9, 4, 1, 128, 18, [2300, 1111], True), (2, 100, 2, 1, 64, 30, [1900, 700], True),
    (70, 1, 2, 1, 16, 24, [(37 * i) % 385 for i in range(70)], False),
    (150, 1, 8, 4, 64, 20, [(97 * i) % 1281 for i in range(150)], False)])
def test_keys_dealt_over_workgroups(dim, batch, queries, heads, kv, page, per, lengths, causal):
    run(np.random.default_rng(page + dim), batch, queries, heads, kv, dim, page, per, lengths, causal=causal)


@pytest.mark.parametrize("batch,queries,heads,kv,page,per,lengths,causal", [
    (300, 1, 8, 4, 64, 20, [(53 * i) % 1281 for i in range(300)], False),
    (5, 40, 64, 64, 64, 6, [384, 1, 0, 200, 333], False), (5, 40, 64, 64, 32, 12, [384, 40, 41, 200, 333], True)])
def test_units_that_fill_the_card(batch, queries, heads, kv, page, per, lengths, causal):
    """More units than are dealt: each is one workgroup's, whatever the lengths."""
    assert nv.cache_attention_workspace(batch, queries, heads, kv, 64, page * per) is None
    run(np.random.default_rng(batch), batch, queries, heads, kv, 64, page, per, lengths, causal=causal)


@pytest.mark.parametrize("queries", [1, 30, 100])
def test_lengths_outside_the_capacity_are_taken_within(queries):
    rng = np.random.default_rng(5)
    cache, k, v = filled(rng, 3, 32, 1, 64)
    q = normal(rng, (3, queries, 2, 64))
    got = nv.cache_attention(q, cache, ints(2 ** 31 - 1, -4, 33))
    check(got, q, k, v, [32, 0, 32])
    got = nv.cache_attention(q, cache, ints(32, 32, 32), starts=ints(-2 ** 31, 2 ** 31 - 1, -queries))
    check(got, q, k, v, [32, 32, 32], [-2 ** 31, 2 ** 31 - 1, -queries])
    assert not got[0].any() and not got[2].any()


@pytest.mark.parametrize("queries", [1, 17, 50, 130])
@pytest.mark.parametrize("dim", [64, 96, 128])
def test_pages_that_are_none_are_not_seen(queries, dim):
    """Also where the pages that the table does not name hold NaN."""
    rng = np.random.default_rng(6)
    cache, k, v = filled(rng, 6, 16, 2, dim)
    for t in (cache.k_scales, cache.v_scales):
        t[0] = 0x7F
    table = np.array([[1, -1, 2, 6, 3], [-7, 2 ** 31 - 1, 4, 5, -1], [-1, -1, -1, -1, -1]], np.int32)
    q = normal(rng, (3, queries, 4, dim))
    got = nv.cache_attention(q, cache, ints(80, 57, 80), table=torch.from_numpy(table).cuda())
    check(got, q, k, v, [80, 57, 80], None, table)
    assert not got[2].any()


@pytest.mark.parametrize("queries", [2, 12, 40, 150])
@pytest.mark.parametrize("dim", [48, 64, 128])
@pytest.mark.parametrize("what", ["key", "value"])
def test_nan_reaches_the_rows_that_see_it(queries, dim, what):
    """A NaN block of a key makes the rows that see it NaN, one of a value the columns
    of its block; other rows and heads stay as without it."""
    rng = np.random.default_rng(queries)
    batch, heads, kv, page, per = 2, 4, 2, 16, 16
    lengths = [200, 231]
    table = shuffled_table(rng, batch, per, batch * per)
    dev_table = torch.from_numpy(table).cuda()
    cache, _, _ = filled(rng, batch * per, page, kv, dim)
    q = normal(rng, (batch, queries, heads, dim))
    starts = [n - queries for n in lengths]
    call = dict(starts=ints(*starts), table=dev_table)
    clean = nv.cache_attention(q, cache, ints(*lengths), **call)
    at = starts[1] + queries // 2                  # a position that only later queries see
    block = dim // 16 - 1
    (cache.k_scales if what == "key" else cache.v_scales)[int(table[1, at // page]), 1, at % page, block] = 0x7F
    # behind the last position of entry 0: never seen
    cache.k_scales[int(table[0, lengths[0] // page]), :, lengths[0] % page:] = 0x7F
    cache.v_scales[int(table[0, lengths[0] // page]), :, lengths[0] % page:] = 0x7F
    got = nv.cache_attention(q, cache, ints(*lengths), **call)
    hit = torch.zeros_like(got, dtype=torch.bool)
    cols = slice(None) if what == "key" else slice(16 * block, 16 * block + 16)
    hit[1, queries // 2:, 2:, cols] = True
    assert torch.equal(torch.isnan(got), hit)
    assert torch.equal(got[~hit], clean[~hit])
    # without the order all rows see it
    got = nv.cache_attention(q, cache, ints(*lengths), table=dev_table)
    hit[1, :, 2:, cols] = True
    assert torch.equal(torch.isnan(got), hit)


@pytest.mark.parametrize("queries", [1, 40, 100])
@pytest.mark.parametrize("where", [0, 700])
def test_nan_in_a_part_of_its_own_is_not_lost(queries, where):
    """Also where its keys weigh nothing beside the others."""
    rng = np.random.default_rng(13)
    cache, _, _ = filled(rng, 1, 1024, 1, 128)
    q = normal(rng, (1, queries, 1, 128), 0.1)
    cache.v_scales[0, 0, where, 2] = 0x7F
    got = nv.cache_attention(q, cache, ints(1024))
    hit = torch.zeros_like(got, dtype=torch.bool)
    hit[..., 32:48] = True
    assert torch.equal(torch.isnan(got), hit)
    cache.k_scales[0, 0, where, 7] = 0x7F
    assert torch.isnan(nv.cache_attention(q, cache, ints(1024))).all()


@pytest.mark.parametrize("queries", [1, 20, 100])
def test_infinite_queries(queries):
    """Scores of -infinity weigh nothing, rows of them alone are zeros; +infinity is NaN."""
    rng = np.random.default_rng(14)
    cache, k, v = filled(rng, 1, 64, 1, 64)
    cache.k_codes[0, 0, :, 0] = 0x22              # elements 0 and 1 of every key: 1, with a scale of their own
    cache.k_scales[0, 0, :, 0] = 0x38
    q = normal(rng, (1, queries, 2, 64))
    clean = nv.cache_attention(q, cache, ints(64))
    bad = q.clone()
    bad[0, 0, 1, 0] = -float("inf")
    got = nv.cache_attention(bad, cache, ints(64))
    assert not got[0, 0, 1].any()
    bad[0, 0, 1, 0] = float("inf")
    got = nv.cache_attention(bad, cache, ints(64))
    assert torch.isnan(got[0, 0, 1]).all()
    mask = torch.ones_like(got, dtype=torch.bool)
    mask[0, 0, 1] = False
    assert torch.equal(got[mask], clean[mask])
    # keys whose element is 1 are out, those whose element is -1 would be +infinity: the
    # second half of the keys has 0 there, which -infinity makes NaN
    cache.k_codes[0, 0, 32:, 0] = 0
    bad[0, 0, 1, 0] = -float("inf")
    assert torch.isnan(nv.cache_attention(bad, cache, ints(64))[0, 0, 1]).all()
    assert not nv.cache_attention(bad, cache, ints(32))[0, 0, 1].any()


@pytest.mark.parametrize("queries", [1, 20, 100])
@pytest.mark.parametrize("power", [-120, -60, 20, 100])
def test_queries_of_any_size(queries, power):
    """fp16 holds them by a power of two a row; the scale undoes it."""
    rng = np.random.default_rng(15)
    cache, k, v = filled(rng, 1, 160, 2, 128)
    q = normal(rng, (1, queries, 4, 128)) * 2.0 ** power
    q[0, 0, 0, 1:] *= 2.0 ** -9                   # one row of very unequal elements
    scale = 2.0 ** -power * 128 ** -0.5
    got = nv.cache_attention(q, cache, ints(160), scale=scale)
    check(got, q, k, v, [160], scale=scale)
    zero = torch.zeros_like(q)
    got = nv.cache_attention(zero, cache, ints(160), scale=scale)
    check(got, zero, k, v, [160], scale=scale)


@pytest.mark.parametrize("queries", [1, 20, 100])
@pytest.mark.parametrize("std", [4.0, 8.0])
def test_sharp_and_growing_scores(queries, std):
    """Scores of hundreds, and maxima that grow along the keys."""
    rng = np.random.default_rng(16)
    cache, k, v = filled(rng, 1, 512, 1, 64, std, k_amax=32.0, v_amax=32.0)
    q = normal(rng, (1, queries, 3, 64), std)
    check(nv.cache_attention(q, cache, ints(512)), q, k, v, [512])
    ramp = torch.linspace(0.05, 1, 512).view(1, 512, 1, 1).cuda()
    x = (ramp * q[:, :1, :1].float()).to(torch.bfloat16).contiguous()
    nv.cache_write(cache, x, normal(rng, (1, 512, 1, 64)), ints(0))
    k, v = numbers_of(cache)
    check(nv.cache_attention(q, cache, ints(512)), q, k, v, [512])


@pytest.mark.parametrize("amax", [(1e-3, 4e4), (2.0 ** 40, 2.0 ** -40)])
def test_tensor_scales(amax):
    rng = np.random.default_rng(17)
    ka, va = float(np.float32(amax[0])), float(np.float32(amax[1]))
    cache = nv.kv_cache(1, 96, 1, 64, ka, va)
    nv.cache_write(cache, normal(rng, (1, 96, 1, 64), ka / 4), normal(rng, (1, 96, 1, 64), va / 4), ints(0))
    k, v = numbers_of(cache)
    for queries in (1, 80):
        q = normal(rng, (1, queries, 1, 64))
        check(nv.cache_attention(q, cache, ints(96), scale=1 / ka), q, k, v, [96], scale=1 / ka)


def test_views_and_outputs():
    rng = np.random.default_rng(18)
    cache, k, v = filled(rng, 2, 64, 2, 64)
    for queries in (1, 9, 120):
        qkv = normal(rng, (2, queries, 8, 64))
        out = torch.full((2, queries, 6, 64), 5.0, dtype=torch.bfloat16, device="cuda")
        got = nv.cache_attention(qkv[:, :, 2:6], cache, ints(64, 50), out=out[:, :, 1:5])
        assert got.data_ptr() == out[:, :, 1:5].data_ptr()
        check(got, qkv[:, :, 2:6].contiguous(), k, v, [64, 50])
        assert bool((out[:, :, 0] == 5).all()) and bool((out[:, :, 5] == 5).all())
        one = nv.cache_attention(qkv[1, :, 2:6], cache, ints(40))       # no batch dimension: entry 0
        assert one.shape == (queries, 4, 64)
        check(one[None], qkv[1:, :, 2:6].contiguous(), k, v, [40])


@pytest.mark.parametrize("queries", [1, 24, 100])
def test_shared_pages_and_repeated_calls(queries):
    """Entries that share a prefix's pages; the same bits every time, whatever the workspace held."""
    rng = np.random.default_rng(19)
    cache, k, v = filled(rng, 24, 64, 1, 128)
    table = np.stack([np.arange(20), np.r_[np.arange(18), 20, 21], np.r_[np.arange(18), 22, 23]]).astype(np.int32)
    dev_table = torch.from_numpy(table).cuda()
    lengths = [1280, 1279, 1153]
    q = normal(rng, (3, queries, 4, 128))
    ws = nv.cache_attention_workspace(3, queries, 4, 1, 128, 1280)
    assert ws is not None
    got = nv.cache_attention(q, cache, ints(*lengths), table=dev_table, workspace=ws)
    check(got, q, k, v, lengths, None, table)
    for fill in (0, 0xFF, 0x7F):
        ws.fill_(fill)
        again = nv.cache_attention(q, cache, ints(*lengths), table=dev_table, workspace=ws)
        assert np.array_equal(bits_of(again), bits_of(got))
    small = nv.cache_attention(q, cache, ints(*lengths), table=dev_table, workspace=ws[:256])
    whole = nv.cache_attention(q, cache, ints(*lengths), table=dev_table, workspace=None)
    assert np.array_equal(bits_of(small), bits_of(whole))
    check(whole, q, k, v, lengths, None, table)


def test_empty_calls():
    rng = np.random.default_rng(20)
    cache, _, _ = filled(rng, 2, 16, 1, 64)
    q = normal(rng, (2, 3, 2, 64))
    assert nv.cache_attention(q[:, :0], cache, ints(1, 1)).shape == (2, 0, 2, 64)
    assert nv.cache_attention(q[:0], cache, ints()).shape == (0, 3, 2, 64)
    for queries in (1, 20, 100):
        out = torch.full((2, queries, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
        nv.cache_attention(normal(rng, (2, queries, 2, 64)), cache, ints(0, 0), out=out)
        assert not out.any()


@pytest.mark.parametrize("queries", [1, 100])
def test_captured_with_changing_lengths_and_tables(queries):
    """One graph, replayed after the lengths, the table and the cache have changed; two
    graphs with workspaces of their own."""
    rng = np.random.default_rng(21)
    cache, k, v = filled(rng, 40, 32, 2, 64)
    q = normal(rng, (2, queries, 4, 64))
    lengths, starts = ints(1, 1), ints(0, 0)
    table = torch.zeros((2, 20), dtype=torch.int32, device="cuda")
    graphs = []
    for causal in (False, True):
        out = torch.empty_like(q)
        ws = nv.cache_attention_workspace(2, queries, 4, 2, 64, 640)

        def step(causal=causal, out=out, ws=ws):
            return nv.cache_attention(q, cache, lengths, starts=starts if causal else None, table=table, out=out,
                                      workspace=ws)
        graphs.append((causal, capture(step), ws))
    for n in ([640, 0], [3, 500], [600, 640]):
        host = shuffled_table(rng, 2, 20, 40)
        table.copy_(torch.from_numpy(host))
        lengths.copy_(ints(*n))
        begin = [max(m - queries, 0) for m in n]
        starts.copy_(ints(*begin))
        for causal, g, _ in graphs:
            got = g.replay()
            torch.cuda.synchronize()
            check(got, q, k, v, n, begin if causal else None, host)


def test_two_streams():
    rng = np.random.default_rng(22)
    cache, _, _ = filled(rng, 2, 2048, 2, 128)
    qs = [normal(rng, (2, n, 8, 128)) for n in (1, 1, 70, 70)]
    want = [nv.cache_attention(q, cache, ints(2048, 1500)) for q in qs]
    lengths = ints(2048, 1500)
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for q, s in zip(qs, streams):
            with torch.cuda.stream(s):
                got.append(nv.cache_attention(q, cache, lengths))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert np.array_equal(bits_of(g), bits_of(want[i % 4]))


def test_offsets_past_32_bits():
    rng = np.random.default_rng(23)
    pages = 41000
    cache = nv.kv_cache(pages, 256, 8, 128, 9.0, 5.0)
    table = ints(pages - 1, 3, 33000, pages - 2).view(2, 2)
    small = nv.kv_cache(4, 256, 8, 128, 9.0, 5.0)
    little = ints(3, 0, 1, 2).view(2, 2)
    k, v = normal(rng, (2, 512, 8, 128)), normal(rng, (2, 512, 8, 128))
    nv.cache_write(cache, k, v, ints(0, 0), table=table)
    nv.cache_write(small, k, v, ints(0, 0), table=little)
    for queries in (1, 20, 70):
        q = normal(rng, (2, queries, 8, 128))
        got = nv.cache_attention(q, cache, ints(512, 300), table=table)
        assert np.array_equal(bits_of(got), bits_of(nv.cache_attention(q, small, ints(512, 300), table=little)))
    del cache
    torch.cuda.empty_cache()


@pytest.mark.parametrize("workspace", ["own", "none"])
@pytest.mark.parametrize("dim", [16, 48, 80, 96, 112])
@pytest.mark.parametrize("batch,queries,heads,kv,page,per,lengths,causal", [
    (2, 1, 8, 2, 64, 80, [5100, 1111], False), (2, 9, 4, 2, 128, 18, [2300, 1000], True),
    (2, 30, 1, 1, 16, 130, [2079, 0], False), (1, 90, 2, 1, 64, 30, [1900], True),
    (2, 40, 2, 2, 64, 18, [1100, 1024], False)])
def test_padded_heads_over_long_caches(dim, batch, queries, heads, kv, page, per, lengths, causal, workspace):
    """Head sizes between those that the kernels have, over keys enough for the rings to turn, and for
    parts that are joined."""
    own = nv.cache_attention_workspace(batch, queries, heads, kv, dim, page * per)
    assert own is not None
    run(np.random.default_rng(page + dim), batch, queries, heads, kv, dim, page, per, lengths, causal=causal,
        workspace=workspace)


@pytest.mark.parametrize("dim", [48, 128])
@pytest.mark.parametrize("queries", [1, 25, 70])
def test_keys_dealt_without_a_table(queries, dim):
    run(np.random.default_rng(queries + dim), 2, queries, 2, 2, dim, 2512, 1, [2512, 1777], paged=False)
    run(np.random.default_rng(queries), 2, queries, 2, 1, dim, 1040, 1, [1040, 601], causal=True, paged=False)


@pytest.mark.parametrize("dim", [64, 112])
def test_many_rows_of_more_entries_than_lanes(dim):
    lengths = [(37 * i) % 385 for i in range(70)]
    assert nv.cache_attention_workspace(70, 20, 2, 1, dim, 384) is not None
    run(np.random.default_rng(dim), 70, 20, 2, 1, dim, 16, 24, lengths)
    run(np.random.default_rng(dim), 70, 20, 2, 1, dim, 16, 24, lengths, causal=True)


@pytest.mark.parametrize("queries", [1, 20, 100])
@pytest.mark.parametrize("amax,k_std,q", [(2.0 ** -88, 2.0 ** -90, 2.0 ** -38), (2688.0, 0.25, 2.0 ** -126),
                                          (2688.0, 2.0 ** -6, 2.0 ** -122)])
def test_the_largest_scale(queries, amax, k_std, q):
    """A scale that times log2(e) is past binary32, over keys or queries that bring the scores back into
    range.  (A row's elements are of one magnitude: at the bottom of bf16's range smaller ones lose bits.)"""
    rng = np.random.default_rng(24)
    cache = nv.kv_cache(1, 96, 1, 64, amax, 4.0)
    nv.cache_write(cache, normal(rng, (1, 96, 1, 64), k_std), normal(rng, (1, 96, 1, 64)), ints(0))
    k, v = numbers_of(cache)
    q = torch.from_numpy(np.sign(rng.standard_normal((1, queries, 1, 64))) * q).to(torch.bfloat16).cuda()
    check(nv.cache_attention(q, cache, ints(96), scale=3.0e38), q, k, v, [96], scale=3.0e38)
