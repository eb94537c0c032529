"""The NVFP4 key/value cache as it is written and read back: bytes equal to the
oracle's, what is not written left as it was."""

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_05_amd as nv
import oracle.cache as oc
from nvfp4_block_scaled_05_amd.graph import capture
from tests.block_util import normal
from tests.cache_util import K_AMAX, V_AMAX, ints, shuffled_table
from tests.gpu_util import bits_of

pytestmark = pytest.mark.gpu

LEFT = 0x25                # what places hold before a call


def marked(pages, page_size, kv_heads, dim, k_amax=K_AMAX, v_amax=V_AMAX):
    cache = nv.kv_cache(pages, page_size, kv_heads, dim, k_amax, v_amax)
    for t in cache[:4]:
        t.fill_(LEFT)
    return cache


def check_written(cache, k, v, starts, counts=None, table=None):
    """Every byte of the cache: the oracle's where tokens went, LEFT elsewhere."""
    pages, heads, size, _ = cache.k_codes.shape
    tab = None if table is None else table.cpu().numpy()
    for x, codes, scales, amax in ((k, cache.k_codes, cache.k_scales, cache.amax[0].item()),
                                   (v, cache.v_codes, cache.v_scales, cache.amax[1].item())):
        c, s, _ = oc.quantized_rows(bits_of(x.contiguous()), amax)
        want_c = np.full(tuple(codes.shape), LEFT, np.uint8)
        want_s = np.full(tuple(scales.shape), LEFT, np.uint8)
        for b in range(x.shape[0]):
            n = x.shape[1] if counts is None else min(max(int(counts[b]), 0), x.shape[1])
            for t in range(n):
                at = oc.place(tab, size, pages, b, int(starts[b]) + t)
                if at is not None:
                    want_c[at[0], :, at[1]] = c[b, t]
                    want_s[at[0], :, at[1]] = s[b, t]
        np.testing.assert_array_equal(codes.cpu().numpy(), want_c)
        np.testing.assert_array_equal(scales.cpu().numpy(), want_s)


def check_read(cache, got, tokens, starts, counts=None, table=None):
    """Every bit of what is read: the oracle's, zeros where there is nothing."""
    pages, heads, size, _ = cache.k_codes.shape
    tab = None if table is None else table.cpu().numpy()
    for y, codes, scales, amax in ((got[0], cache.k_codes, cache.k_scales, cache.amax[0].item()),
                                   (got[1], cache.v_codes, cache.v_scales, cache.amax[1].item())):
        c, s = codes.cpu().numpy(), scales.cpu().numpy()
        ts = np.float32(1.0) / (np.float32(2688.0) / np.float32(amax))
        want = np.zeros(tuple(y.shape), np.uint16)
        for b in range(y.shape[0]):
            n = tokens if counts is None else min(max(int(counts[b]), 0), tokens)
            for t in range(n):
                at = oc.place(tab, size, pages, b, int(starts[b]) + t)
                if at is not None:
                    want[b, t] = oc.read_bits(c[at[0], :, at[1]], s[at[0], :, at[1]], ts)
        np.testing.assert_array_equal(bits_of(y.contiguous()), want)


@pytest.mark.parametrize("batch,tokens,heads,dim,page,per,starts,counts", [
    (1, 1, 1, 16, 16, 1, [0], None), (1, 1, 1, 128, 16, 1, [15], None), (3, 1, 8, 128, 64, 2, [0, 63, 64], None),
    (2, 33, 3, 64, 16, 4, [0, 7], None), (2, 33, 5, 80, 32, 3, [1, 40], [33, 12]),
    (4, 20, 2, 112, 16, 3, [0, 5, 16, 31], [20, 0, 1, 17]), (2, 9, 1, 96, 128, 1, [100, 119], [9, 9]),
    (1, 300, 2, 128, 256, 2, [200], None), (5, 3, 24, 32, 16, 1, [0, 1, 2, 3, 13], None)])
def test_write_and_read_paged(batch, tokens, heads, dim, page, per, starts, counts):
    rng = np.random.default_rng(tokens * dim + batch)
    pages = batch * per + 2
    table = torch.from_numpy(shuffled_table(rng, batch, per, pages)).cuda()
    cache = marked(pages, page, heads, dim)
    k, v = normal(rng, (batch, tokens, heads, dim), 2.0), normal(rng, (batch, tokens, heads, dim), 0.7)
    n = None if counts is None else ints(*counts)
    nv.cache_write(cache, k, v, ints(*starts), counts=n, table=table)
    check_written(cache, k, v, starts, counts, table)
    got = nv.cache_read(cache, tokens, ints(*starts), counts=n, table=table)
    check_read(cache, got, tokens, starts, counts, table)
    # from before what was written to past the last page
    early = [s - 5 for s in starts]
    got = nv.cache_read(cache, tokens + per * page, ints(*early), table=table)
    check_read(cache, got, tokens + per * page, early, None, table)


@pytest.mark.parametrize("size", [16, 48, 80, 1008])
@pytest.mark.parametrize("dim", [48, 64, 128])
def test_write_and_read_without_a_table(size, dim):
    rng = np.random.default_rng(size)
    cache = marked(4, size, 3, dim)
    tokens = size + 3                                     # past the page: dropped
    k, v = normal(rng, (3, tokens, 3, dim)), normal(rng, (3, tokens, 3, dim))
    starts = [0, -2, 5]
    nv.cache_write(cache, k, v, ints(*starts))
    check_written(cache, k, v, starts)
    check_read(cache, nv.cache_read(cache, tokens, ints(*starts)), tokens, starts)
    got = nv.cache_read(cache, size)                      # every page from its start
    assert got[0].shape == (4, size, 3, dim)
    check_read(cache, got, size, [0] * 4)
    # one entry, without a batch dimension
    again = marked(4, size, 3, dim)
    nv.cache_write(again, k[0], v[0], ints(0))
    check_written(again, k[:1], v[:1], [0])


def test_bytes_are_those_of_quantize():
    rng = np.random.default_rng(5)
    x, y = normal(rng, (1, 64, 2, 128), 3.0), normal(rng, (1, 64, 2, 128), 0.01)
    cache = nv.kv_cache(1, 64, 2, 128, 12.0, 0.0625)
    nv.cache_write(cache, x, y, ints(0))
    k, v = nv.cache_read(cache, 64)
    for z, codes, scales, amax, back in ((x, cache.k_codes, cache.k_scales, 12.0, k),
                                         (y, cache.v_codes, cache.v_scales, 0.0625, v)):
        q = nv.quantize(z.reshape(128, 128), amax=torch.tensor([amax], device="cuda"))
        assert torch.equal(codes[0].transpose(0, 1).reshape(128, 64), q.codes)
        assert torch.equal(scales[0].transpose(0, 1).reshape(128, 8), q.scales)
        assert torch.equal(back.reshape(128, 128), nv.dequantize(q))


def test_values_at_the_formats_edges():
    """Zeros of both signs, the smallest numbers, the amax, what lies far above it, and
    blocks whose scale rounds to 0."""
    row = torch.zeros(8, 128)
    row[0, ::2] = -0.0
    row[1, :] = 2.0 ** -133
    row[2, 5], row[3, 7] = 9.0, -9.0
    row[4, :] = torch.linspace(-40, 40, 128)
    row[5, :] = 3e38
    row[6, :] = torch.linspace(1e-3, 2e-3, 128)
    row[7, ::16] = 9.0 * 2.0 ** -16
    x = row.to(torch.bfloat16).cuda().view(1, 8, 1, 128)
    cache = marked(1, 16, 1, 128)
    status = torch.ones(1, dtype=torch.int32, device="cuda")
    nv.cache_write(cache, x, x, ints(0), dev_status=status)
    assert status.item() == 0
    check_written(cache, x, x, [0])
    check_read(cache, nv.cache_read(cache, 16), 16, [0])


def test_views_of_a_fused_projection():
    rng = np.random.default_rng(6)
    qkv = normal(rng, (2, 21, 3, 4, 64))
    cache = marked(2, 32, 4, 64)
    nv.cache_write(cache, qkv[:, :, 1], qkv[:, :, 2], ints(3, 0))
    check_written(cache, qkv[:, :, 1], qkv[:, :, 2], [3, 0])
    out = torch.full((2, 21, 2, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    got = nv.cache_read(cache, 21, ints(3, 0), counts=ints(21, 4), out=(out[:, :, 0], out[:, :, 1]))
    assert got[0].data_ptr() == out.data_ptr()
    check_read(cache, got, 21, [3, 0], [21, 4])


def test_pages_that_are_none():
    """Table entries below 0 and past the last page: their tokens are dropped and read as zeros."""
    rng = np.random.default_rng(7)
    table = ints(2, -1, 0, 5, 1, 2 ** 31 - 1).view(2, 3)
    cache = marked(3, 16, 2, 64)
    k, v = normal(rng, (2, 48, 2, 64)), normal(rng, (2, 48, 2, 64))
    nv.cache_write(cache, k, v, ints(0, 0), table=table)
    check_written(cache, k, v, [0, 0], None, table)
    check_read(cache, nv.cache_read(cache, 48, table=table), 48, [0, 0], None, table)


def test_starts_that_would_pass_32_bits():
    rng = np.random.default_rng(8)
    cache = marked(2, 16, 1, 64)
    k, v = normal(rng, (2, 40, 1, 64)), normal(rng, (2, 40, 1, 64))
    starts = [2 ** 31 - 1, -2 ** 31]
    nv.cache_write(cache, k, v, ints(*starts), counts=ints(-5, 2 ** 31 - 1))
    check_written(cache, k, v, starts, [-5, 2 ** 31 - 1])
    check_read(cache, nv.cache_read(cache, 40, ints(*starts)), 40, starts)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_non_finite_blocks_read_as_nan(bad):
    rng = np.random.default_rng(9)
    k, v = normal(rng, (2, 8, 2, 64)), normal(rng, (2, 8, 2, 64))
    k[0, 3, 1, 17] = bad
    v[1, 7, 0, 63] = bad
    cache = marked(2, 16, 2, 64)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    nv.cache_write(cache, k, v, ints(0, 0), dev_status=status)
    assert status.item() == -8
    check_written(cache, k, v, [0, 0])
    gk, gv = nv.cache_read(cache, 8)
    for got, want in ((gk, (0, 3, 1, slice(16, 32))), (gv, (1, 7, 0, slice(48, 64)))):
        nan = torch.zeros_like(got, dtype=torch.bool)
        nan[want] = True
        assert torch.equal(torch.isnan(got), nan)
    # tokens that are not written are not looked at
    nv.cache_write(cache, k, v, ints(0, 0), counts=ints(3, 7), dev_status=status)
    assert status.item() == 0


def test_amax_set_on_the_device():
    rng = np.random.default_rng(10)
    x = normal(rng, (1, 32, 2, 64), 5.0)
    cache = marked(1, 32, 2, 64)
    cache.amax[1:].copy_(x.abs().max())
    nv.cache_write(cache, x, x, ints(0))
    check_written(cache, x, x, [0])
    cache.amax.zero_()                                    # degenerate: all zeros, as in quantize
    nv.cache_write(cache, x, x, ints(0))
    assert not cache.k_scales.any() and not cache.v_scales.any()
    k, v = nv.cache_read(cache, 32)
    assert not k.any() and not v.any()


def test_empty_calls():
    cache = marked(2, 16, 2, 64)
    status = torch.ones(1, dtype=torch.int32, device="cuda")
    none = torch.empty((2, 0, 2, 64), dtype=torch.bfloat16, device="cuda")
    nv.cache_write(cache, none, none, ints(0, 0), dev_status=status)
    nv.cache_write(cache, none[:0].reshape(0, 3, 2, 64), none[:0].reshape(0, 3, 2, 64), ints())
    assert status.item() == 0
    assert all(bool((t == LEFT).all()) for t in cache[:4])
    k, v = nv.cache_read(cache, 0)
    assert k.shape == v.shape == (2, 0, 2, 64)


def test_offsets_past_32_bits():
    """Pages more than 4 GiB into a pool of 5 GiB of codes."""
    rng = np.random.default_rng(11)
    pages = 41000
    cache = nv.kv_cache(pages, 256, 8, 128, K_AMAX, V_AMAX)
    table = ints(pages - 1, 3, 33000, pages - 2).view(2, 2)
    k, v = normal(rng, (2, 300, 8, 128)), normal(rng, (2, 300, 8, 128))
    nv.cache_write(cache, k, v, ints(100, 0), table=table)
    small = nv.kv_cache(4, 256, 8, 128, K_AMAX, V_AMAX)
    nv.cache_write(small, k, v, ints(100, 0), table=ints(3, 0, 1, 2).view(2, 2))
    order = torch.tensor([3, 33000, pages - 2, pages - 1], device="cuda")
    for big, little in zip(cache[:4], small[:4]):
        assert torch.equal(big[order], little)
    got = nv.cache_read(cache, 300, ints(100, 0), table=table)
    want = nv.cache_read(small, 300, ints(100, 0), table=ints(3, 0, 1, 2).view(2, 2))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    del cache
    torch.cuda.empty_cache()


def test_captured_and_on_another_stream():
    rng = np.random.default_rng(12)
    k, v = normal(rng, (2, 5, 2, 64)), normal(rng, (2, 5, 2, 64))
    cache, starts = marked(2, 32, 2, 64), ints(0, 0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = (torch.empty_like(k), torch.empty_like(v))

    def step():
        nv.cache_write(cache, k, v, starts, dev_status=status)
        return nv.cache_read(cache, 5, starts, out=out)

    g = capture(step)
    for i in range(4):
        for t in cache[:4]:
            t.fill_(LEFT)
        k.copy_(normal(rng, (2, 5, 2, 64)))
        starts.copy_(ints(3 * i, 20 - i))
        got = g.replay()
        torch.cuda.synchronize()
        check_written(cache, k, v, starts.tolist())
        check_read(cache, got, 5, starts.tolist())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    check_written(cache, k, v, starts.tolist())
