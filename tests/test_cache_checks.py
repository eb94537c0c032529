"""Argument checks of the NVFP4 cache and the weight-only product that need no GPU: the
Python layer raises ValueError before any pointer reaches the library, the C entry
points report errors before touching a device (fake pointers, never dereferenced)."""

import re

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_05_amd as nv
import oracle.cache as oc
from nvfp4_block_scaled_05_amd import _binding
from nvfp4_block_scaled_05_amd.block_ops import _VIEW
from nvfp4_block_scaled_05_amd.cache_ops import _CACHE
from tests.test_abi import HEADER, lib  # noqa: F401

OK, NULL, SHAPE, ALIGN, WORKSPACE, DEVICE, ARG = 0, -1, -2, -3, -4, -5, -6
A = 1 << 20


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def raises(match, fn, *args, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*args, **kw)


def cache(pages=4, size=16, heads=2, dim=64):
    return nv.kv_cache(pages, size, heads, dim, 4.0, 2.0, device="cpu")


def test_kv_cache_rejects():
    f = nv.kv_cache
    for args in ((0, 16, 1, 64), (1, 0, 1, 64), (1, 24, 1, 64), (1, 16, 0, 64)):
        raises("must be positive", f, *args, device="cpu")
    for dim in (0, 8, 24, 144, 256):
        raises("dim must be", f, 1, 16, 1, dim, device="cpu")
    for amax in (0.0, -1.0, float("inf"), float("nan"), 2.0 ** -97, 2.0 ** 97):
        raises("k_amax", f, 1, 16, 1, 64, k_amax=amax, device="cpu")
        raises("v_amax", f, 1, 16, 1, 64, v_amax=amax, device="cpu")
    c = cache()
    assert c.k_codes.shape == (4, 2, 16, 32) and c.v_scales.shape == (4, 2, 16, 4)
    assert c.amax.tolist() == [4.0, 2.0] and not any(t.any() for t in c[:4])


def wrong_caches(fn, *args, **kw):
    """Every call refuses these in the cache's place."""
    c = cache()
    raises("expected a KvCache", fn, tuple(c), *args, **kw)
    raises("4-D", fn, c._replace(k_codes=u8(4, 16, 32)), *args, **kw)
    raises("not that of a cache", fn, c._replace(k_codes=u8(4, 2, 24, 32)), *args, **kw)
    raises("not that of a cache", fn, c._replace(k_codes=u8(4, 2, 16, 36)), *args, **kw)
    raises("not that of a cache", fn, c._replace(k_codes=u8(0, 2, 16, 32)), *args, **kw)
    raises("k_scales: shape", fn, c._replace(k_scales=u8(4, 2, 16, 5)), *args, **kw)
    raises("v_codes: dtype", fn, c._replace(v_codes=c.v_codes.to(torch.int8)), *args, **kw)
    raises("v_scales: must be contiguous", fn, c._replace(v_scales=u8(4, 2, 4, 16).transpose(2, 3)), *args, **kw)
    raises("amax: shape", fn, c._replace(amax=torch.zeros(1)), *args, **kw)
    raises("amax: dtype", fn, c._replace(amax=torch.zeros(2, dtype=torch.float64)), *args, **kw)


def test_cache_write_rejects():
    f, c, x, s = nv.cache_write, cache(), bf16(2, 5, 2, 64), i32(2)
    raises("GPU tensor", f, c, x, x, s)
    wrong_caches(f, x, x, s)
    raises("3-D or 4-D", f, c, bf16(5, 128), x, s)
    raises("dtype", f, c, x.float(), x, s)
    raises("do not go together", f, c, x, bf16(2, 5, 2, 32), s)
    raises("do not go together", f, c, x, bf16(2, 4, 2, 64), s)
    raises("heads of", f, c, bf16(2, 5, 4, 32), bf16(2, 5, 4, 32), s)
    raises("starts: expected", f, c, x, x, None)
    raises("starts: dtype", f, c, x, x, torch.zeros(2, dtype=torch.int64))
    raises("starts: shape", f, c, x, x, i32(3))
    raises("counts: shape", f, c, x, x, s, counts=i32(2, 1))
    raises("5 entries", f, c, bf16(5, 1, 2, 64), bf16(5, 1, 2, 64), i32(5))
    raises("table: expected a 2-D", f, c, x, x, s, table=i32(2))
    raises("table: dtype", f, c, x, x, s, table=torch.zeros(2, 2, dtype=torch.int64))
    raises("table: shape", f, c, x, x, s, table=i32(3, 2))
    raises("table: must be contiguous", f, c, x, x, s, table=i32(2, 2).t())
    raises("a page for each", f, c, x, x, s, table=i32(2, 0))
    raises("power of two", f, cache(size=48), x, x, s, table=i32(2, 2))
    raises("dev_status: dtype", f, c, x, x, s, dev_status=torch.zeros(1))
    raises("multiples of 8", f, c, bf16(2, 5, 2, 68)[..., :64], x, s)


def test_cache_read_rejects():
    f, c, s = nv.cache_read, cache(), i32(2)
    raises("GPU tensor", f, c, 5, s)
    wrong_caches(f, 5, s)
    raises("negative", f, c, -1, s)
    raises("starts: dtype", f, c, 5, torch.zeros(2))
    raises("counts: shape", f, c, 5, s, counts=i32(2, 2))
    raises("starts: shape", f, c, 5, i32(3), counts=i32(2))
    raises("tuple of 2", f, c, 5, s, out=bf16(2, 5, 2, 64))
    raises("out v: shape", f, c, 5, s, out=(bf16(2, 5, 2, 64), bf16(2, 4, 2, 64)))
    raises("out k: shape", f, c, 5, out=(bf16(2, 5, 2, 64), bf16(2, 5, 2, 64)))
    raises("out k: elements overlap", f, c, 5, s, out=(bf16(2, 1, 2, 64).expand(2, 5, 2, 64), bf16(2, 5, 2, 64)))
    same = bf16(2, 5, 2, 64)
    raises("same buffer", f, c, 5, s, out=(same, same))
    raises("table: shape", f, c, 5, s, table=i32(1, 4))


def test_cache_attention_rejects():
    f, c, q, n = nv.cache_attention, cache(), bf16(2, 3, 4, 64), i32(2)
    raises("GPU tensor", f, q, c, n)
    wrong_caches(lambda cc, *a: f(q, cc, *a), n)
    raises("3-D or 4-D", f, bf16(3, 64), c, n)
    raises("dtype", f, q.half(), c, n)
    raises("head size 32", f, bf16(2, 3, 4, 32), c, n)
    raises("3 heads", f, bf16(2, 3, 3, 64), c, n)
    raises("0 heads", f, bf16(2, 3, 0, 64), c, n)
    raises("5 entries", f, bf16(5, 1, 4, 64), c, i32(5))
    raises("lengths: expected", f, q, c, None)
    raises("lengths: shape", f, q, c, i32(1))
    raises("starts: dtype", f, q, c, n, starts=torch.zeros(2))
    raises("table: shape", f, q, c, n, table=i32(1, 2))
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        raises("scale must", f, q, c, n, scale=scale)
    raises("out: shape", f, q, c, n, out=bf16(2, 3, 4, 32))
    raises("out: elements overlap", f, q, c, n, out=bf16(1, 3, 4, 64).expand(2, 3, 4, 64))
    raises("workspace: dtype", f, q, c, n, workspace=torch.zeros(256))


def test_gemm_weight_only_rejects():
    f, x = nv.gemm_weight_only, bf16(2, 64)
    w = nv.Nvfp4Tensor(u8(8, 32), u8(8, 4), torch.zeros(1), 64)
    raises("GPU tensor", f, x, w)
    raises("2-D", f, bf16(64), w)
    raises("dtype", f, x.half(), w)
    raises("contiguous", f, bf16(64, 2).t(), w)
    raises("Nvfp4Tensor", f, x, tuple(w))
    raises("K mismatch", f, bf16(2, 80), w)
    raises("scales: shape", f, x, w._replace(scales=u8(8, 5)))
    raises("bias: shape", f, x, w, bias=bf16(9))
    raises("epilogue must be", f, x, w, epilogue="relu")
    raises("y_amax: dtype", f, x, w, y_amax=bf16(1))
    raises("out: shape", f, x, w, out=bf16(2, 9))


def test_declared_and_exported(lib):  # noqa: F811
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b((?:kv|w4)_\w+)\s*\(", text)))
    assert names == ["kv_cache_attention", "kv_cache_attention_workspace_bytes", "kv_cache_read", "kv_cache_write",
                     "w4_gemm_weight_only"]
    for n in names:
        assert n in _binding.SIGNATURES and hasattr(lib, n)


def late(status):
    """What a call with nothing wrong in its arguments gives without a gfx950."""
    return status == DEVICE


def gpu():
    return torch.cuda.is_available()


def cview(kc=A, ks=A, vc=A, vs=A, amax=A, pages=4, size=16, heads=2, dim=64, table=0, per=0):
    return _CACHE(kc, ks, vc, vs, amax, pages, size, heads, dim, table, per)


BAD_CACHES = [dict(pages=0), dict(pages=1 << 31), dict(size=0), dict(size=24), dict(size=-16), dict(heads=0),
              dict(heads=1 << 17), dict(dim=0), dict(dim=72), dict(dim=144), dict(pages=1),
              dict(table=A, per=-1), dict(table=A, per=2, size=48), dict(table=A, per=1 << 28),
              dict(size=(1 << 31) - 16)]
BAD_PLACES = [dict(kc=A + 8), dict(vc=A + 4), dict(ks=A + 2), dict(vs=A + 1), dict(amax=A + 2),
              dict(table=A + 2, per=2)]


@pytest.mark.skipif(gpu(), reason="fake pointers")
def test_write_and_read_c(lib):  # noqa: F811
    for name, status in (("kv_cache_write", True), ("kv_cache_read", False)):
        def f(c=cview(), k=_VIEW(A, 640, 128, 64), v=_VIEW(A, 640, 128, 64), batch=2, tokens=5, starts=A, counts=None,
              word=None):
            fn = getattr(lib, name)
            return fn(c, k, v, batch, tokens, starts, counts, word, None) if status else fn(
                c, k, v, batch, tokens, starts, counts, None)
        assert late(f()) and late(f(c=cview(table=A, per=2))) and late(f(batch=0)) and late(f(tokens=0))
        assert f(c=None) == NULL and f(k=None) == NULL and f(v=None) == NULL
        assert f(k=_VIEW(0, 640, 128, 64)) == NULL and f(c=cview(kc=0)) == NULL and f(c=cview(amax=0)) == NULL
        assert f(starts=None) == (NULL if status else DEVICE)
        for kw in BAD_CACHES:
            assert f(c=cview(**kw)) == SHAPE, kw
        for kw in BAD_PLACES:
            assert f(c=cview(**kw)) == ALIGN, kw
        assert f(batch=-1) == SHAPE and f(tokens=1 << 31) == SHAPE and f(batch=5) == SHAPE
        assert f(c=cview(table=A, per=2), batch=1 << 20, tokens=1 << 10) == SHAPE
        assert f(k=_VIEW(A, 640, 124, 64)) == SHAPE and f(v=_VIEW(A, -8, 128, 64)) == SHAPE
        assert f(k=_VIEW(A + 8, 640, 128, 64)) == ALIGN and f(counts=A + 1) == ALIGN and f(starts=A + 2) == ALIGN
        if status:
            assert f(word=A + 2) == ALIGN


@pytest.mark.skipif(gpu(), reason="fake pointers")
def test_attention_c(lib):  # noqa: F811
    def f(c=cview(), q=_VIEW(A, 768, 256, 64), lengths=A, starts=None, batch=2, queries=3, heads=4, scale=0.125,
          out=_VIEW(A, 768, 256, 64), ws=None, n=0):
        return lib.kv_cache_attention(c, q, lengths, starts, batch, queries, heads, scale, out, ws, n, None)
    assert late(f()) and late(f(c=cview(table=A, per=2), starts=A)) and late(f(batch=0)) and late(f(queries=0))
    assert f(c=None) == NULL and f(q=None) == NULL and f(out=None) == NULL and f(lengths=None) == NULL
    assert f(q=_VIEW(0, 768, 256, 64)) == NULL and f(c=cview(vs=0)) == NULL
    for kw in BAD_CACHES:
        assert f(c=cview(**kw)) == SHAPE, kw
    for kw in BAD_PLACES:
        assert f(c=cview(**kw)) == ALIGN, kw
    assert f(heads=3) == SHAPE and f(heads=0) == SHAPE and f(heads=1 << 17) == SHAPE and f(queries=-1) == SHAPE
    assert f(c=cview(table=A, per=2), batch=1 << 29) == SHAPE
    # rows times tiles past 32 bits
    assert f(c=cview(table=A, per=1 << 20), batch=64, queries=4096) == SHAPE
    assert f(q=_VIEW(A, 768, 252, 64)) == SHAPE and f(out=_VIEW(A, 768, 256, -64)) == SHAPE
    assert f(q=_VIEW(A + 2, 768, 256, 64)) == ALIGN and f(lengths=A + 1) == ALIGN and f(starts=A + 1) == ALIGN
    assert f(ws=A + 128, n=1 << 20) == ALIGN
    for scale in (0.0, -1.0, float("nan"), float("inf"), 1e-39):
        assert f(scale=scale) == ARG
    assert lib.kv_cache_attention_workspace_bytes(2, 3, 3, 2, 64, 64) == 0
    assert lib.kv_cache_attention_workspace_bytes(-1, 3, 4, 2, 64, 64) == 0
    assert lib.kv_cache_attention_workspace_bytes(2, 3, 4, 2, 72, 64) == 0


@pytest.mark.skipif(gpu(), reason="fake pointers")
def test_weight_only_c(lib):  # noqa: F811
    def f(x=A, codes=A, scales=A, ts=A, bias=None, m=2, n=8, k=64, epi=0, y=A, amax=None):
        return lib.w4_gemm_weight_only(x, codes, scales, ts, bias, m, n, k, epi, y, amax, None)
    assert late(f()) and late(f(m=0, x=None)) and late(f(n=0, codes=None))
    for kw in (dict(x=None), dict(codes=None), dict(scales=None), dict(ts=None), dict(y=None)):
        assert f(**kw) == NULL
    for kw in (dict(m=-1), dict(k=0), dict(k=72), dict(k=1 << 30), dict(m=1 << 20), dict(n=1 << 27)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(x=A + 8), dict(codes=A + 4), dict(ts=A + 2), dict(bias=A + 1), dict(y=A + 4), dict(amax=A + 2)):
        assert f(**kw) == ALIGN, kw
    assert f(epi=2) == ARG


# ------------------------------------------------------------------------ the oracle

def test_oracle_places():
    table = np.array([[2, -1, 0], [1, 3, 4]], np.int32)
    assert oc.place(table, 16, 4, 0, 0) == (2, 0) and oc.place(table, 16, 4, 0, 47) == (0, 15)
    assert oc.place(table, 16, 4, 0, 16) is None and oc.place(table, 16, 4, 1, 32) is None
    assert oc.place(table, 16, 4, 0, 48) is None and oc.place(table, 16, 4, 0, -1) is None
    assert oc.place(None, 16, 4, 3, 15) == (3, 15) and oc.place(None, 16, 4, 3, 16) is None


def test_oracle_held_and_attention():
    codes, scales = np.array([[0x21, 0xF0] * 4], np.uint8), np.array([[0x38]], np.uint8)
    # 0x21: 0.5 then 1; 0xF0: 0 then -6; E4M3 0x38 is 1
    assert oc.held(codes, scales, 2.0).tolist() == [[1.0, 2.0, 0.0, -12.0] * 4]
    assert np.isnan(oc.held(codes, np.array([[0x7F]], np.uint8), 1.0)).all()
    q, k, v = np.zeros((2, 2, 4)), np.ones((3, 1, 4)), np.arange(12.0).reshape(3, 1, 4)
    visible = np.array([[True, False, True], [False] * 3])
    out, size = oc.attention(q, k, v, visible, 1.0)
    assert np.allclose(out[0], (v[0] + v[2]) / 2) and np.allclose(size[0], out[0]) and not out[1].any()
    bits = np.full((1, 32), 0x3F80, np.uint16)
    bits[0, 20] = 0x7F80
    c, s, _ = oc.quantized_rows(bits, 6.0)
    assert s[0, 1] == 0x7F and s[0, 0] < 0x7F and c[0, :8].all() and not c[0, 8:].any()


def test_prompts_in_4_bits_need_the_projections_amax(monkeypatch):
    """Values are quantized under the amax of the projection's epilogue, which a projection in bf16 has
    not: a block that would hold them under some other is refused."""
    from nvfp4_block_scaled_05_amd import dit_block
    monkeypatch.setattr(dit_block, "layer_is_quantized", lambda name: name != "transformer_blocks.0.attn.add_kv_proj")
    raises("add_kv_proj", dit_block.DitCrossBlock, {"w_q": bf16(64, 64)}, 1, 16, 16, 1, 1, None, None, None, held="nvfp4")


def test_gemm_weight_only_does_not_write_over_its_input():
    """Workgroups read all of x while others write their columns of out."""
    x, w = bf16(3, 64), nv.Nvfp4Tensor(u8(64, 32), u8(64, 4), torch.zeros(1), 64)
    raises("same buffer", nv.gemm_weight_only, x, w, out=x)
    raises("same buffer", nv.gemm_weight_only, x, w, out=x.view(3, 64))
    raises("GPU tensor", nv.gemm_weight_only, x, w, out=bf16(3, 64))


@pytest.mark.skipif(gpu(), reason="fake pointers")
def test_sizes_on_both_sides_of_the_documented_limits(lib):  # noqa: F811
    one = _VIEW(A, 768, 256, 64)
    # batch * tokens * kv_heads * dim / 16 below 2^31
    c = cview(table=A, per=2)
    for batch, tokens, want in ((89478485, 3, DEVICE), (89478486, 3, SHAPE), (1, 268435455, DEVICE), (1, 1 << 28, SHAPE)):
        assert lib.kv_cache_write(c, one, one, batch, tokens, A, None, None, None) == want, (batch, tokens)
        assert lib.kv_cache_read(c, one, one, batch, tokens, None, None, None) == want, (batch, tokens)
    # 192 units of (tiles of 64 keys and six): below 2^31
    for per, want in ((44739216, DEVICE), (44739220, SHAPE)):
        assert lib.kv_cache_attention(cview(table=A, per=per), one, A, None, 96, 1, 4, 0.125, one, None, 0, None) == want, per
    # a capacity below 2^31 - 256
    for size, want in (((1 << 31) - 272, DEVICE), ((1 << 31) - 256, SHAPE)):
        assert lib.kv_cache_attention(cview(size=size), one, A, None, 1, 1, 4, 0.125, one, None, 0, None) == want, size
        assert lib.kv_cache_write(cview(size=size), one, one, 1, 1, A, None, None, None) == want, size
    assert lib.kv_cache_attention_workspace_bytes(1, 1, 4, 2, 64, (1 << 31) - 272) != 0
    assert lib.kv_cache_attention_workspace_bytes(1, 1, 4, 2, 64, (1 << 31) - 256) == 0
