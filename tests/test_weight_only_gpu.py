"""gemm_weight_only against its definition in binary64.

Bounds, fixed before the first run, on W = sW sum_k |x w|: products are exact, their
binary32 sum over K terms and the waves' is off by at most (K + 8) U32 W, the tensor
scale, bias and a GELU of slope at most 1.13 (and 2e-5 of its own value) add a few
more; the output rounding is UBF of the value."""

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_05_amd as nv
import oracle
import oracle.cache as oc
from nvfp4_block_scaled_05_amd.graph import capture
from tests.block_util import U32, UBF, assert_within, f64, normal
from tests.gpu_util import bits_of

pytestmark = pytest.mark.gpu


def values(w):
    return oc.held(w.codes.cpu().numpy(), w.scales.cpu().numpy(), w.tensor_scale.item())


def check(got, x, w, bias=None, gelu=False):
    ww, xx = values(w), f64(x)
    want, size = xx @ ww.T, np.abs(xx) @ np.abs(ww).T
    if bias is not None:
        want = want + f64(bias)
        size = size + np.abs(f64(bias))
    off = (x.shape[1] + 8) * U32 * size
    if gelu:
        want = oracle.gelu_f64(want)
        off = 1.13 * off + 2e-5 * np.abs(want)
    assert_within(got, want, off * (1 + UBF) + UBF * np.abs(want))


def weight(rng, n, k, std=0.05):
    return nv.quantize_weight(normal(rng, (n, k), std))


@pytest.mark.parametrize("n,k", [(1, 16), (1, 128), (3, 48), (16, 2048), (17, 144), (100, 528), (1111, 2064), (64, 16),
                                 (4096, 256), (33, 8192), (2000, 1040)])
@pytest.mark.parametrize("rows", [1, 2, 5, 16, 17, 40, 64])
def test_shapes(rows, n, k):
    rng = np.random.default_rng(n + k + rows)
    x, w = normal(rng, (rows, k)), weight(rng, n, k)
    check(nv.gemm_weight_only(x, w), x, w)


@pytest.mark.parametrize("n,k", [(6150, 256), (6144, 528), (12300, 512), (12288, 272), (16500, 768), (500, 4096)])
@pytest.mark.parametrize("rows", [1, 2, 3, 8, 9, 16, 31, 50])
def test_every_kernel(rows, n, k):
    """Output counts and inner sizes on both sides of the launch's rules, ragged last tiles; NaN and
    infinite rows of x beside the others."""
    rng = np.random.default_rng(n + k + rows)
    x, w = normal(rng, (rows, k)), weight(rng, n, k)
    bias, amax = normal(rng, (n,)), torch.zeros(1, device="cuda")
    got = nv.gemm_weight_only(x, w, bias=bias, y_amax=amax)
    check(got, x, w, bias)
    assert amax.item() == got.abs().max().item()
    if rows > 1:
        x[rows // 2, k - 1] = float("nan")
        bad = nv.gemm_weight_only(x, w, bias=bias)
        keep = [r for r in range(rows) if r != rows // 2]
        assert torch.isnan(bad[rows // 2]).all() and torch.equal(bad[keep], got[keep])


@pytest.mark.parametrize("steps", [1, 3, 4, 9])
@pytest.mark.parametrize("rows", [3, 15, 16])
@pytest.mark.parametrize("tiles", [-1, 0, 1])
@pytest.mark.parametrize("part", [1, 2])
def test_rings_of_a_compute_unit(part, tiles, rows, steps):
    """Tiles of 16 outputs on both sides of one and two a compute unit, the last one ragged; steps of 256
    that leave some waves without one and some with more than others."""
    n = 16 * (part * torch.cuda.get_device_properties(0).multi_processor_count + tiles) - 5
    rng = np.random.default_rng(n + rows + steps)
    x, w, bias = normal(rng, (rows, 256 * steps)), weight(rng, n, 256 * steps), normal(rng, (n,))
    check(nv.gemm_weight_only(x, w), x, w)
    check(nv.gemm_weight_only(x, w, bias=bias, epilogue="gelu"), x, w, bias, True)


@pytest.mark.parametrize("rows", [1, 2, 7, 20])
def test_weights_at_any_place(rows):
    """Codes at 8 bytes and scales at any byte, as slices of one checkpoint buffer lie."""
    rng = np.random.default_rng(rows)
    n, k = 12300, 512
    w, x = weight(rng, n, k), normal(rng, (rows, k))
    buffer = torch.zeros(n * k // 2 + n * k // 16 + 64, dtype=torch.uint8, device="cuda")
    codes = buffer[8:8 + n * k // 2].view(n, k // 2)
    scales = buffer[8 + n * k // 2 + 3:][:n * k // 16].view(n, k // 16)
    codes.copy_(w.codes)
    scales.copy_(w.scales)
    moved = nv.Nvfp4Tensor(codes, scales, w.tensor_scale, k)
    assert codes.data_ptr() % 16 == 8 and scales.data_ptr() % 2 == 1
    check(nv.gemm_weight_only(x, moved), x, w)


@pytest.mark.parametrize("rows", [65, 129, 300])
def test_more_rows_than_one_pass(rows):
    rng = np.random.default_rng(rows)
    x, w = normal(rng, (rows, 272)), weight(rng, 70, 272)
    check(nv.gemm_weight_only(x, w), x, w)


@pytest.mark.parametrize("rows", [1, 7, 33, 64, 70])
@pytest.mark.parametrize("n", [32, 77])
@pytest.mark.parametrize("gelu", [False, True])
def test_bias_epilogue_and_amax(rows, n, gelu):
    rng = np.random.default_rng(rows + n)
    x, w, bias = normal(rng, (rows, 320)), weight(rng, n, 320, 0.2), normal(rng, (n,))
    amax = torch.full((1,), 1e9, device="cuda")
    got = nv.gemm_weight_only(x, w, bias=bias, epilogue="gelu" if gelu else "none", y_amax=amax)
    check(got, x, w, bias, gelu)
    assert amax.item() == got.abs().max().item()
    # the amax is what the quantizer takes
    if n % 16 == 0:
        a, b = nv.quantize(got, amax=amax), nv.quantize(got)
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)


def test_rows_do_not_depend_on_each_other():
    """A row's bits are the same wherever it stands; NaN stays in its row."""
    rng = np.random.default_rng(1)
    x, w = normal(rng, (16, 1040)), weight(rng, 50, 1040)
    y = nv.gemm_weight_only(x, w)
    order = torch.from_numpy(rng.permutation(16)).cuda()
    assert np.array_equal(bits_of(nv.gemm_weight_only(x[order].contiguous(), w)), bits_of(y[order]))
    x[3, 1000] = float("nan")
    x[5, 0] = float("inf")
    amax = torch.zeros(1, device="cuda")
    z = nv.gemm_weight_only(x, w, y_amax=amax)
    assert torch.isnan(z[3]).all() and not torch.isfinite(z[5]).any() and not torch.isfinite(amax).any()
    keep = [r for r in range(16) if r not in (3, 5)]
    assert torch.equal(z[keep], y[keep])


@pytest.mark.parametrize("power", [-100, 60, 110])
def test_activations_of_any_size(power):
    rng = np.random.default_rng(2)
    x, w = normal(rng, (4, 256)) * 2.0 ** power, weight(rng, 24, 256)
    check(nv.gemm_weight_only(x, w), x, w)


def test_outlier_columns():
    rng = np.random.default_rng(3)
    x = normal(rng, (9, 1024))
    x[:, ::97] *= 1000
    w = weight(rng, 48, 1024)
    w.scales[5] = 0                                # a row of zeros
    w.scales[6, ::2] = 0x7E                        # the largest scale beside small ones
    check(nv.gemm_weight_only(x, w), x, w)


def test_zero_rows_and_columns():
    rng = np.random.default_rng(4)
    w = weight(rng, 32, 64)
    amax = torch.ones(1, device="cuda")
    y = nv.gemm_weight_only(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), w, y_amax=amax)
    assert y.shape == (0, 32) and amax.item() == 0


def test_linear_and_out():
    rng = np.random.default_rng(5)
    x, w, bias = normal(rng, (3, 128)), weight(rng, 64, 128), normal(rng, (64,))
    name = "transformer_blocks.0.attn.to_q"
    y = nv.linear(x, w, name, bias=bias, weight_only=True)
    out = torch.empty_like(y)
    assert nv.gemm_weight_only(x, w, bias=bias, out=out) is out
    assert torch.equal(y, out)
    # a layer that is not quantized has a bf16 weight and stays what it is
    dense = normal(rng, (64, 128))
    a = nv.linear(x, dense, "proj_out", weight_only=True)
    assert torch.equal(a, nv.linear(x, dense, "proj_out"))
    # adapters are added from the same x
    down, up = normal(rng, (2, 8, 128), 0.1), normal(rng, (2, 64, 8), 0.1)
    ids = torch.tensor([1, -1, 0], dtype=torch.int32, device="cuda")
    got = nv.linear(x, w, name, lora=(down, up, ids, None), weight_only=True)
    assert torch.equal(got, nv.lora_add(nv.gemm_weight_only(x, w), x, down, up, ids))


def test_captured():
    rng = np.random.default_rng(6)
    x, w = normal(rng, (5, 512)), weight(rng, 96, 512)
    out, amax = torch.empty((5, 96), dtype=torch.bfloat16, device="cuda"), torch.zeros(1, device="cuda")
    g = capture(lambda: nv.gemm_weight_only(x, w, epilogue="gelu", y_amax=amax, out=out))
    for _ in range(4):
        x.copy_(normal(rng, (5, 512)))
        g.replay()
        torch.cuda.synchronize()
        check(out, x, w, gelu=True)
        assert amax.item() == out.abs().max().item()
        assert torch.equal(out, nv.gemm_weight_only(x, w, epilogue="gelu"))


def test_offsets_past_32_bits():
    """A weight of more than 2^32 bytes of codes: its last rows as if they were alone."""
    rng = np.random.default_rng(7)
    n, k = 524320, 16384                           # 4.3 GB of codes
    codes = torch.zeros((n, k // 2), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((n, k // 16), dtype=torch.uint8, device="cuda")
    last = weight(rng, 32, k)
    codes[-32:], scales[-32:] = last.codes, last.scales
    x = normal(rng, (2, k))
    y = nv.gemm_weight_only(x, nv.Nvfp4Tensor(codes, scales, last.tensor_scale, k))
    assert torch.equal(y[:, -32:], nv.gemm_weight_only(x, last)) and not y[:, :-32].any()
    del codes, scales
    torch.cuda.empty_cache()


@pytest.mark.parametrize("steps", [9, 17, 20])
def test_many_rows_in_rings_that_turn(steps):
    """17 rows and more of a large weight, whose steps of 256 are eight waves' in turn: one to three of a
    wave, unequal over the waves, so that both stages, the wait for all but the next step's loads and
    both turns of the loop are run."""
    n = 48 * torch.cuda.get_device_properties(0).multi_processor_count + 5
    rng = np.random.default_rng(steps)
    w, bias = weight(rng, n, 256 * steps), normal(rng, (n,))
    ww = values(w)
    for rows in (17, 31, 50):
        x, amax = normal(rng, (rows, 256 * steps)), torch.zeros(1, device="cuda")
        got = nv.gemm_weight_only(x, w, bias=bias, y_amax=amax)
        xx = f64(x)
        want, size = xx @ ww.T + f64(bias), np.abs(xx) @ np.abs(ww).T + np.abs(f64(bias))
        assert_within(got, want, (256 * steps + 8) * U32 * size * (1 + UBF) + UBF * np.abs(want), f"{rows} rows")
        assert amax.item() == got.abs().max().item()


@pytest.mark.parametrize("k", [8208, 10000, 28672])
@pytest.mark.parametrize("rows", [1, 2])
def test_one_or_two_rows_in_several_chunks_a_wave(rows, k):
    """Inner sizes past four waves' chunks of 2048, a ragged last one among them."""
    rng = np.random.default_rng(k + rows)
    x, w, bias = normal(rng, (rows, k)), weight(rng, 70, k), normal(rng, (70,))
    check(nv.gemm_weight_only(x, w, bias=bias, epilogue="gelu"), x, w, bias, True)


@pytest.mark.parametrize("k", [16384, 16400])
def test_offsets_past_32_bits_of_every_kernel(k):
    """As above against binary64; 16400 is not a multiple of 256, so its codes go straight to registers."""
    rng = np.random.default_rng(k)
    n = 524320
    codes = torch.zeros((n, k // 2), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((n, k // 16), dtype=torch.uint8, device="cuda")
    assert codes.numel() > 2 ** 32
    last = weight(rng, 32, k)
    codes[-32:], scales[-32:] = last.codes, last.scales
    w = nv.Nvfp4Tensor(codes, scales, last.tensor_scale, k)
    for rows in (1, 2, 9, 20):
        x = normal(rng, (rows, k))
        y = nv.gemm_weight_only(x, w)
        check(y[:, -32:], x, last)
        assert not y[:, :-32].any()
    del codes, scales, w
    torch.cuda.empty_cache()
