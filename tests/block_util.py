"""Helpers of the block operators' GPU tests: seeded bf16 / float32 device
tensors with their float64 values, and element-wise bounds.

U32 and UBF are half a step relative to the value: what one rounding to
binary32 / bf16 can be off by."""

import numpy as np
import torch

U32 = 2.0 ** -24
UBF = 2.0 ** -8


def normal(rng, shape, std=1.0, mean=0.0, dtype=torch.bfloat16):
    v = torch.from_numpy(rng.standard_normal(shape) * std + mean).to(dtype)
    return v.cuda()


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def assert_within(got, want, bound, what=""):
    """|got - want| <= bound element by element; got a device tensor."""
    g = f64(got)
    assert g.shape == want.shape, (g.shape, want.shape)
    assert np.isfinite(g).all(), f"{what}: {np.count_nonzero(~np.isfinite(g))} non-finite"
    off = np.abs(g - want) - bound
    if g.size and off.max() > 0:
        i = np.unravel_index(off.argmax(), off.shape)
        b = np.broadcast_to(bound, g.shape)[i]
        raise AssertionError(f"{what} at {i}: got {g[i]!r}, want {want[i]!r}, bound {b:.3e}; "
                             f"{np.count_nonzero(off > 0)} of {g.size} outside")
