"""The sizes of test_gpu_b8_paths.py still reach the kernels they are there for, and the torch reference agrees with the
numpy one (no device needed)."""
import numpy as np
import pytest
import torch

import b8_ref as ref
import b8_torch as bt
from test_gpu_b8_paths import LINEAR, PRODUCTS


def test_products_reach_every_tiled_kernel_with_one_and_several_tiles_a_cta():
    seen = set()
    for m, n, k in PRODUCTS:
        for fp32 in (False, True):
            kind, bn, lng, tiles = bt.product_kernel(m, n, k, fp32)
            seen.add((bn, lng, fp32, min(tiles, 3)))
    for bn in (128, 256):
        for lng, fp32 in ((False, False), (False, True), (True, True)):
            assert (bn, lng, fp32, 1) in seen, (bn, lng, fp32)
            assert {(bn, lng, fp32, 2), (bn, lng, fp32, 3)} & seen, (bn, lng, fp32)
    assert (256, True, True, 3) in seen and (256, False, False, 3) in seen


def test_linears_reach_the_segmented_gradient():
    kinds = {bt.product_kernel(o, k, t, True)[:3] for t, o, k in LINEAR if t > 4096}
    assert ("tiles", 256, True) in kinds and ("tiles", 128, True) in kinds


@pytest.mark.parametrize("typ", [ref.E4M3, ref.E5M2, ref.I8])
def test_torch_reference_is_the_numpy_one(typ):
    r = np.random.Generator(np.random.PCG64(typ))
    x = r.standard_normal((40, 400)) * np.exp2(r.integers(-40, 40, (40, 1)))
    x[3] = 0
    x[4, 130:] = 448 * 2.0 ** -130
    x = x.astype(np.float32).astype(np.float64)
    y, e = bt.quantize(torch.from_numpy(x), typ)
    wy, we = ref.quantize(x, typ)
    assert np.array_equal(y.numpy(), wy) and np.array_equal(e.numpy(), we)
