"""A linear with more outputs than one call takes, as slabs of its rows: Y and dY are columns of the whole matrices, dW
rows of the whole gradient, and the slabs' dX add up."""
import pytest
import torch

import b8_ref as ref
import b8_torch as bt
from gpu_case import sbl_mod

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [3, 40, 300])
def test_linear_in_slabs_of_rows(t):
    sbl = sbl_mod()
    o, k, slab = 131_200, 144, 65_536
    g = torch.Generator(device="cuda").manual_seed(t)
    w = torch.randn(o, k, generator=g, device="cuda") * 0.02
    x = torch.randn(t, k, generator=g, device="cuda").to(torch.bfloat16)
    dy = (torch.randn(t, o, generator=g, device="cuda") * 1e-3).to(torch.bfloat16)
    y, dw = torch.empty(t, o, dtype=torch.bfloat16, device="cuda"), torch.full((o, k), 7.0, device="cuda")
    dx, part = torch.zeros(t, k, device="cuda"), torch.empty(t, k, device="cuda")
    xd = sbl.b8_desc(t, k)
    xq, weights = sbl.alloc_b8(xd), []
    ws = sbl.alloc_workspace(sbl.sbl_b8_linear_workspace_bytes(sbl.b8_desc(slab, k), t))
    for at in range(0, o, slab):
        n = min(slab, o - at)
        wd = sbl.b8_desc(n, k)
        wq, wt = sbl.alloc_b8(wd), sbl.alloc_b8(sbl.b8_desc(k, n))
        sbl.sbl_b8_quantize(wd, w[at:at + n], wq, wt, sbl.SBL_B8_TILES)
        sbl.sbl_b8_linear_forward(wd, wq, x, t, xq, y[:, at:at + n])
        sbl.sbl_b8_linear_backward(wd, wt, xq, dy[:, at:at + n], t, part, dw[at:at + n], ws)
        dx += part
        weights.append(bt.stored(wq, wd))
    wv = torch.cat(weights)
    x8 = bt.decode(*bt.quantize(x.double(), ref.E4M3))

    def check(got, a, b, half, parts):
        # truncating accumulation as in test_gpu_b8.py; a rounded addition a slab
        want, mags = a @ b.t(), a.abs() @ b.abs().t()
        bound = (1 + half) * ((-(-a.shape[1] // 32) + 5) * 2.0 ** -23 + parts * 2.0 ** -24) * mags
        assert bool(((got.double() - want).abs() <= half * want.abs() + bound).all())

    check(y, x8, wv, 2.0 ** -8, 0)
    # the blocks of the undivided dY, along its rows and along tokens
    check(dx, bt.decode(*bt.quantize(dy.double(), ref.E4M3)), wv.t().contiguous(), 2.0 ** -24, 3)
    check(dw, bt.decode(*bt.quantize(dy.double().t().contiguous(), ref.E4M3)),
          bt.decode(*bt.quantize(x8.t().contiguous(), ref.E4M3)), 2.0 ** -24, 0)
    assert sbl.sbl_device_error() == 0
