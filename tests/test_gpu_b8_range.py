"""RMSNorm's backward over the range of its inputs: rows whose squares, or whose dU x, leave fp32's range while the
gradient does not, tiny and absent eps, rows of zeros, blocks far apart.

Bounds.  s1 = sum x^2 has only positive terms, added in a chain of 16 and a tree of at most 12 levels: off by
32 2^-24 of itself with its scalings, so r (half of that, rsqrtf's 2 units, two roundings) by less than 24 2^-24.  n = x r
adds one rounding.  s2 = sum v x is off by 32 2^-24 of the sum of magnitudes and m = r s2 / K by less than
60 2^-24 of mean |v n|.  dX = r (v - n m) is then off by less than 90 2^-24 of r |n| mean |v n|, 30 2^-24 of |r v|
and half a bf16 step of itself; a sum of t terms du n by (t + 32) 2^-24 of its magnitudes."""
import numpy as np
import pytest
import torch

import b8_ref as ref
from gpu_case import sbl_mod

pytestmark = pytest.mark.gpu

TYPES = [ref.E4M3, ref.E5M2, ref.I8]
U = 2.0 ** -24


def rng(*key):
    return np.random.Generator(np.random.PCG64([k & 0xFFFFFFFF for k in key]))


def bf16(a):
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)
    return t.cuda(), t.double().numpy()


def backward(typ, x, du, gain, eps):
    """(dX, dg) of the library and the checkpointed x, all float64."""
    sbl = sbl_mod()
    t, k = x.shape
    d = sbl.b8_desc(t, k, typ)
    x8 = sbl.alloc_b8(d)
    sbl.sbl_b8_quantize(d, x, x8)
    dx, dg = torch.empty_like(x), torch.empty(k, dtype=torch.float32, device="cuda")
    ws = sbl.alloc_workspace(sbl.sbl_rmsnorm_backward_workspace_bytes(t, k))
    sbl.sbl_rmsnorm_backward(d, x8, gain, eps, du, None, dx, dg, ws)
    return dx.double().cpu().numpy(), dg.double().cpu().numpy()


def check(typ, xv, x, du, duv, g, gv, eps):
    dx, dg = backward(typ, x, du, g.view(-1), eps)
    xq = ref.value(xv, typ)
    v = duv * gv
    rr = 1 / np.sqrt(np.maximum((xq * xq).mean(1, keepdims=True) + eps, 2.0 ** -252))
    n = xq * rr
    want = rr * (v - n * (v * n).mean(1, keepdims=True))
    slack = U * (90 * rr * np.abs(n) * (np.abs(v) * np.abs(n)).mean(1, keepdims=True) + 30 * np.abs(rr * v))
    bad = ~(np.abs(dx - want) <= (2.0 ** -8 + 30 * U) * np.abs(want) + slack)
    assert not bad.any(), (int(bad.sum()), dx[bad][:4], want[bad][:4])
    bad = ~(np.abs(dg - (duv * n).sum(0)) <= U * (x.shape[0] + 32) * np.abs(duv * n).sum(0))
    assert not bad.any(), int(bad.sum())


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("t,k", [(5, 144), (3, 2064), (2, 8208), (2, 20000)])
@pytest.mark.parametrize("px,pdu", [(-118, -10), (-80, 0), (-66, 20), (0, -100), (56, -40), (56, 0), (80, 30), (110, 0), (118, 40)])
def test_small_and_large_rows_and_gradients(typ, t, k, px, pdu):
    r = rng(typ, t, k, px, pdu)
    (x, xv), (du, duv) = bf16(r.standard_normal((t, k)) * 2.0 ** px), bf16(r.standard_normal((t, k)) * 2.0 ** pdu)
    g, gv = bf16(1 + 0.2 * r.standard_normal((1, k)))
    check(typ, xv, x, du, duv, g, gv, 0.0)


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("eps", [0.0, 1e-300, 2.0 ** -200, 1e-45, 1e-30, 1e-5, 1.0, 3e38])
def test_rows_of_zeros_between_others(typ, eps):
    """A row of zeros: n = 0, dX = dU g / sqrt(eps), at most 2^126 of it; the gains' gradient has the other rows' terms."""
    r = rng(typ, 41)
    t, k = 9, 272
    xs, dus = r.standard_normal((t, k)), r.standard_normal((t, k)) * 2.0 ** -10
    xs[[0, 4, 8]] = 0
    dus[8] = 0
    (x, xv), (du, duv), (g, gv) = bf16(xs), bf16(dus), bf16(1 + 0.2 * r.standard_normal((1, k)))
    check(typ, xv, x, du, duv, g, gv, eps)


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("k", [400, 1040, 4112, 16400])
def test_blocks_far_apart(typ, k):
    """Blocks of one row up to 2^60 apart, some of them zero; eps near the smaller ones."""
    r = rng(typ, k, 42)
    t = 4
    scale = np.exp2(r.integers(-60, 1, (t, -(-k // 128)))) * (r.random((t, -(-k // 128))) < 0.8)
    (x, xv) = bf16(r.standard_normal((t, k)) * np.repeat(scale, 128, axis=1)[:, :k])
    (du, duv), (g, gv) = bf16(r.standard_normal((t, k))), bf16(1 + 0.2 * r.standard_normal((1, k)))
    for eps in (0.0, 2.0 ** -70, 2.0 ** -20):
        check(typ, xv, x, du, duv, g, gv, eps)


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("k", [144, 2064, 20000])
def test_marked_blocks_make_their_row_nan(typ, k):
    r = rng(typ, k, 43)
    xs = r.standard_normal((4, k))
    xs[2, 130] = np.inf
    (x, _), (du, _), (g, _) = bf16(xs), bf16(r.standard_normal((4, k))), bf16(np.ones((1, k)))
    dx, dg = backward(typ, x, du, g.view(-1), 1e-5)
    assert np.isnan(dx[2]).all() and np.isfinite(np.delete(dx, 2, 0)).all() and np.isnan(dg).all()
