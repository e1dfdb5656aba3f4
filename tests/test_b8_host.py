"""The 8-bit block operators' argument checks, on the host: every refusal
comes before the device is looked up, so no fake pointer reaches a kernel."""
import ctypes
import random

import numpy as np
import pytest

import b8_ref as ref

P = ctypes.c_void_p
GOOD, ODD = 0x10000, 0x10008
OK, INVALID, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE, DEVICE = 0, 1, 2, 3, 4, 5, 7


@pytest.fixture(scope="module")
def sbl():
    from sparsity_sbl_quantize_b200 import build
    build.build()
    from sparsity_sbl_quantize_b200 import sbl as m
    code = ctypes.c_uint32(0)
    if m._lib.sbl_device_error(ctypes.byref(code), 0) != DEVICE:
        pytest.skip("a device is present: fake pointers must not reach kernels")
    return m


def m8(sbl, codes=GOOD, scales=GOOD):
    return ctypes.byref(sbl.sbl_b8(codes, scales))


def d8(sbl, rows, cols, typ=0):
    return ctypes.byref(sbl.b8_desc(rows, cols, typ))


@pytest.mark.parametrize("rows,cols,row_bytes,scales", [(1, 16, 16, 512), (128, 512, 512, 512), (129, 513, 528, 2048), (5, 1, 16, 512),
                                                        (0, 16, 16, 0), (300, 11008, 11008, 4 * 384 * 22)])
def test_sizes(sbl, rows, cols, row_bytes, scales):
    d = sbl.b8_desc(rows, cols)
    assert (sbl.sbl_b8_row_bytes(d), sbl.sbl_b8_scale_bytes(d)) == (row_bytes, scales)


def test_sizes_of_invalid_descriptors(sbl):
    for d in ((-1, 16, 0), (4, 0, 0), (4, -16, 0), (4, 16, 3), (4, 16, -1), ((1 << 30) + 1, 16, 0)):
        assert sbl.sbl_b8_row_bytes(sbl.b8_desc(*d)) == 0 and sbl.sbl_b8_scale_bytes(sbl.b8_desc(*d)) == 0
    assert sbl._lib.sbl_b8_row_bytes(None) == 0
    assert sbl.sbl_b8_linear_workspace_bytes(sbl.b8_desc(40, 64, 0), 4) == 0  # rows not a multiple of 16
    assert sbl.sbl_b8_linear_workspace_bytes(sbl.b8_desc(32, 64, 2), 4) == 0  # int8 has no product
    assert sbl.sbl_b8_linear_workspace_bytes(sbl.b8_desc(32, 64, 0), -1) == 0
    assert sbl.sbl_rmsnorm_backward_workspace_bytes(4, 40) == 0
    assert sbl.sbl_rmsnorm_backward_workspace_bytes(-1, 64) == 0


def test_quantize_refusals(sbl):
    f = sbl._lib.sbl_b8_quantize

    def call(d=(4, 64, 0), x=GOOD, fp32=0, ld=64, blocks=0, out=True, out_t=None):
        o = m8(sbl) if out is True else out
        return f(d8(sbl, *d), x, fp32, ld, blocks, o, out_t, None)

    assert call() == DEVICE and call(out=None, out_t=m8(sbl)) == DEVICE and call(blocks=1) == DEVICE
    assert call(d=(0, 64, 0), x=None) == OK
    assert f(None, GOOD, 0, 64, 0, m8(sbl), None, None) == INVALID
    assert call(d=(4, 64, 3)) == INVALID and call(blocks=2) == INVALID and call(out=None) == INVALID
    assert call(x=None) == INVALID and call(out=m8(sbl, None)) == INVALID and call(out=m8(sbl, GOOD, None)) == INVALID
    assert call(out_t=m8(sbl, None)) == INVALID
    for d in ((-1, 64, 0), (4, 40, 0), (4, 8, 0), (4, 65552, 0), ((1 << 30) + 16, 64, 0)):
        assert call(d=d, ld=1 << 20) == SHAPE
    assert call(ld=56) == SHAPE and call(ld=68) == SHAPE and call(fp32=1, ld=68) == DEVICE and call(fp32=1, ld=66) == SHAPE
    assert call(x=ODD) == ALIGN and call(out=m8(sbl, ODD)) == ALIGN and call(out_t=m8(sbl, GOOD, ODD)) == ALIGN


def test_transpose_and_dequantize_refusals(sbl):
    f, g = sbl._lib.sbl_b8_transpose, sbl._lib.sbl_b8_dequantize
    assert f(d8(sbl, 4, 64), m8(sbl), 1, m8(sbl), None) == DEVICE
    assert f(d8(sbl, 0, 64), None, 1, None, None) == OK
    assert f(d8(sbl, 4, 60), m8(sbl), 1, m8(sbl), None) == SHAPE
    assert f(d8(sbl, 4, 64), m8(sbl), 3, m8(sbl), None) == INVALID
    assert f(d8(sbl, 4, 64), None, 0, m8(sbl), None) == INVALID and f(d8(sbl, 4, 64), m8(sbl), 0, None, None) == INVALID
    assert f(d8(sbl, 4, 64), m8(sbl, ODD), 0, m8(sbl), None) == ALIGN
    assert g(d8(sbl, 4, 64), m8(sbl), GOOD, 64, None) == DEVICE
    assert g(d8(sbl, 4, 64), m8(sbl), GOOD, 60, None) == SHAPE and g(d8(sbl, 4, 64), m8(sbl), GOOD, 68, None) == SHAPE
    assert g(d8(sbl, 4, 64), m8(sbl), None, 64, None) == INVALID and g(d8(sbl, 4, 64), m8(sbl), ODD, 64, None) == ALIGN


def test_gemm_refusals(sbl):
    f = sbl._lib.sbl_b8_gemm

    def call(a=(4, 100, 0), b=(32, 100, 0), am=True, bm=True, d=GOOD, ld=32, fp32=0, acc=0):
        return f(d8(sbl, *a), m8(sbl) if am is True else am, d8(sbl, *b), m8(sbl) if bm is True else bm, d, ld, fp32, acc, None)

    assert call() == DEVICE and call(fp32=1, acc=1) == DEVICE and call(a=(4, 100, 1)) == DEVICE
    assert call(a=(0, 100, 0), am=None, d=None) == OK
    assert call(a=(4, 100, 2)) == UNSUPPORTED and call(b=(32, 100, 2)) == UNSUPPORTED
    assert call(a=(4, 99, 0)) == SHAPE and call(b=(40, 100, 0), ld=40) == SHAPE and call(b=(0, 100, 0)) == SHAPE
    assert call(ld=24) == SHAPE and call(ld=36) == SHAPE and call(ld=36, fp32=1) == DEVICE
    assert call(acc=1) == INVALID  # only an fp32 D accumulates
    assert call(am=None) == INVALID and call(bm=m8(sbl, GOOD, None)) == INVALID and call(d=None) == INVALID
    assert call(d=ODD) == ALIGN and call(am=m8(sbl, ODD)) == ALIGN
    # more tiles than a launch's 32-bit tile numbers
    assert call(a=(1 << 30, 100, 0), b=(1 << 30, 100, 0), ld=1 << 30) in (SHAPE, DEVICE)


def test_linear_refusals(sbl):
    f, b = sbl._lib.sbl_b8_linear_forward, sbl._lib.sbl_b8_linear_backward

    def fwd(w=(32, 64, 0), wm=True, x=GOOD, ldx=64, t=4, xt=0, xq=True, y=GOOD, ldy=32):
        return f(d8(sbl, *w), m8(sbl) if wm is True else wm, x, ldx, t, xt, m8(sbl) if xq is True else xq, y, ldy, 0, None)

    assert fwd() == DEVICE and fwd(t=0, x=None, xq=None) == OK
    assert fwd(w=(40, 64, 0)) == SHAPE and fwd(w=(32, 72, 0), ldx=72) == SHAPE and fwd(t=-1) == SHAPE and fwd(w=(65552, 64, 0)) == SHAPE
    assert fwd(w=(32, 64, 2)) == UNSUPPORTED and fwd(xt=2) == UNSUPPORTED and fwd(xt=7) == INVALID
    assert fwd(wm=None) == INVALID and fwd(xq=None) == INVALID and fwd(x=None) == INVALID and fwd(y=None) == INVALID
    assert fwd(ldx=60) == SHAPE and fwd(ldy=30) == SHAPE and fwd(x=ODD) == ALIGN and fwd(xq=m8(sbl, GOOD, ODD)) == ALIGN

    need = sbl.sbl_b8_linear_workspace_bytes(sbl.b8_desc(32, 64, 0), 4)

    def bwd(w=(32, 64, 0), wt=True, xq=True, dy=GOOD, t=4, gt=0, dx=GOOD, dw=GOOD, ws=GOOD, n=need):
        return b(d8(sbl, *w), m8(sbl) if wt is True else wt, m8(sbl) if xq is True else xq, 0, dy, 32, t, gt, dx, 0, dw, 0, ws, n, None)

    assert bwd() == DEVICE and bwd(dx=None, wt=None) == DEVICE and bwd(dw=None, xq=None) == DEVICE and bwd(gt=1) == DEVICE
    assert bwd(dx=None, dw=None) == INVALID and bwd(wt=None) == INVALID and bwd(xq=None) == INVALID and bwd(dy=None) == INVALID
    assert bwd(ws=None) == WORKSPACE and bwd(n=need - 1) == WORKSPACE and bwd(ws=GOOD + 16) == ALIGN
    assert bwd(dw=ODD) == ALIGN and bwd(dx=ODD) == ALIGN and bwd(dy=ODD) == ALIGN and bwd(gt=2) == UNSUPPORTED and bwd(t=-4) == SHAPE


def test_glu_refusals(sbl):
    f, b = sbl._lib.sbl_glu_forward, sbl._lib.sbl_glu_backward

    def fwd(d=(4, 64, 0), act=0, g=GOOD, ldg=128, u=GOOD, ldu=128, h=GOOD, ldh=64, g8=True, u8=True):
        return f(d8(sbl, *d), act, g, ldg, u, ldu, h, ldh, m8(sbl) if g8 is True else g8, m8(sbl) if u8 is True else u8, None)

    assert fwd() == DEVICE and fwd(u=None, ldu=0, u8=None) == DEVICE and fwd(h=None, ldh=0) == DEVICE and fwd(g8=None, u8=None) == DEVICE
    assert fwd(d=(0, 64, 0), g=None, u=None, u8=None) == OK
    assert fwd(act=2) == INVALID and fwd(h=None, g8=None, u8=None) == INVALID and fwd(u=None) == INVALID and fwd(g=None) == INVALID
    assert fwd(d=(4, 60, 0)) == SHAPE and fwd(ldg=60) == SHAPE and fwd(ldu=132) == SHAPE and fwd(ldh=68) == SHAPE
    assert fwd(g=ODD) == ALIGN and fwd(u=ODD) == ALIGN and fwd(h=ODD) == ALIGN and fwd(g8=m8(sbl, ODD)) == ALIGN

    def bwd(d=(4, 64, 0), act=1, g8=True, u8=True, dh=GOOD, dg=GOOD, du=GOOD, ld=64):
        return b(d8(sbl, *d), act, m8(sbl) if g8 is True else g8, m8(sbl) if u8 is True else u8, dh, ld, dg, 64, du, 64, None)

    assert bwd() == DEVICE and bwd(u8=None, du=None) == DEVICE and bwd(d=(0, 64, 0), dh=None) == OK
    assert bwd(u8=None) == INVALID and bwd(du=None) == INVALID and bwd(g8=None) == INVALID and bwd(dh=None) == INVALID and bwd(dg=None) == INVALID
    assert bwd(act=-1) == INVALID and bwd(ld=56) == SHAPE and bwd(dg=ODD) == ALIGN and bwd(u8=m8(sbl, GOOD, ODD)) == ALIGN


def test_norm_refusals(sbl):
    f, b = sbl._lib.sbl_quantize_act_rmsnorm_checkpoint, sbl._lib.sbl_rmsnorm_backward

    def fwd(d=(4, 64, 0), x=GOOD, g=GOOD, eps=1e-5, q=GOOD, s=GOOD, x8=True):
        return f(d8(sbl, *d), x, g, eps, q, s, m8(sbl) if x8 is True else x8, None)

    assert fwd() == DEVICE and fwd(g=None) == DEVICE and fwd(d=(0, 64, 0), x=None) == OK
    assert fwd(x8=None) == INVALID and fwd(x=None) == INVALID and fwd(eps=-1.0) == INVALID and fwd(eps=float("nan")) == INVALID
    assert fwd(eps=float("inf")) == INVALID and fwd(d=(4, 50, 0)) == SHAPE and fwd(g=ODD) == ALIGN and fwd(x8=m8(sbl, ODD)) == ALIGN

    need = sbl.sbl_rmsnorm_backward_workspace_bytes(4, 64)

    def bwd(d=(4, 64, 0), x8=True, g=GOOD, eps=1e-5, du=GOOD, dr=None, dx=GOOD, dg=GOOD, ws=GOOD, n=need):
        return b(d8(sbl, *d), m8(sbl) if x8 is True else x8, g, eps, du, dr, dx, dg, ws, n, None)

    assert bwd() == DEVICE and bwd(dg=None, ws=None, n=0) == DEVICE and bwd(g=None, dg=None) == DEVICE
    assert bwd(g=None) == INVALID and bwd(x8=None) == INVALID and bwd(du=None) == INVALID and bwd(dx=None) == INVALID
    assert bwd(ws=None) == WORKSPACE and bwd(n=need - 1) == WORKSPACE and bwd(ws=GOOD + 128) == ALIGN
    assert bwd(dr=ODD) == ALIGN and bwd(dg=ODD) == ALIGN and bwd(eps=-1e-9) == INVALID and bwd(d=(4, 24, 0)) == SHAPE


def test_random_arguments_return_documented_statuses(sbl):
    r = random.Random(5)
    ints = [-1, 0, 1, 15, 16, 48, 64, 128, 1040, 65536, 65552, 1 << 30, (1 << 31) - 1, -(1 << 31)]

    def p():
        return r.choice([None, GOOD, ODD, 0x20000])

    def d():
        return r.choice([None, d8(sbl, r.choice(ints), r.choice(ints), r.choice([-1, 0, 1, 2, 3]))])

    def m():
        return r.choice([None, m8(sbl, p(), p())])

    def i():
        return r.choice(ints)

    L, seen = sbl._lib, set()
    for _ in range(6000):
        seen.add(r.choice([
            lambda: L.sbl_b8_quantize(d(), p(), i() & 1, i(), i() & 3, m(), m(), None),
            lambda: L.sbl_b8_transpose(d(), m(), i() & 3, m(), None),
            lambda: L.sbl_b8_dequantize(d(), m(), p(), i(), None),
            lambda: L.sbl_b8_gemm(d(), m(), d(), m(), p(), i(), i() & 1, i() & 1, None),
            lambda: L.sbl_b8_linear_forward(d(), m(), p(), i(), i(), i() & 3, m(), p(), i(), i() & 1, None),
            lambda: L.sbl_b8_linear_backward(d(), m(), m(), i() & 3, p(), i(), i(), i() & 3, p(), i() & 1, p(), i() & 1, p(), 1 << 40, None),
            lambda: L.sbl_glu_forward(d(), i() & 3, p(), i(), p(), i(), p(), i(), m(), m(), None),
            lambda: L.sbl_glu_backward(d(), i() & 3, m(), m(), p(), i(), p(), i(), p(), i(), None),
            lambda: L.sbl_quantize_act_rmsnorm_checkpoint(d(), p(), p(), 1e-5, p(), p(), m(), None),
            lambda: L.sbl_rmsnorm_backward(d(), m(), p(), 1e-5, p(), p(), p(), p(), p(), 1 << 40, None)])())
    assert seen <= set(range(8))


def test_binding_refuses_what_it_cannot_describe(sbl):
    import torch
    with pytest.raises(ValueError):
        sbl._ld(torch.zeros(4, 8).t())
    with pytest.raises(ValueError):
        sbl._ld(torch.zeros(8))
    assert sbl._ld(torch.zeros(4, 32)[:, :16]) == 32 and sbl._ld(torch.zeros(1, 16)) == 16 and sbl._ld(None) == 0


# ------------------------------------------------------- the reference itself

@pytest.mark.parametrize("typ", [ref.E4M3, ref.E5M2, ref.I8])
def test_reference_rounds_to_the_nearest_code(typ):
    """round_to against a search over all codes, ties to the even one."""
    vals = ref.code_values(typ)
    codes = np.arange(256)[np.isfinite(vals) & (np.abs(vals) <= ref.MAX[typ])]
    grid = vals[codes]
    r = np.random.Generator(np.random.PCG64(1))
    mids = (np.sort(np.unique(grid))[1:] + np.sort(np.unique(grid))[:-1]) / 2
    x = np.concatenate([mids, grid, r.uniform(-1, 1, 400) * ref.MAX[typ], r.standard_normal(400) * 2.0 ** -8])
    got = ref.round_to(x, typ)
    d = np.abs(x[:, None] - grid[None, :])
    best = d.min(1)
    assert np.array_equal(np.abs(x - got), best)
    for k in np.nonzero(np.isin(x, mids))[0]:
        near = codes[d[k] == best[k]]
        near = near[vals[near] == got[k]]
        assert (near & 1 == 0).any() or got[k] == 0


def test_reference_against_torch_casts():
    import torch
    x = np.random.Generator(np.random.PCG64(2)).standard_normal(4000) * np.exp2(np.random.Generator(np.random.PCG64(3)).integers(-12, 8, 4000))
    x = np.clip(x, -448, 448).astype(np.float32)
    for typ, dt in ((ref.E4M3, torch.float8_e4m3fn), (ref.E5M2, torch.float8_e5m2)):
        assert np.array_equal(ref.round_to(x.astype(np.float64), typ), torch.from_numpy(x).to(dt).double().numpy())


def test_scale_order_covers_every_byte_once():
    e = np.arange(300 * 9).reshape(300, 9) % 100
    s = ref.scale_bytes(e)
    assert s.size == 4 * 384 * 3 and np.array_equal(np.sort(s[s != 127]), np.sort((e + 127).ravel()[(e + 127).ravel() != 127].astype(np.uint8)))
