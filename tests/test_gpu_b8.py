"""The 8-bit block operators on the GPU against their definitions in 64 bits.

Codes, scales and everything built only from them are compared bit for bit.
Tolerances elsewhere come from the formats: a result rounded once to bf16 is
off by half a step (2^-8 of the value) plus what the fp32 arithmetic before it
adds, stated at each test."""
import numpy as np
import pytest
import torch

import b8_ref as ref
from gpu_case import sbl_mod

pytestmark = pytest.mark.gpu

TYPES = [ref.E4M3, ref.E5M2, ref.I8]
F8 = [ref.E4M3, ref.E5M2]


def rng(*key):
    return np.random.Generator(np.random.PCG64(list(key)))


def bf16(a):
    """float array -> (bf16 CUDA tensor, its exact float64 values)."""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)
    return t.cuda(), t.double().numpy()


def strided(t, pad=8, fill=777.0):
    """The same matrix inside a wider buffer (row stride + pad)."""
    buf = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device=t.device)
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]]


def host_values(m, cols, typ):
    """Values of a stored matrix's codes (unscaled) and its scale bytes."""
    return ref.code_values(typ)[m.codes.cpu().numpy()][:, :cols], m.scales.cpu().numpy()


def check_stored(m, cols, typ, want_y, want_e):
    y, s = host_values(m, cols, typ)
    assert np.array_equal(s, ref.scale_bytes(want_e))
    assert np.array_equal(y, want_y)


def new(sbl, rows, cols, typ):
    d = sbl.b8_desc(rows, cols, typ)
    m = sbl.alloc_b8(d)
    m.codes.fill_(0xA5)
    m.scales.fill_(0xA5)
    return d, m


def wide(r, rows, cols):
    """Values over many binades, with zero blocks, exact maxima and ties."""
    x = r.standard_normal((rows, cols)) * np.exp2(r.integers(-20, 20, (rows, 1)))
    x[r.random((rows, cols)) < 0.1] = 0
    x[:, :16] = np.round(x[:, :16] * 8) / 8
    if rows > 2:
        x[1] = 0
        x[2, :] = 448.0
    if rows > 5:
        x[3, :] = 57344.0 * 2.0 ** -30
        x[4, :] = 127.0 * 2.0 ** 40
        x[5, :] = 2.0 ** -130
    return x


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 128), (7, 144), (130, 640), (128, 512), (257, 1040), (33, 2064)])
@pytest.mark.parametrize("src", ["bf16", "fp32"])
def test_quantize_rows(rows, cols, typ, src):
    sbl = sbl_mod()
    x = wide(rng(rows, cols, typ), rows, cols).astype(np.float32)
    t, v = bf16(x) if src == "bf16" else (torch.from_numpy(x).cuda(), x.astype(np.float64))
    d, m = new(sbl, rows, cols, typ)
    sbl.sbl_b8_quantize(d, strided(t), m)
    check_stored(m, cols, typ, *ref.quantize(v, typ))


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 16), (16, 128), (7, 144), (130, 640), (257, 1040)])
@pytest.mark.parametrize("src", ["bf16", "fp32"])
@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("which", ["both", "rows", "transposed"])
def test_quantize_both_orders(rows, cols, typ, src, tiles, which):
    sbl = sbl_mod()
    x = wide(rng(rows, cols, typ, 1), rows, cols).astype(np.float32)
    t, v = bf16(x) if src == "bf16" else (torch.from_numpy(x).cuda(), x.astype(np.float64))
    d, m = new(sbl, rows, cols, typ)
    _, mt = new(sbl, cols, rows, typ)
    sbl.sbl_b8_quantize(d, strided(t), m if which != "transposed" else None, mt if which != "rows" else None,
                        sbl.SBL_B8_TILES if tiles else sbl.SBL_B8_ROWS)
    y, e = ref.quantize(v, typ, tiles)
    if which != "transposed":
        check_stored(m, cols, typ, y, e)
    if which != "rows":
        if tiles:
            b = -(-rows // 128)
            et = np.stack([np.repeat(e[128 * i, :], 128)[:cols] for i in range(b)], 1)
            check_stored(mt, rows, typ, y.T, et)
        else:
            check_stored(mt, rows, typ, *ref.quantize(np.ascontiguousarray(v.T), typ))
        assert not mt.codes[:, rows:].any()  # padding codes are zero


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("typ_t", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 16), (200, 272), (129, 128)])
def test_transpose(rows, cols, typ, typ_t):
    sbl = sbl_mod()
    t, v = bf16(rng(rows, cols, typ, 2).standard_normal((rows, cols)) * np.exp2(rng(3).integers(-4, 4, (rows, 1))))
    d, m = new(sbl, rows, cols, typ)
    _, mt = new(sbl, cols, rows, typ_t)
    sbl.sbl_b8_quantize(d, t, m)
    sbl.sbl_b8_transpose(d, m, mt, typ_t)
    check_stored(mt, rows, typ_t, *ref.quantize(np.ascontiguousarray(ref.value(v, typ).T), typ_t))


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 16), (5, 144), (131, 1040)])
def test_dequantize(rows, cols, typ):
    sbl = sbl_mod()
    t, v = bf16(wide(rng(rows, cols, typ, 4), rows, cols))
    d, m = new(sbl, rows, cols, typ)
    sbl.sbl_b8_quantize(d, t, m)
    out = torch.full((rows, cols + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    sbl.sbl_b8_dequantize(d, m, out[:, :cols])
    want = torch.from_numpy(ref.value(v, typ).astype(np.float32)).to(torch.bfloat16)
    assert torch.equal(out[:, :cols].cpu(), want)
    assert bool((out[:, cols:] == 5.0).all())


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_non_finite_blocks_become_nan(typ, bad):
    sbl = sbl_mod()
    x = rng(typ, 5).standard_normal((6, 400))
    x[2, 130] = bad
    t, v = bf16(x)
    d, m = new(sbl, 6, 400, typ)
    sbl.sbl_b8_quantize(d, t, m)
    check_stored(m, 400, typ, *ref.quantize(v, typ))
    out = torch.empty((6, 400), dtype=torch.bfloat16, device="cuda")
    sbl.sbl_b8_dequantize(d, m, out)
    nan = torch.isnan(out).cpu().numpy()
    assert nan[2, 128:256].all() and nan.sum() == 128
    _, mt = new(sbl, 400, 6, typ)
    sbl.sbl_b8_transpose(d, m, mt)
    s = mt.scales.cpu().numpy().reshape(-1, 4)[:, 0]
    assert (s == 255).sum() == 128  # the rows of the transpose that hold a NaN


# ------------------------------------------------------------------ product

def operands(sbl, r, rows, cols, typ):
    """A stored matrix of any width (as the transpose of a [cols, rows16] one) and its values."""
    rows16 = -(-rows // 16) * 16
    t, v = bf16(r.standard_normal((cols, rows16)) * np.exp2(r.integers(-3, 4, (cols, 1))))
    d, m = new(sbl, rows16, cols, typ)
    sbl.sbl_b8_quantize(sbl.b8_desc(cols, rows16, typ), t, None, m)
    return d, m, ref.value(np.ascontiguousarray(v.T), typ)


def product_bound(a, b, k):
    """|error| of the fp32 accumulation: the exact products of 32 k's are added to the accumulator in
    ceil(k / 32) steps, each off by at most one unit of the larger magnitude's last place (2^-23; the
    tensor core may truncate), and by five levels of additions inside a step."""
    return (-(-k // 32) + 5) * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T)


def check_product(got, a, b, half):
    want = a @ b.T
    tol = half * np.abs(want) + (1 + half) * product_bound(a, b, a.shape[1])
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) - tol).max())


@pytest.mark.parametrize("m,n,k", [(16, 16, 128), (16, 128, 512), (128, 128, 2048), (144, 272, 640), (16, 16, 1), (32, 48, 100),
                                   (304, 144, 1040), (16, 4096, 130), (1040, 16, 520), (2064, 1040, 400)])
@pytest.mark.parametrize("ta,tb", [(0, 0), (1, 0), (0, 1), (1, 1)])
@pytest.mark.parametrize("fp32", [False, True])
def test_gemm(m, n, k, ta, tb, fp32):
    sbl = sbl_mod()
    ad, a, av = operands(sbl, rng(m, n, k, ta, 6), m, k, ta)
    bd, b, bv = operands(sbl, rng(m, n, k, tb, 7), n, k, tb)
    out = torch.full((m, n + 8), 3.0, dtype=torch.float32 if fp32 else torch.bfloat16, device="cuda")
    sbl.sbl_b8_gemm(ad, a, bd, b, out[:, :n])
    check_product(out[:, :n].double().cpu().numpy(), av, bv, ref.HALF["fp32" if fp32 else "bf16"])
    assert bool((out[:, n:] == 3.0).all())
    if fp32:
        sbl.sbl_b8_gemm(ad, a, bd, b, out[:, :n], accumulate=True)
        once = torch.empty((m, n), dtype=torch.float32, device="cuda")
        sbl.sbl_b8_gemm(ad, a, bd, b, once)
        assert torch.equal(out[:, :n], once + once)
    assert sbl.sbl_device_error() == 0


@pytest.mark.parametrize("m", [1, 2, 5, 13, 16, 17, 31, 33, 64, 100, 127, 129, 250, 300])
@pytest.mark.parametrize("n,k", [(16, 64), (144, 2064), (1024, 528)])
def test_gemm_any_rows(m, n, k):
    """A's rows of any number: what a linear sees for any count of tokens."""
    sbl = sbl_mod()
    t, v = bf16(rng(m, n, k, 8).standard_normal((m, k)))
    ad, a = new(sbl, m, k, ref.E4M3)
    sbl.sbl_b8_quantize(ad, t, a)
    bd, b, bv = operands(sbl, rng(m, n, k, 9), n, k, ref.E4M3)
    out = torch.full((m + 2, n), 3.0, dtype=torch.bfloat16, device="cuda")
    sbl.sbl_b8_gemm(ad, a, bd, b, out[:m])
    check_product(out[:m].double().cpu().numpy(), ref.value(v, ref.E4M3), bv, ref.HALF["bf16"])
    assert bool((out[m:] == 3.0).all())


def test_gemm_scales_are_applied_per_block():
    """Operands whose rows and blocks differ by powers of two as far as the exponents go."""
    sbl = sbl_mod()
    r = rng(10)
    m, n, k = 160, 144, 1536
    x = r.choice([-1.0, 1.0], (m, k)) * np.exp2(r.integers(-30, 30, (m, k // 128))).repeat(128, 1)
    w = r.choice([-1.0, 1.0], (n, k)) * np.exp2(r.integers(-30, 30, (n, k // 128))).repeat(128, 1)
    (tx, vx), (tw, vw) = bf16(x), bf16(w)
    (ad, a), (bd, b) = new(sbl, m, k, ref.E4M3), new(sbl, n, k, ref.E5M2)
    sbl.sbl_b8_quantize(ad, tx, a)
    sbl.sbl_b8_quantize(bd, tw, b)
    out = torch.empty((m, n), dtype=torch.float32, device="cuda")
    sbl.sbl_b8_gemm(ad, a, bd, b, out)
    check_product(out.double().cpu().numpy(), vx, vw, ref.HALF["fp32"])


def test_gemm_marked_blocks_give_nan_rows():
    sbl = sbl_mod()
    x = rng(11).standard_normal((40, 304))
    x[7, 200] = np.inf
    t, _ = bf16(x)
    ad, a = new(sbl, 40, 288, ref.E4M3)
    sbl.sbl_b8_quantize(ad, t[:, :288], a)
    bd, b, _ = operands(sbl, rng(12), 32, 288, ref.E4M3)
    out = torch.empty((40, 32), dtype=torch.float32, device="cuda")
    sbl.sbl_b8_gemm(ad, a, bd, b, out)
    nan = torch.isnan(out).cpu().numpy()
    assert nan[7].all() and nan.sum() == 32


# ------------------------------------------------------------------- linear

@pytest.mark.parametrize("t", [1, 3, 16, 65, 300])
@pytest.mark.parametrize("o,k", [(16, 16), (272, 400), (128, 1024)])
@pytest.mark.parametrize("wt,xt,gt", [(0, 0, 0), (0, 0, 1), (1, 0, 1)])
def test_linear_training_step(t, o, k, wt, xt, gt):
    sbl = sbl_mod()
    r = rng(t, o, k, wt, gt, 13)
    w = (r.standard_normal((o, k)) * 0.02).astype(np.float32)
    (x, xv), (dy, dyv) = bf16(r.standard_normal((t, k))), bf16(r.standard_normal((t, o)) * 1e-3)
    wd, wq = new(sbl, o, k, wt)
    _, wqt = new(sbl, k, o, wt)
    sbl.sbl_b8_quantize(wd, torch.from_numpy(w).cuda(), wq, wqt, sbl.SBL_B8_TILES)
    _, xq = new(sbl, t, k, xt)
    y = torch.empty((t, o), dtype=torch.bfloat16, device="cuda")
    sbl.sbl_b8_linear_forward(wd, wq, strided(x), t, xq, y, x_type=xt)
    wv, x8 = ref.value(w.astype(np.float64), wt, True), ref.value(xv, xt)
    check_stored(xq, k, xt, *ref.quantize(xv, xt))
    check_product(y.double().cpu().numpy(), x8, wv, ref.HALF["bf16"])
    dx = torch.empty((t, k), dtype=torch.bfloat16, device="cuda")
    dw = torch.full((o, k), 2.0, dtype=torch.float32, device="cuda")
    ws = sbl.alloc_workspace(sbl.sbl_b8_linear_workspace_bytes(wd, t))
    ws.fill_(0xFF)
    sbl.sbl_b8_linear_backward(wd, wqt, xq, strided(dy), t, dx, dw, ws, x_type=xt, g_type=gt)
    check_product(dx.double().cpu().numpy(), ref.value(dyv, gt), np.ascontiguousarray(wv.T), ref.HALF["bf16"])
    gt_v, xt_v = ref.value(np.ascontiguousarray(dyv.T), gt), ref.value(np.ascontiguousarray(x8.T), xt)
    check_product(dw.double().cpu().numpy(), gt_v, xt_v, ref.HALF["fp32"])
    # accumulation, and each gradient alone, give the same values
    one, dx32 = dw.clone(), torch.empty((t, k), dtype=torch.float32, device="cuda")
    sbl.sbl_b8_linear_backward(wd, None, xq, dy, t, None, dw, ws, x_type=xt, g_type=gt, accumulate=True)
    assert torch.equal(dw, one + one)
    sbl.sbl_b8_linear_backward(wd, wqt, None, dy, t, dx32, None, ws, x_type=xt, g_type=gt)
    assert torch.equal(dx32.to(torch.bfloat16), dx)
    assert sbl.sbl_device_error() == 0


def test_no_tokens():
    sbl = sbl_mod()
    wd, wq = new(sbl, 32, 64, 0)
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    dw = torch.full((32, 64), 2.0, dtype=torch.float32, device="cuda")
    _, xq = new(sbl, 0, 64, 0)
    sbl.sbl_b8_linear_forward(wd, wq, e, 0, xq, torch.empty((0, 32), dtype=torch.bfloat16, device="cuda"))
    sbl.sbl_b8_linear_backward(wd, None, xq, e, 0, None, dw, None, accumulate=True)
    assert bool((dw == 2.0).all())
    sbl.sbl_b8_linear_backward(wd, None, xq, e, 0, None, dw, None)
    assert not dw.any()
    g = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    dg = torch.full((64,), 2.0, device="cuda")
    sbl.sbl_rmsnorm_backward(sbl.b8_desc(0, 64, 0), xq, g, 1e-5, e, None, e, dg, None)
    assert not dg.any()


# --------------------------------------------------------------- activation

@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("t,f", [(1, 16), (3, 144), (130, 528), (5, 2064)])
def test_glu(act, typ, gated, t, f):
    """fp32 arithmetic before the one rounding: __expf and __fdividef are off by at most 2 + |x| 2^-23
    units and 2 units; with |g| < 90 the factors together stay below 2^-15 of |act| + |g| terms."""
    sbl = sbl_mod()
    r = rng(act, typ, t, f, 14)
    gx = r.standard_normal((t, f)) * 4
    gx[:, ::7] *= 8
    (g, gv), (u, uv) = bf16(gx), bf16(r.standard_normal((t, f)))
    both = torch.full((t, 2 * f), 9.0, dtype=torch.bfloat16, device="cuda")  # gate and up side by side
    both[:, :f], both[:, f:] = g, u
    d, g8 = new(sbl, t, f, typ)
    _, u8 = new(sbl, t, f, typ)
    h = torch.full((t, f + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    sbl.sbl_glu_forward(d, act, both[:, :f], both[:, f:] if gated else None, h[:, :f], g8, u8 if gated else None)
    a, _ = ref.act(gv, act)
    want = a * uv if gated else a
    err = np.abs(h[:, :f].double().cpu().numpy() - want)
    assert (err <= (2.0 ** -8 + 2.0 ** -15) * np.abs(want) + 2.0 ** -126).all()
    assert bool((h[:, f:] == 7.0).all())
    check_stored(g8, f, typ, *ref.quantize(gv, typ))
    if gated:
        check_stored(u8, f, typ, *ref.quantize(uv, typ))
    # backward, from the checkpoint alone
    dh, dhv = bf16(r.standard_normal((t, f)) * 1e-2)
    out = torch.full((t, 2 * f), 7.0, dtype=torch.bfloat16, device="cuda")
    sbl.sbl_glu_backward(d, act, g8, u8 if gated else None, strided(dh), out[:, :f], out[:, f:] if gated else None)
    gq, uq = ref.value(gv, typ), ref.value(uv, typ)
    a, da = ref.act(gq, act)
    # silu' = s (1 + g (1 - s)) cancels near its zero: its error is relative to s (1 + |g|)
    s = 1.0 if act else 1 / (1 + np.exp(-gq))
    slack = 2.0 ** -15 * (np.abs(da) + (s * (1 + np.abs(gq)) if act == 0 else 0))
    up = uq if gated else np.ones_like(uq)
    got = out[:, :f].double().cpu().numpy()
    assert (np.abs(got - dhv * up * da) <= 2.0 ** -8 * np.abs(dhv * up * da) + 2 * np.abs(dhv * up) * slack + 2.0 ** -126).all()
    got = out[:, f:].double().cpu().numpy()
    if gated:
        assert (np.abs(got - dhv * a) <= (2.0 ** -8 + 2.0 ** -15) * np.abs(dhv * a) + 2.0 ** -126).all()
    else:
        assert (got == 7.0).all()


@pytest.mark.parametrize("act", [0, 1])
def test_glu_backward_against_differences(act):
    """dG from the kernel against (L(g + h) - L(g - h)) / 2h in 64 bits at the checkpointed values."""
    sbl = sbl_mod()
    r = rng(act, 15)
    t, f = 4, 64
    (g, gv), (u, uv), (dh, dhv) = (bf16(r.standard_normal((t, f))) for _ in range(3))
    d, g8 = new(sbl, t, f, ref.I8)
    _, u8 = new(sbl, t, f, ref.I8)
    sbl.sbl_glu_forward(d, act, g, u, None, g8, u8)
    dg, du = torch.empty_like(g), torch.empty_like(g)
    sbl.sbl_glu_backward(d, act, g8, u8, dh, dg, du)
    gq, uq, h = ref.value(gv, ref.I8), ref.value(uv, ref.I8), 1e-5
    num = dhv * uq * (ref.act(gq + h, act)[0] - ref.act(gq - h, act)[0]) / (2 * h)
    # half a bf16 step, and the difference quotient's own h^2 and rounding error
    assert (np.abs(dg.double().cpu().numpy() - num) <= 2.0 ** -8 * np.abs(num) + 2e-5 * np.abs(dhv * uq)).all()
    num = dhv * (ref.act(gq, act)[0] * (uq + h) - ref.act(gq, act)[0] * (uq - h)) / (2 * h)
    assert (np.abs(du.double().cpu().numpy() - num) <= 2.0 ** -7 * np.abs(num) + 1e-9).all()


def test_marked_blocks_stay_nan_through_the_activation():
    sbl = sbl_mod()
    x = rng(16).standard_normal((3, 256))
    x[1, 5] = np.nan
    g, _ = bf16(x)
    for act in (0, 1):
        d, g8 = new(sbl, 3, 256, ref.E4M3)
        sbl.sbl_glu_forward(d, act, g, None, None, g8)
        dg = torch.empty_like(g)
        sbl.sbl_glu_backward(d, act, g8, None, torch.ones_like(g), dg, None)
        nan = torch.isnan(dg).cpu().numpy()
        assert nan[1, :128].all() and nan.sum() == 128


# --------------------------------------------------------------------- norm

@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("t,k", [(1, 16), (9, 896), (130, 144), (3, 2048), (5, 4112), (700, 256), (2, 11008), (2, 20000), (2, 65536)])
@pytest.mark.parametrize("gains,residual", [(True, True), (True, False), (False, True)])
def test_rmsnorm(typ, t, k, gains, residual):
    sbl = sbl_mod()
    r = rng(typ, t, k, 17)
    (x, xv), (du, duv), (dr, drv) = bf16(r.standard_normal((t, k)) * 3), bf16(r.standard_normal((t, k))), bf16(r.standard_normal((t, k)))
    g, gv = bf16(1 + 0.2 * r.standard_normal((1, k)))
    g = g.view(-1) if gains else None
    gv = gv if gains else np.ones((1, k))
    eps = float(np.float32(1e-5))  # the same number for both entry points
    d, x8 = new(sbl, t, k, typ)
    q, q0 = (torch.empty((t, k), dtype=torch.int8, device="cuda") for _ in range(2))
    s, s0 = (torch.empty(t, dtype=torch.float32, device="cuda") for _ in range(2))
    sbl.sbl_quantize_act_rmsnorm_checkpoint(d, x, g, eps, q, s, x8)
    sbl.sbl_quantize_act_rmsnorm(x, t, k, g, eps, q0, s0)
    # the forward's scales are the other entry point's; its codes are those of the factor 127 * (1 / a), which the
    # quantiser's definition puts within one of the other's
    assert torch.equal(s, s0) and int((q.int() - q0.int()).abs().max()) <= 1
    rn = torch.from_numpy(1 / np.sqrt((xv * xv).sum(1, keepdims=True) / k + eps)).float()
    un = torch.from_numpy(xv).float() * rn
    un = un * torch.from_numpy(gv).float() if gains else un
    an = un.abs().amax(1, keepdim=True)
    assert torch.equal(q.cpu(), torch.round(un * (an.reciprocal() * 127)).to(torch.int8))
    check_stored(x8, k, typ, *ref.quantize(xv, typ))
    dx = torch.empty((t, k), dtype=torch.bfloat16, device="cuda")
    dg = torch.full((k + 4,), 6.0, dtype=torch.float32, device="cuda")
    ws = sbl.alloc_workspace(sbl.sbl_rmsnorm_backward_workspace_bytes(t, k))
    ws.fill_(0xFF)
    if residual:
        dx.copy_(dr)  # in place: the residual gradient's buffer receives the sum
    sbl.sbl_rmsnorm_backward(d, x8, g, 1e-5, du, dx if residual else None, dx, dg[:k] if gains else None, ws)
    xq = ref.value(xv, typ)
    wx, wg = ref.rmsnorm_backward(xq, gv, 1e-5, duv, drv if residual else None)
    rr = 1 / np.sqrt((xq * xq).mean(1, keepdims=True) + 1e-5)
    # fp32: row sums of k terms, a thread's share (at most 64) in a chain, then a tree: below 2^-24 (64 + 12) of the sum
    # of magnitudes; a handful of roundings after it
    slack = 2.0 ** -24 * (90 * np.abs(xq) * rr ** 3 * (np.abs(duv * gv) * np.abs(xq)).mean(1, keepdims=True) +
                          90 * np.abs(rr * duv * gv) + 2 * np.abs(wx))
    assert (np.abs(dx.double().cpu().numpy() - wx) <= 2.0 ** -8 * np.abs(wx) + 2 * slack).all()
    if gains:
        got = dg[:k].double().cpu().numpy()
        mags = np.abs(duv * xq * rr).sum(0)
        # t terms in chains of at most t, each term rounded three times, r itself as above
        assert (np.abs(got - wg) <= 2.0 ** -24 * (t + 90) * mags).all()
    assert bool((dg[k:] == 6.0).all())


def test_rmsnorm_backward_against_differences():
    sbl = sbl_mod()
    r = rng(18)
    t, k, h = 3, 48, 1e-5
    (x, xv), (du, duv) = bf16(r.standard_normal((t, k))), bf16(r.standard_normal((t, k)))
    g, gv = bf16(1 + 0.2 * r.standard_normal((1, k)))
    d, x8 = new(sbl, t, k, ref.I8)
    sbl.sbl_b8_quantize(d, x, x8)
    dx = torch.empty_like(x)
    sbl.sbl_rmsnorm_backward(d, x8, g.view(-1), 1e-5, du, None, dx, None, None)
    xq = ref.value(xv, ref.I8)

    def loss(z):
        return (duv * z / np.sqrt((z * z).mean(1, keepdims=True) + 1e-5) * gv).sum(1)

    num = np.empty((t, k))
    for j in range(k):
        e = np.zeros((1, k))
        e[0, j] = h
        num[:, j] = (loss(xq + e) - loss(xq - e)) / (2 * h)
    assert (np.abs(dx.double().cpu().numpy() - num) <= 2.0 ** -8 * np.abs(num) + 1e-6).all()


def test_results_do_not_depend_on_the_run():
    """The gains' gradient and an accumulated dW, twice on the same inputs."""
    sbl = sbl_mod()
    r = rng(19)
    t, k = 900, 640
    (x, _), (du, _) = bf16(r.standard_normal((t, k))), bf16(r.standard_normal((t, k)))
    g = torch.ones(k, dtype=torch.bfloat16, device="cuda")
    d, x8 = new(sbl, t, k, 0)
    sbl.sbl_b8_quantize(d, x, x8)
    ws = sbl.alloc_workspace(sbl.sbl_rmsnorm_backward_workspace_bytes(t, k))
    got = []
    for _ in range(2):
        dx, dg = torch.empty_like(x), torch.empty(k, device="cuda")
        sbl.sbl_rmsnorm_backward(d, x8, g, 1e-5, du, None, dx, dg, ws)
        got.append((dx, dg))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("spread", [0, 3, 5, 6, 12, 40])
@pytest.mark.parametrize("rows,cols", [(128, 128), (200, 272)])
def test_transpose_of_scales_near_and_far_apart(spread, rows, cols):
    """e4m3 to e4m3 over rows whose scales differ by up to 2^spread, columns far below the rest and empty ones."""
    sbl = sbl_mod()
    r = rng(spread, rows, 20)
    x = r.standard_normal((rows, cols)) * np.exp2(r.integers(-spread, 1, (rows, 1)))
    x[:, 5] *= 2.0 ** -7
    x[:, 9] *= 2.0 ** -12
    x[:, 11] *= 2.0 ** -16
    x[:, 17] = 0
    x[:, 40:44] = 448.0 * np.exp2(r.integers(-10, 1, (rows, 4)))
    t, v = bf16(x)
    d, m = new(sbl, rows, cols, ref.E4M3)
    _, mt = new(sbl, cols, rows, ref.E4M3)
    sbl.sbl_b8_quantize(d, t, m)
    sbl.sbl_b8_transpose(d, m, mt)
    check_stored(mt, rows, ref.E4M3, *ref.quantize(np.ascontiguousarray(ref.value(v, ref.E4M3).T), ref.E4M3))


@pytest.mark.parametrize("m,n,fp32", [(16, 16, False), (64, 48, True), (80, 32, False)])
def test_gemm_over_a_very_long_k(m, n, fp32):
    """A reduction whose scales no longer fit beside the few-row kernel's accumulators."""
    sbl = sbl_mod()
    k = 250_000
    ad, a, av = operands(sbl, rng(m, n, 21), m, k, ref.E4M3)
    bd, b, bv = operands(sbl, rng(m, n, 22), n, k, ref.E4M3)
    out = torch.empty((m, n), dtype=torch.float32 if fp32 else torch.bfloat16, device="cuda")
    sbl.sbl_b8_gemm(ad, a, bd, b, out)
    check_product(out.double().cpu().numpy(), av, bv, ref.HALF["fp32" if fp32 else "bf16"])


class Guarded:
    """A tensor between two guard bands of 512 bytes."""

    def __init__(self, *shape, dtype=torch.uint8):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        self.raw = torch.full((1024 + -(-n // 512) * 512,), 0xC3, dtype=torch.uint8, device="cuda")
        self.n = n
        self.t = self.raw[512:512 + n].view(dtype).view(*shape)

    def intact(self):
        return bool((self.raw[:512] == 0xC3).all()) and bool((self.raw[512 + self.n:] == 0xC3).all())


@pytest.mark.parametrize("t,k,o", [(1, 16, 16), (13, 400, 272), (130, 1040, 144), (300, 656, 528)])
def test_nothing_is_written_past_the_outputs(t, k, o):
    sbl = sbl_mod()
    r = rng(t, k, o, 23)
    held = []

    def g(*shape, dtype=torch.uint8):
        held.append(Guarded(*shape, dtype=dtype))
        return held[-1].t

    def mat(rows, cols, typ):
        d = sbl.b8_desc(rows, cols, typ)
        return d, sbl.Block8(codes=g(rows, sbl.sbl_b8_row_bytes(d)), scales=g(sbl.sbl_b8_scale_bytes(d)))

    bf, f32 = torch.bfloat16, torch.float32
    (x, _), (dy, _), (u, _) = bf16(r.standard_normal((t, k))), bf16(r.standard_normal((t, o))), bf16(r.standard_normal((t, k)))
    w = torch.from_numpy(r.standard_normal((o, k)).astype(np.float32)).cuda()
    wd, wq = mat(o, k, 0)
    _, wt = mat(k, o, 0)
    xd, xq = mat(t, k, 0)
    sbl.sbl_b8_quantize(wd, w, wq, wt, sbl.SBL_B8_TILES)
    sbl.sbl_b8_linear_forward(wd, wq, x, t, xq, g(t, o, dtype=bf))
    ws = g(sbl.sbl_b8_linear_workspace_bytes(wd, t))
    sbl.sbl_b8_linear_backward(wd, wt, xq, dy, t, g(t, k, dtype=bf), g(o, k, dtype=f32), ws)
    for typ in TYPES:
        d, m = mat(t, k, typ)
        _, mt = mat(k, t, typ)
        sbl.sbl_b8_quantize(d, x, m)
        sbl.sbl_b8_quantize(d, x, m, mt)
        sbl.sbl_b8_transpose(d, m, mt)
        sbl.sbl_b8_dequantize(d, m, g(t, k, dtype=bf))
        (_, g8), (_, u8) = mat(t, k, typ), mat(t, k, typ)
        sbl.sbl_glu_forward(d, 0, x, u, g(t, k, dtype=bf), g8, u8)
        sbl.sbl_glu_backward(d, 0, g8, u8, u, g(t, k, dtype=bf), g(t, k, dtype=bf))
        _, x8 = mat(t, k, typ)
        gain = torch.ones(k, dtype=bf, device="cuda")
        sbl.sbl_quantize_act_rmsnorm_checkpoint(d, x, gain, 1e-5, g(t, k, dtype=torch.int8), g(t, dtype=f32), x8)
        sbl.sbl_rmsnorm_backward(d, x8, gain, 1e-5, u, None, g(t, k, dtype=bf), g(k, dtype=f32),
                                 g(sbl.sbl_rmsnorm_backward_workspace_bytes(t, k)))
    torch.cuda.synchronize()
    assert all(h.intact() for h in held)
    assert sbl.sbl_device_error() == 0


@pytest.mark.parametrize("t", [1, 20, 64, 100, 300])
@pytest.mark.parametrize("fp32", [False, True])
def test_linear_forward_into_a_wider_buffer(t, fp32):
    sbl = sbl_mod()
    o, k = 272, 1040
    r = rng(t, 24)
    w = r.standard_normal((o, k)).astype(np.float32)
    x, xv = bf16(r.standard_normal((t, k)))
    wd, wq = new(sbl, o, k, 0)
    _, xq = new(sbl, t, k, 0)
    sbl.sbl_b8_quantize(wd, torch.from_numpy(w).cuda(), wq, None, sbl.SBL_B8_TILES)
    out = torch.full((t, o + 16), 3.0, dtype=torch.float32 if fp32 else torch.bfloat16, device="cuda")
    sbl.sbl_b8_linear_forward(wd, wq, x, t, xq, out[:, :o])
    check_product(out[:, :o].double().cpu().numpy(), ref.value(xv, 0), ref.value(w.astype(np.float64), 0, True),
                  ref.HALF["fp32" if fp32 else "bf16"])
    assert bool((out[:, o:] == 3.0).all())
    check_stored(xq, k, 0, *ref.quantize(xv, 0))


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("outputs", ["h", "g", "u", "hg", "gu", "hu"])
def test_glu_any_outputs(gated, outputs):
    sbl = sbl_mod()
    if not gated and "u" in outputs:
        return  # refused: no checkpoint of an absent input
    t, f = 37, 272
    r = rng(25)
    (g, gv), (u, uv) = bf16(r.standard_normal((t, f))), bf16(r.standard_normal((t, f)))
    d, g8 = new(sbl, t, f, 0)
    _, u8 = new(sbl, t, f, 0)
    h = torch.full((t, f), 7.0, dtype=torch.bfloat16, device="cuda")
    sbl.sbl_glu_forward(d, 1, g, u if gated else None, h if "h" in outputs else None, g8 if "g" in outputs else None,
                        u8 if "u" in outputs else None)
    want = ref.act(gv, 1)[0] * (uv if gated else 1.0)
    if "h" in outputs:
        assert (np.abs(h.double().cpu().numpy() - want) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(want) + 2.0 ** -126).all()
    else:
        assert bool((h == 7.0).all())
    for m, v, name in ((g8, gv, "g"), (u8, uv, "u")):
        if name in outputs:
            check_stored(m, f, 0, *ref.quantize(v, 0))
        else:
            assert bool((m.codes == 0xA5).all()) and bool((m.scales == 0xA5).all())


@pytest.mark.parametrize("offset", [8, 16, 24])
def test_rows_aligned_to_16_bytes_only(offset):
    """Inputs and outputs that start `offset` elements into a buffer (16 bytes each step of 8)."""
    sbl = sbl_mod()
    t, f = 21, 528
    r = rng(offset, 26)

    def shifted(a=None):
        buf = torch.zeros(t * f + 64, dtype=torch.bfloat16, device="cuda")
        v = buf[offset:offset + t * f].view(t, f)
        if a is not None:
            v.copy_(a)
        return v

    (g, gv), (u, uv), (dh, dhv) = (bf16(r.standard_normal((t, f))) for _ in range(3))
    d, g8 = new(sbl, t, f, 2)
    _, u8 = new(sbl, t, f, 2)
    h, dg, du, back = shifted(), shifted(), shifted(), shifted()
    sbl.sbl_glu_forward(d, 1, shifted(g), shifted(u), h, g8, u8)
    sbl.sbl_glu_backward(d, 1, g8, u8, shifted(dh), dg, du)
    sbl.sbl_b8_dequantize(d, g8, back)
    h2, dg2, du2, back2 = (torch.empty_like(g) for _ in range(4))
    sbl.sbl_glu_forward(d, 1, g, u, h2, g8, u8)
    sbl.sbl_glu_backward(d, 1, g8, u8, dh, dg2, du2)
    sbl.sbl_b8_dequantize(d, g8, back2)
    for a, b in ((h, h2), (dg, dg2), (du, du2), (back, back2)):
        assert torch.equal(a, b)
    x8, x8s = new(sbl, t, f, 0)[1], new(sbl, t, f, 0)[1]
    d0 = sbl.b8_desc(t, f)
    sbl.sbl_b8_quantize(d0, g, x8)
    sbl.sbl_b8_quantize(d0, shifted(g), x8s)
    assert torch.equal(x8.codes, x8s.codes) and torch.equal(x8.scales, x8s.scales)
    dx, dxs = torch.empty_like(g), shifted()
    sbl.sbl_rmsnorm_backward(d0, x8, None, 1e-5, u, dh, dx, None, None)
    sbl.sbl_rmsnorm_backward(d0, x8, None, 1e-5, shifted(u), shifted(dh), dxs, None, None)
    assert torch.equal(dx, dxs)


def test_offsets_past_32_bits():
    """Matrices of more than 2^32 elements: their last rows."""
    sbl = sbl_mod()
    rows, cols, n = 65700, 65536, 150
    assert rows * cols > 1 << 32
    tail, tv = bf16(rng(27).standard_normal((n, cols)))
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    x[-n:] = tail
    d = sbl.b8_desc(rows, cols)
    q = sbl.alloc_b8(d)
    sbl.sbl_b8_quantize(d, x, q)
    y, e = ref.quantize(tv, 0)
    assert np.array_equal(ref.code_values(0)[q.codes[-n:].cpu().numpy()], y)
    out = torch.zeros_like(x)
    sbl.sbl_b8_dequantize(d, q, out)
    want = torch.from_numpy(ref.decode(y, e).astype(np.float32)).to(torch.bfloat16)
    assert torch.equal(out[-n:].cpu(), want)
    assert not out[:-n].any()
    bd, b, bv = operands(sbl, rng(28), 16, cols, 0)
    prod = torch.empty((rows, 16), dtype=torch.float32, device="cuda")
    sbl.sbl_b8_gemm(d, q, bd, b, prod)
    check_product(prod[-n:].double().cpu().numpy(), ref.decode(y, e), bv, ref.HALF["fp32"])
    assert not prod[:-n].any()
    dg = torch.zeros_like(x)
    sbl.sbl_glu_backward(d, 1, q, None, x, dg, None)
    g = ref.decode(y, e)
    want = tv * 2 * np.maximum(g, 0)
    assert (np.abs(dg[-n:].double().cpu().numpy() - want) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(want) + 2.0 ** -126).all()
    del out, dg, prod
    qt = sbl.alloc_b8(sbl.b8_desc(cols, rows))
    sbl.sbl_b8_transpose(d, q, qt)
    # the last rows of the source are the last columns of the transpose; its blocks of 128 start at multiples of 128
    first = (rows - n) // 128 * 128
    lead = rows - n - first
    blk = np.concatenate([np.zeros((lead, 64)), g[:, -64:]])
    yt, _ = ref.quantize(np.ascontiguousarray(blk.T), 0)
    assert np.array_equal(ref.code_values(0)[qt.codes[-64:, first:rows].cpu().numpy()], yt)


def test_first_call_of_a_process_inside_a_capture():
    import subprocess
    import sys
    code = """
import torch
from sparsity_sbl_quantize_b200 import sbl
wd = sbl.b8_desc(256, 512)
w, x8 = sbl.alloc_b8(wd), sbl.alloc_b8(sbl.b8_desc(80, 512))
W, X = torch.randn(256, 512, device="cuda"), torch.randn(80, 512, device="cuda").bfloat16()
Y = torch.zeros(80, 256, device="cuda", dtype=torch.bfloat16)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    sbl.sbl_b8_quantize(wd, W, w, None, sbl.SBL_B8_TILES)
    sbl.sbl_b8_linear_forward(wd, w, X, 80, x8, Y)
g.replay()
torch.cuda.synchronize()
got = Y.clone()
sbl.sbl_b8_linear_forward(wd, w, X, 80, x8, Y)
torch.cuda.synchronize()
assert torch.equal(got, Y) and bool(got.any()) and sbl.sbl_device_error() == 0
print("ok")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "ok" in r.stdout, r.stderr


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("t,k", [(5, 144), (3, 2064), (2, 8208)])
@pytest.mark.parametrize("power", [-58, -45, 45, 56])
def test_rmsnorm_backward_of_small_and_large_rows(typ, t, k, power):
    """Rows whose r^3 is outside fp32's range while the gradient is not; eps 0.  The bounds are test_rmsnorm's."""
    sbl = sbl_mod()
    r = rng(typ, t, k, power + 100, 31)
    (x, xv), (du, duv) = bf16(r.standard_normal((t, k)) * 2.0 ** power), bf16(r.standard_normal((t, k)))
    g, gv = bf16(1 + 0.2 * r.standard_normal((1, k)))
    d, x8 = new(sbl, t, k, typ)
    sbl.sbl_b8_quantize(d, x, x8)
    dx, dg = torch.empty_like(x), torch.empty(k, dtype=torch.float32, device="cuda")
    ws = sbl.alloc_workspace(sbl.sbl_rmsnorm_backward_workspace_bytes(t, k))
    sbl.sbl_rmsnorm_backward(d, x8, g.view(-1), 0.0, du, None, dx, dg, ws)
    xq = ref.value(xv, typ)
    wx, wg = ref.rmsnorm_backward(xq, gv, 0.0, duv)
    rr = 1 / np.sqrt((xq * xq).mean(1, keepdims=True))
    slack = 2.0 ** -24 * (90 * np.abs(xq) * rr ** 3 * (np.abs(duv * gv) * np.abs(xq)).mean(1, keepdims=True) +
                          90 * np.abs(rr * duv * gv) + 2 * np.abs(wx))
    assert (np.abs(dx.double().cpu().numpy() - wx) <= 2.0 ** -8 * np.abs(wx) + 2 * slack).all()
    assert (np.abs(dg.double().cpu().numpy() - wg) <= 2.0 ** -24 * (t + 90) * np.abs(duv * xq * rr).sum(0)).all()


def test_rmsnorm_backward_of_an_empty_row_with_a_small_eps():
    """x = 0: dX = dU g / sqrt(eps), with r^3 = 1e45 out of range."""
    sbl = sbl_mod()
    r = rng(32)
    du, duv = bf16(r.standard_normal((3, 272)))
    x = torch.zeros_like(du)
    x[1] = 1.0
    d, x8 = new(sbl, 3, 272, 0)
    sbl.sbl_b8_quantize(d, x, x8)
    dx = torch.empty_like(x)
    sbl.sbl_rmsnorm_backward(d, x8, None, 1e-30, du, None, dx, None, None)
    want = duv[[0, 2]] * 1e15
    got = dx.double().cpu().numpy()
    assert np.isfinite(got).all()
    assert (np.abs(got[[0, 2]] - want) <= (2.0 ** -8 + 2.0 ** -20) * np.abs(want)).all()
