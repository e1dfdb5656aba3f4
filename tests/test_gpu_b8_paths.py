"""The paths of the 8-bit block operators that only large or odd sizes take, against their definitions in 64 bits on the
device: several tiles a CTA and segmented sums in the product, gradients over many tokens, e5m2 activations, the row
loop of the norm's backward in every variant, several scale words a warp and a CTA per row in the element-wise kernels,
and silu over its whole range."""
import pytest
import torch

import b8_ref as ref
import b8_torch as bt
from gpu_case import sbl_mod

pytestmark = pytest.mark.gpu

TYPES = [ref.E4M3, ref.E5M2, ref.I8]
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24

# D [m, n] over k.  Which kernel each takes (tile width, segments, tiles a CTA) is asserted in test_b8_paths_host.py.
PRODUCTS = [(2064, 1040, 400), (2560, 4096, 384), (2561, 4112, 1000), (2816, 1664, 128), (300, 1040, 130),
            (2064, 1040, 4400), (2560, 4096, 8336), (2816, 1664, 4300), (300, 144, 12400), (3001, 4112, 4224)]
LINEAR = [(4500, 2048, 1552), (5000, 400, 272), (9001, 1040, 2064), (300, 272, 528)]  # tokens, outputs, inputs


def gen(*key):
    g = torch.Generator(device="cuda")
    g.manual_seed(sum((i + 1) * 1000003 ** i * (k + 7) for i, k in enumerate(key)) % (1 << 62))
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float64)


def operand(sbl, g, rows, k, typ):
    """A stored matrix [rows, k] of values over several binades (as a transpose: any k), and its values."""
    r16 = -(-rows // 16) * 16
    x = (randn(g, k, r16) * torch.exp2(torch.randint(-3, 4, (k, 1), generator=g, device="cuda").double())).to(BF)
    d = sbl.b8_desc(r16, k, typ)
    m = sbl.alloc_b8(d)
    sbl.sbl_b8_quantize(sbl.b8_desc(k, r16, typ), x, None, m)
    v = bt.stored(m, d)
    if r16 != rows:  # the stored rows of a smaller matrix, in its own scale order
        e, d16 = bt.exponents(m, d)[:rows], d
        d = sbl.b8_desc(rows, k, typ)
        s = sbl.alloc_b8(d)
        s.codes.copy_(m.codes[:rows])
        s.scales.fill_(127)
        i, j = torch.arange(rows, device="cuda").view(-1, 1), torch.arange(e.shape[1], device="cuda").view(1, -1)
        rp = -(-rows // 128) * 128
        s.scales[4 * ((j // 4) * rp + 128 * (i // 128) + 4 * (i % 32) + (i % 128) // 32) + j % 4] = (e + 127).to(torch.uint8)
        assert d16.rows == r16
        m, v = s, v[:rows]
    return d, m, v


def check_product(got, a, b, half, segmented):
    """Truncating accumulation: (K / 32 + 5) 2^-23 of the sum of magnitudes, K at most 4096 where it is cut into segments,
    which are then added with rounding."""
    k = a.shape[1]
    want, mags = a @ b.t(), a.abs() @ b.abs().t()
    steps = (-(-min(k, 4096) // 32) + 5) * 2.0 ** -23 + -(-k // 4096) * U if segmented else (-(-k // 32) + 5) * 2.0 ** -23
    err = (got.double() - want).abs() - half * want.abs() - (1 + half) * steps * mags
    assert bool((err <= 0).all()), float(err.max())


@pytest.mark.parametrize("ta,tb", [(0, 0), (1, 0)])
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_products(m, n, k, ta, tb):
    sbl = sbl_mod()
    (ad, a, av), (bd, b, bv) = operand(sbl, gen(m, k, ta), m, k, ta), operand(sbl, gen(n, k, tb, 1), n, k, tb)
    for fp32 in (False, True):
        out = torch.full((m + 1, n + 16), 3.0, dtype=F32 if fp32 else BF, device="cuda")
        sbl.sbl_b8_gemm(ad, a, bd, b, out[:m, :n])
        check_product(out[:m, :n], av, bv, ref.HALF["fp32" if fp32 else "bf16"], bt.product_kernel(m, n, k, fp32)[2])
        assert bool((out[m:] == 3.0).all()) and bool((out[:, n:] == 3.0).all())
    once = out[:m, :n].clone()
    sbl.sbl_b8_gemm(ad, a, bd, b, out[:m, :n], accumulate=True)
    assert torch.equal(out[:m, :n], once + once)
    assert sbl.sbl_device_error() == 0


@pytest.mark.parametrize("xt,gt", [(ref.E4M3, ref.E4M3), (ref.E5M2, ref.E5M2), (ref.E5M2, ref.E4M3)])
@pytest.mark.parametrize("t,o,k", LINEAR)
def test_linear_over_many_tokens(t, o, k, xt, gt):
    sbl = sbl_mod()
    g = gen(t, o, k, xt, gt)
    w, x, dy = (randn(g, o, k) * 0.02).float(), randn(g, t, k).to(BF), (randn(g, t, o) * 1e-3).to(BF)
    wd, xd, gd = sbl.b8_desc(o, k), sbl.b8_desc(t, k, xt), sbl.b8_desc(t, o, gt)
    wq, wt, xq = sbl.alloc_b8(wd), sbl.alloc_b8(sbl.b8_desc(k, o)), sbl.alloc_b8(xd)
    sbl.sbl_b8_quantize(wd, w, wq, wt, sbl.SBL_B8_TILES)
    y, dx, dw = torch.empty(t, o, dtype=BF, device="cuda"), torch.empty(t, k, dtype=BF, device="cuda"), torch.empty(o, k, device="cuda")
    ws = sbl.alloc_workspace(sbl.sbl_b8_linear_workspace_bytes(wd, t))
    ws.fill_(0xFF)
    sbl.sbl_b8_linear_forward(wd, wq, x, t, xq, y, x_type=xt)
    sbl.sbl_b8_linear_backward(wd, wt, xq, dy, t, dx, dw, ws, x_type=xt, g_type=gt)
    codes, e = bt.quantize(x.double(), xt)
    assert torch.equal(bt.code_values(xq, xd), codes) and torch.equal(bt.exponents(xq, xd), e)
    x8, wv = bt.decode(codes, e), bt.stored(wq, wd)
    assert torch.equal(bt.stored(wt, sbl.b8_desc(k, o)), wv.t())
    check_product(y, x8, wv, ref.HALF["bf16"], False)
    check_product(dx, bt.decode(*bt.quantize(dy.double(), gt)), wv.t(), ref.HALF["bf16"], False)
    a = bt.decode(*bt.quantize(dy.double().t().contiguous(), gt))
    b = bt.decode(*bt.quantize(x8.t().contiguous(), xt))
    check_product(dw, a, b, ref.HALF["fp32"], t > 4096)
    once = dw.clone()
    sbl.sbl_b8_linear_backward(wd, None, xq, dy, t, None, dw, ws, x_type=xt, g_type=gt, accumulate=True)
    assert torch.equal(dw, once + once)
    assert gd.rows == t and sbl.sbl_device_error() == 0


@pytest.mark.parametrize("t", [1, 5, 16, 17, 33, 64, 65])
@pytest.mark.parametrize("o,k", [(272, 400), (1040, 2064), (144, 9232)])
@pytest.mark.parametrize("wt", [ref.E4M3, ref.E5M2])
@pytest.mark.parametrize("fp32", [False, True])
def test_few_tokens_in_e5m2(t, o, k, wt, fp32):
    """Activations quantised to e5m2 inside the few-row kernel and before it."""
    sbl = sbl_mod()
    g = gen(t, o, k, wt)
    wd, xd = sbl.b8_desc(o, k, wt), sbl.b8_desc(t, k, ref.E5M2)
    w, x8 = sbl.alloc_b8(wd), sbl.alloc_b8(xd)
    x8.codes.fill_(0xA5)
    x8.scales.fill_(0xA5)
    sbl.sbl_b8_quantize(wd, randn(g, o, k).float(), w, None, sbl.SBL_B8_TILES)
    x = (randn(g, t, k) * torch.exp2(torch.randint(-8, 8, (t, 1), generator=g, device="cuda").double())).to(BF)
    y = torch.full((t + 1, o), 3.0, dtype=F32 if fp32 else BF, device="cuda")
    sbl.sbl_b8_linear_forward(wd, w, x, t, x8, y[:t], x_type=ref.E5M2)
    codes, e = bt.quantize(x.double(), ref.E5M2)
    assert torch.equal(bt.code_values(x8, xd), codes) and torch.equal(bt.exponents(x8, xd), e)
    blocks, rp = -(-k // 128), -(-t // 128) * 128
    scales = x8.scales.view(-1, rp, 4)
    assert int((scales != 127).sum()) == int((e != 0).sum()) and scales.shape[0] == -(-blocks // 4)  # padding is 127
    check_product(y[:t], bt.decode(codes, e), bt.stored(w, wd), ref.HALF["fp32" if fp32 else "bf16"], False)
    assert bool((y[t:] == 3.0).all()) and sbl.sbl_device_error() == 0


# One size for each variant of the norm's backward, tokens for two steps of its row loop and part of a third on 148 SMs.
NORM = [(144, 5000), (656, 2600), (1040, 1300), (4096, 650), (4112, 333), (8208, 170), (20000, 91), (65536, 45)]


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("k,t", NORM)
@pytest.mark.parametrize("gains,residual", [(True, True), (False, False)])
def test_norm_backward_over_several_rows_a_cta(typ, k, t, gains, residual):
    """The bounds of test_gpu_b8_range.py."""
    sbl = sbl_mod()
    rng = gen(typ, k, t)
    x, du, dr = (randn(rng, t, k) * 3).to(BF), randn(rng, t, k).to(BF), randn(rng, t, k).to(BF)
    g = (1 + 0.2 * randn(rng, k)).to(BF) if gains else None
    d = sbl.b8_desc(t, k, typ)
    x8 = sbl.alloc_b8(d)
    sbl.sbl_b8_quantize(d, x, x8)
    dx = dr.clone() if residual else torch.full((t, k), 7.0, dtype=BF, device="cuda")
    dg = torch.full((k + 4,), 6.0, device="cuda")
    ws = sbl.alloc_workspace(sbl.sbl_rmsnorm_backward_workspace_bytes(t, k))
    ws.fill_(0xFF)
    sbl.sbl_rmsnorm_backward(d, x8, g, 1e-5, du, dx if residual else None, dx, dg[:k] if gains else None, ws)
    xv, duv = bt.stored(x8, d), du.double()
    v = duv * g.double() if gains else duv
    r = 1 / torch.sqrt((xv * xv).mean(1, keepdim=True) + 1e-5)
    n = xv * r
    dn = r * (v - n * (v * n).mean(1, keepdim=True))
    want = dn + dr.double() if residual else dn
    slack = U * (90 * r * n.abs() * (v * n).abs().mean(1, keepdim=True) + 30 * (r * v).abs() + 30 * dn.abs() + 2 * want.abs())
    err = (dx.double() - want).abs() - 2.0 ** -8 * want.abs() - (1 + 2.0 ** -8) * slack
    assert bool((err <= 0).all()), float(err.max())
    if gains:
        terms = duv * n
        err = (dg[:k].double() - terms.sum(0)).abs() - U * (t + 32) * terms.abs().sum(0)
        assert bool((err <= 0).all()), float(err.max())
    assert bool((dg[k if gains else 0:] == 6.0).all())


# (rows, cols): two, three and four scale words a warp, the last warp of a row with fewer; then a CTA per row
WALKS = [(8000, 2064), (20000, 1040), (16000, 2064), (1000, 65536), (1300, 4112)]


@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("rows,cols", WALKS)
@pytest.mark.parametrize("src", [BF, F32])
def test_quantise_and_read_many_rows(typ, rows, cols, src):
    sbl = sbl_mod()
    g = gen(typ, rows, cols)
    x = (randn(g, rows, cols) * torch.exp2(torch.randint(-20, 20, (rows, 1), generator=g, device="cuda").double())).to(src)
    x[5] = 0
    d = sbl.b8_desc(rows, cols, typ)
    m = sbl.alloc_b8(d)
    m.codes.fill_(0xA5)
    m.scales.fill_(0xA5)
    sbl.sbl_b8_quantize(d, x, m)
    y, e = bt.quantize(x.double(), typ)
    assert torch.equal(bt.code_values(m, d), y) and torch.equal(bt.exponents(m, d), e)
    assert int((m.scales != 127).sum()) == int((e != 0).sum())  # padded rows and blocks are 127
    out = torch.empty(rows, cols, dtype=BF, device="cuda")
    sbl.sbl_b8_dequantize(d, m, out)
    assert torch.equal(out, bt.decode(y, e).to(BF))


def silu(g):
    s, rest = torch.special.expit(g), torch.special.expit(-g)
    return g * s, s + g * s * rest, s


def act_bounds(g, act):
    """act(g), act'(g) and bounds of their fp32 errors.  relu2: one rounding.  silu: e^-|g| is the square of an ex2.approx
    (2^-22 each) of a product off by 1.5 2^-24 of itself, so off by (1.5 |g| + 9) 2^-24; 1 + t, its rcp.approx (2^-23) and two
    products add 6; silu' = s (1 + g rest) loses that against s (1 + |g|).  Below 2^-126 each of t, s and their product
    with g is off by half of 2^-149 more, g times over."""
    if act == 1:
        p = g.clamp(min=0)
        return p * p, 2 * p, U * p * p, torch.zeros_like(g)
    a, da, s = silu(g)
    rel, tail = U * (1.5 * g.abs() + 16), 2.0 ** -149 * (2 + 2 * g.abs())
    return a, da, rel * a.abs() + tail, 2 * rel * s * (1 + g.abs()) + tail


def check_act(got, factor, value, bound, roundings):
    """bf16 of factor * value, the value off by bound; `roundings` fp32 products besides."""
    want = factor * value
    slack = factor.abs() * bound + roundings * U * want.abs()
    err = (got.double() - want).abs() - slack - 2.0 ** -8 * (want.abs() + slack) - 2.0 ** -134 - roundings * 2.0 ** -149
    assert bool((err <= 0).all()), float(err.max())


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("typ", TYPES)
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("t,f", WALKS[:1] + WALKS[2:3] + WALKS[4:])
def test_activation_over_many_rows(act, typ, gated, t, f):
    sbl = sbl_mod()
    r = gen(act, typ, t, f)
    g, u, dh = (randn(r, t, f) * 4).to(BF), randn(r, t, f).to(BF), (randn(r, t, f) * 1e-2).to(BF)
    d = sbl.b8_desc(t, f, typ)
    g8, u8 = sbl.alloc_b8(d), sbl.alloc_b8(d)
    for m in (g8, u8):
        m.codes.fill_(0xA5)
        m.scales.fill_(0xA5)
    h, dg, du = (torch.empty(t, f, dtype=BF, device="cuda") for _ in range(3))
    sbl.sbl_glu_forward(d, act, g, u if gated else None, h, g8, u8 if gated else None)
    a, _, ba, _ = act_bounds(g.double(), act)
    check_act(h, u.double() if gated else torch.ones_like(a), a, ba, 1)
    for m, x in ((g8, g), (u8, u)) if gated else ((g8, g),):
        y, e = bt.quantize(x.double(), typ)
        assert torch.equal(bt.code_values(m, d), y) and torch.equal(bt.exponents(m, d), e)
        assert int((m.scales != 127).sum()) == int((e != 0).sum())
    sbl.sbl_glu_backward(d, act, g8, u8 if gated else None, dh, dg, du if gated else None)
    a, da, ba, bda = act_bounds(bt.stored(g8, d), act)
    check_act(dg, dh.double() * (bt.stored(u8, d) if gated else 1.0), da, bda, 2)
    if gated:
        check_act(du, dh.double(), a, ba, 1)


def test_silu_over_its_whole_range():
    """Forward: every bf16 value from -104 to 104 (below -104 the result is less than half of bf16's smallest)."""
    sbl = sbl_mod()
    bits = torch.arange(0, 1 << 15, dtype=torch.int32, device="cuda")
    v = torch.cat([bits, bits - (1 << 15)]).to(torch.int16).view(BF)
    v = v[torch.isfinite(v) & (v.float().abs() <= 104)]
    v = torch.nn.functional.pad(v, (0, -v.numel() % 1040)).view(-1, 1040)
    d = sbl.b8_desc(*v.shape)
    h = torch.empty_like(v)
    for power in (0, 20):  # up factors of 1 and 2^20: the tail itself, and what the gate leaves of it
        u = torch.full_like(v, 2.0 ** power)
        sbl.sbl_glu_forward(d, 0, v, u, h)
        a, _, ba, _ = act_bounds(v.double(), 0)
        check_act(h, u.double(), a, ba, 1)
    sbl.sbl_glu_forward(d, 0, v, None, h)
    check_act(h, torch.ones_like(a), a, ba, 0)


@pytest.mark.parametrize("power", [-3, -1, 0])
def test_silu_gradient_over_its_whole_range(power):
    """Every int8 code at a scale of 2^power: g from -127 2^power to 127 2^power."""
    sbl = sbl_mod()
    g = torch.arange(-127, 129, device="cuda").double().clamp(max=127).view(2, 128).repeat(4, 2) * 2.0 ** power
    g[:, 0], g[:, 128] = 127 * 2.0 ** power, -127 * 2.0 ** power  # a block's largest, so that its scale is 2^power
    gb = g.to(BF)
    assert torch.equal(gb.double(), g)
    d = sbl.b8_desc(*g.shape, ref.I8)
    g8, u8 = sbl.alloc_b8(d), sbl.alloc_b8(d)
    u = torch.ones_like(gb) * 127
    sbl.sbl_glu_forward(d, 0, gb, u, None, g8, u8)
    assert torch.equal(bt.stored(g8, d), g)
    for scale in (1.0, 2.0 ** 30):
        dh, dg, du = torch.full_like(gb, scale), torch.empty_like(gb), torch.empty_like(gb)
        sbl.sbl_glu_backward(d, 0, g8, u8, dh, dg, du)
        a, da, ba, bda = act_bounds(g, 0)
        check_act(dg, dh.double() * 127, da, bda, 2)
        check_act(du, dh.double(), a, ba, 1)
