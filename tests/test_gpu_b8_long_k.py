"""Products over a K of half a million and more: D in bf16 is the fp32 result rounded once, whatever K."""
import pytest
import torch

from gpu_case import sbl_mod

pytestmark = pytest.mark.gpu


def operand(sbl, rows, k, gen):
    """A stored [rows, k] matrix (the transpose of [k, rows]: a row may be longer than the quantiser's)."""
    d = sbl.b8_desc(rows, k)
    m = sbl.alloc_b8(d)
    sbl.sbl_b8_quantize(sbl.b8_desc(k, rows), torch.rand(k, rows, generator=gen, device="cuda").to(torch.bfloat16), None, m)
    return d, m


@pytest.mark.parametrize("m,n,k", [(80, 256, 600_000), (144, 528, 1_000_016)])
def test_bf16_result_of_a_very_long_k_is_the_fp32_one_rounded(m, n, k):
    sbl = sbl_mod()
    gen = torch.Generator(device="cuda").manual_seed(k)
    (ad, a), (bd, b) = operand(sbl, m, k, gen), operand(sbl, n, k, gen)
    want = torch.empty((m, n), dtype=torch.float32, device="cuda")
    got = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    sbl.sbl_b8_gemm(ad, a, bd, b, want)
    sbl.sbl_b8_gemm(ad, a, bd, b, got)
    # the fp32 sums of the positive products themselves: segments of 4096 in tensor memory (129 truncations),
    # K / 4096 rounded additions
    exact = torch.zeros((m, n), dtype=torch.float64, device="cuda")
    for at in range(0, k, 1 << 16):
        e = min(at + (1 << 16), k)
        exact += values(sbl, a, ad, at, e) @ values(sbl, b, bd, at, e).t()
    bound = (133 * 2.0 ** -23 + (k / 4096) * 2.0 ** -24) * exact
    assert bool(((want.double() - exact).abs() <= bound).all())
    assert torch.equal(got, want.to(torch.bfloat16))
    assert sbl.sbl_device_error() == 0


def values(sbl, m, d, at, e):
    """Columns at .. e (at a multiple of 128) of a stored e4m3 matrix in float64."""
    codes = m.codes[:, at:e].view(torch.float8_e4m3fn).double()
    rp = -(-d.rows // 128) * 128
    r = torch.arange(d.rows, device="cuda").view(-1, 1)
    j = torch.arange(at // 128, -(-e // 128), device="cuda").view(1, -1)
    byte = m.scales[4 * ((j // 4) * rp + 128 * (r // 128) + 4 * (r % 32) + (r % 128) // 32) + j % 4]
    return codes * torch.exp2(byte.double() - 127).repeat_interleave(128, 1)[:, :e - at]
