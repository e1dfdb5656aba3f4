"""The b8 format's definitions in float64 with torch (tests/b8_ref.py for sizes where numpy's loops take too long), and
which kernel a product takes, read from the library's source."""
from __future__ import annotations

import os
import re

import torch

import b8_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def quantize(x, typ):
    """x float64 [R, C], finite -> (values of the codes [R, C], exponents [R, B]) in row blocks."""
    r, c = x.shape
    b = -(-c // 128)
    a = torch.nn.functional.pad(x.abs(), (0, 128 * b - c)).view(r, b, 128).amax(2)
    top = ref.MAX[typ]
    e = torch.full_like(a, -126.0)
    for _ in range(260):  # the smallest e >= -126 with a <= MAX 2^e
        e = torch.where(a > top * torch.exp2(e), e + 1, e)
    e = torch.where(a == 0, torch.zeros_like(e), e)
    y = x * torch.exp2(-e).repeat_interleave(128, 1)[:, :c]
    if typ == ref.I8:
        return torch.round(y), e
    _, p = torch.frexp(torch.where(y == 0, torch.ones_like(y), y.abs()))
    step = torch.exp2((p.double() - 1).clamp(min=ref.EMIN[typ]) - ref.MANT[typ])
    return torch.round(y / step) * step, e


def decode(y, e):
    return y * torch.exp2(e).repeat_interleave(128, 1)[:, :y.shape[1]]


def code_values(m, d):
    """The codes of a stored matrix as float64 values [rows, cols]."""
    t = {ref.E4M3: torch.float8_e4m3fn, ref.E5M2: torch.float8_e5m2, ref.I8: torch.int8}[d.type]
    return m.codes[:, :d.cols].view(t).double()


def exponents(m, d):
    """The exponents [rows, blocks] of a stored matrix (its scale bytes less 127)."""
    rows, blocks = d.rows, -(-d.cols // 128)
    rp = -(-rows // 128) * 128
    r = torch.arange(rows, device=m.scales.device).view(-1, 1)
    j = torch.arange(blocks, device=m.scales.device).view(1, -1)
    return m.scales[4 * ((j // 4) * rp + 128 * (r // 128) + 4 * (r % 32) + (r % 128) // 32) + j % 4].double() - 127


def stored(m, d):
    return decode(code_values(m, d), exponents(m, d))


# ------------------------------------------------- which kernel a product takes

def _source(name):
    with open(os.path.join(ROOT, "sparsity_sbl_quantize_b200", "csrc", name)) as f:
        return f.read()


def _constant(text, name):
    return int(re.search(rf"constexpr int {name} = (\d+);", text).group(1))


def product_kernel(m, n, k, fp32, sms=148):
    """("few rows",) or ("tiles", BN, LONG, most tiles of a CTA) for D [m, n] with m above 128 rows or few tiles: the cost rule and
    the segment lengths as the library's source states them."""
    api, gemm = _source("sbl_b8_api.cu"), _source("sbl_b8_gemm.cuh")
    seg, longest = _constant(gemm, "kB8SegBlocks"), _constant(gemm, "kB8MaxBf16Blocks")
    few = re.search(r"if \(args\.M <= (\d+) \|\| \(args\.M <= (\d+) && (\d+) \* tiles_w <= hd\.num_sms\)\)", api)
    if m <= int(few.group(1)) or (m <= int(few.group(2)) and int(few.group(3)) * -(-n // 128) <= sms):
        return ("few rows",)
    rule = re.search(r"const bool wide = (\d+) \+ rounds\(256\) \* \((\d+)ll \* args\.k_blocks \+ (\d+)\) <= "
                     r"(\d+) \+ rounds\(128\) \* \((\d+)ll \* args\.k_blocks \+ (\d+)\);", api)
    a, b, c, d, e, f = map(int, rule.groups())
    assert re.search(r"const bool lng = args\.k_blocks > \(fp32 \? kB8SegBlocks : kB8MaxBf16Blocks\);", api)
    kb = -(-k // 128)
    tiles = {bn: -(-m // 128) * -(-n // bn) for bn in (128, 256)}
    rounds = {bn: -(-t // sms) for bn, t in tiles.items()}
    bn = 256 if a + rounds[256] * (b * kb + c) <= d + rounds[128] * (e * kb + f) else 128
    return "tiles", bn, kb > (seg if fp32 else longest), rounds[bn]
