"""The 8-bit block ("b8") operators: block-scaled linear layers, the gated activation and the RMSNorm with 8-bit
activation checkpoints. Cases, inputs, the plain form of each operator and its values in 64 bits.

A b8 matrix [R, C] holds 8-bit codes (e4m3, e5m2 or int8), rows padded with zeros to a multiple of 16 bytes, and one
power of two 2^e for every 128 codes of a row (or for a tile of 128 x 128), stored as the byte e + 127. Scale bytes lie
four blocks to a word; the words of 128 rows are contiguous, row r at 4 (r % 32) + r / 32; padding bytes are 127.
"""
import math

import torch

own = False

#: The largest code of a type as mantissa * 2^exponent with mantissa in [0.5, 1).
_TOP = {"e4m3": (0.875, 9), "e5m2": (0.875, 16), "i8": (127.0 / 128.0, 7)}
_TORCH = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2, "i8": torch.int8}


def listed():
    return [
        # one token through a BitNet-2B up projection: the weights' bytes and the launch are all there is
        {"name": "linear_t1_2560_6912", "kind": "linear", "T": 1, "K": 2560, "O": 6912, "type": "e4m3"},
        # a small ragged decode batch through the down projection: few rows, a long reduction
        {"name": "linear_t13_6912_2560", "kind": "linear", "T": 13, "K": 6912, "O": 2560, "type": "e4m3"},
        # a short prompt of odd length through a Qwen2.5-0.5B up projection
        {"name": "linear_t1000_896_4864", "kind": "linear", "T": 1000, "K": 896, "O": 4864, "type": "e4m3"},
        # the Qwen2.5-3B up projection of a training batch
        {"name": "linear_t16384_2048_11008", "kind": "linear", "T": 16384, "K": 2048, "O": 11008, "type": "e4m3"},
        # training steps of one linear (weights quantised anew, forward, both gradients): an odd length with gradients
        # in e5m2, and the Qwen2.5-3B down projection at full batch
        {"name": "train_t777_1536_1536_e5m2", "kind": "train", "T": 777, "K": 1536, "O": 1536, "type": "e4m3", "gtype": "e5m2"},
        {"name": "train_t16384_11008_2048", "kind": "train", "T": 16384, "K": 11008, "O": 2048, "type": "e4m3", "gtype": "e4m3"},
        # the gated activation between the MLP's linears with its checkpoint: a small batch, a full one
        {"name": "glu_fwd_t64_4864_relu2", "kind": "glu_fwd", "T": 64, "F": 4864, "act": "relu2", "type": "e4m3", "gated": True},
        {"name": "glu_fwd_t16384_11008_silu", "kind": "glu_fwd", "T": 16384, "F": 11008, "act": "silu", "type": "i8", "gated": True},
        # and its backward from the checkpoint: an odd length, a full batch
        {"name": "glu_bwd_t333_8960_relu2", "kind": "glu_bwd", "T": 333, "F": 8960, "act": "relu2", "type": "e4m3", "gated": True},
        {"name": "glu_bwd_t16384_11008_silu", "kind": "glu_bwd", "T": 16384, "F": 11008, "act": "silu", "type": "i8", "gated": True},
        # the norm before a block's first linear, forward with its checkpoint and backward: an odd length at the
        # Qwen2.5-0.5B width, a full batch at the 3B width
        {"name": "norm_t501_896", "kind": "norm", "T": 501, "K": 896, "type": "i8", "gains": True, "residual": False},
        {"name": "norm_t16384_2048", "kind": "norm", "T": 16384, "K": 2048, "type": "e4m3", "gains": True, "residual": True},
    ]


def _log(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(step, v // step * step)


def draw(rng):
    kind = rng.choice(["linear", "linear", "train", "glu_fwd", "glu_bwd", "norm"])
    act, typ = rng.choice(["silu", "relu2"]), rng.choice(["e4m3", "i8", "e5m2"])
    if kind in ("linear", "train"):
        c = {"kind": kind, "T": _log(rng, 1, 16384), "K": _log(rng, 64, 11008, 16), "O": _log(rng, 64, 11008, 16), "type": "e4m3"}
        while c["T"] * c["K"] * c["O"] > 16384 * 2048 * 11008:
            c["T"] = c["T"] // 2
        if kind == "train":
            c["gtype"] = rng.choice(["e4m3", "e5m2"])
        return c
    if kind == "norm":
        return {"kind": kind, "T": _log(rng, 1, 16384), "K": _log(rng, 64, 11008, 16), "type": typ,
                "gains": rng.random() < 0.8, "residual": rng.random() < 0.5}
    return {"kind": kind, "T": _log(rng, 1, 16384), "F": _log(rng, 64, 11008, 16), "act": act, "type": typ,
            "gated": rng.random() < 0.8}


# ------------------------------------------------------------------ the plain form

def _blocks(x, tile):
    """The largest magnitudes [R, ceil(C / 128)] of the 1 x 128 blocks (or 128 x 128 tiles) of x."""
    rows, cols = x.shape
    nb, nr = -(-cols // 128), -(-rows // 128)
    a = torch.nn.functional.pad(x.abs(), (0, nb * 128 - cols)).view(rows, nb, 128).amax(2)
    if tile:
        a = torch.nn.functional.pad(a, (0, 0, 0, nr * 128 - rows)).view(nr, 128, nb).amax(1)
        a = a.repeat_interleave(128, 0)[:rows]
    return a


def _exponents(a, typ):
    top, shift = _TOP[typ]
    m, x = torch.frexp(a)
    e = torch.where(m <= top, x - shift, x - shift + 1).clamp(min=-126)
    return torch.where(a == 0, torch.zeros_like(e), e)


def _spread(e, cols):
    return e.repeat_interleave(128, 1)[:, :cols]


def _quantize(x, typ, tile=False):
    """fp32 [R, C] -> (codes in the type, exponents)."""
    e = _exponents(_blocks(x, tile), typ)
    y = torch.ldexp(x, -_spread(e, x.shape[1]))
    return (y.round().to(torch.int8) if typ == "i8" else y.to(_TORCH[typ])), e


def _decode(codes, e):
    return torch.ldexp(codes.float(), _spread(e, codes.shape[1]))


def _pack_scales(e):
    """Exponents [R, B] -> the scale bytes in memory order."""
    r, b = e.shape
    rp, w = -(-r // 128) * 128, -(-b // 4)
    s = torch.full((rp, 4 * w), 127, dtype=torch.uint8, device=e.device)
    s[:r, :b] = (e + 127).to(torch.uint8)
    return s.view(rp // 128, 4, 32, w, 4).permute(3, 0, 2, 1, 4).contiguous().view(-1)


def _unpack_scales(s, r, b):
    rp, w = -(-r // 128) * 128, -(-b // 4)
    s = s.view(w, rp // 128, 32, 4, 4).permute(1, 3, 2, 0, 4).reshape(rp, 4 * w)
    return s[:r, :b].to(torch.int32) - 127


def _load(m):
    """The values of a stored b8 matrix (codes as bytes, scales in memory order) in fp32."""
    codes, cols = m["codes"].view(_TORCH[m["type"]]), m["cols"]
    return _decode(codes[:, :cols], _unpack_scales(m["scales"], codes.shape[0], -(-cols // 128)))


def _store(x, typ, tile=False):
    """fp32 [R, C], C a multiple of 16 -> a stored b8 matrix."""
    codes, e = _quantize(x, typ, tile)
    return {"codes": codes.view(torch.uint8).contiguous(), "scales": _pack_scales(e), "type": typ, "cols": x.shape[1]}


def _act(g, act):
    """The activation and its derivative."""
    if act == "relu2":
        p = torch.relu(g)
        return p * p, 2 * p
    s = 1 / (1 + torch.exp(-g))
    return g * s, s * (1 + g * (1 - s))


def _bf16(x):
    return x.to(torch.bfloat16)


def _plain(s):
    c = s["case"]
    kind = c["kind"]
    if kind == "linear":
        codes, e = _quantize(s["X"].float(), c["type"])
        return {"Y": _bf16(_decode(codes, e) @ _load(s["W"]).t()), "codes": codes, "scales": _pack_scales(e)}
    if kind == "train":
        W = _decode(*_quantize(s["W"], c["type"], True))
        X = _decode(*_quantize(s["X"].float(), c["type"]))
        dY = s["dY"].float()
        dYr, dYc = _decode(*_quantize(dY, c["gtype"])), _decode(*_quantize(dY.t().contiguous(), c["gtype"]))
        Xc = _decode(*_quantize(X.t().contiguous(), c["type"]))
        return {"Y": _bf16(X @ W.t()), "dX": _bf16(dYr @ W), "dW": dYc @ Xc.t()}
    if kind == "glu_fwd":
        g, out = s["G"].float(), {}
        h = _act(g, c["act"])[0]
        codes, e = _quantize(g, c["type"])
        out["g_codes"], out["g_scales"] = codes, _pack_scales(e)
        if c["gated"]:
            u = s["U"].float()
            h = h * u
            codes, e = _quantize(u, c["type"])
            out["u_codes"], out["u_scales"] = codes, _pack_scales(e)
        out["H"] = _bf16(h)
        return out
    if kind == "glu_bwd":
        a, da = _act(_load(s["G8"]), c["act"])
        dh = s["dH"].float()
        if not c["gated"]:
            return {"dG": _bf16(dh * da)}
        return {"dG": _bf16(dh * _load(s["U8"]) * da), "dU": _bf16(dh * a)}
    # norm: the int8 activations of the forward, the checkpoint, and the gradients from the checkpoint
    x, eps = s["X"].float(), s["eps"]
    g = s["gains"].float() if c["gains"] else torch.ones(c["K"], device=x.device)
    r = (1 / torch.sqrt(x.double().square().sum(1, keepdim=True) / c["K"] + eps)).float()
    u = x * r * g if c["gains"] else x * r
    amax = u.abs().amax(1, keepdim=True)
    q = torch.where(amax > 0, (u * (127 / amax)).round(), torch.zeros_like(u)).to(torch.int8)
    codes, e = _quantize(x, c["type"])
    x8, du = _decode(codes, e), s["dU"].float()
    r8 = 1 / torch.sqrt(x8.square().mean(1, keepdim=True) + eps)
    dx = r8 * (du * g) - x8 * (r8 * r8 * r8 * (du * g * x8).mean(1, keepdim=True))
    if c["residual"]:
        dx = dx + s["dR"].float()
    out = {"Xq": q, "d": amax[:, 0] / 127, "codes": codes, "scales": _pack_scales(e), "dX": _bf16(dx)}
    if c["gains"]:
        out["dgain"] = (du * x8 * r8).sum(0)
    return out


# ------------------------------------------------------------------ inputs, runs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _acts(g, t, k):
    """Activations: unit normal, one channel in a hundred twenty times as wide."""
    wide = 1 + 19 * (torch.rand(k, generator=g, device="cuda") < 0.01).float()
    return _bf16(_randn(g, t, k) * wide)


def _b8(sbl, rows, cols, typ):
    d = sbl.b8_desc(rows, cols, {"e4m3": sbl.SBL_B8_E4M3, "e5m2": sbl.SBL_B8_E5M2, "i8": sbl.SBL_B8_I8}[typ])
    return d, sbl.alloc_b8(d)


def prepare(case, seed):
    g, c = _gen(seed), case
    s = {"case": c, "eps": 1e-5}
    T, kind = c["T"], c["kind"]
    if kind in ("linear", "train"):
        s["X"] = _acts(g, T, c["K"])
        W = _randn(g, c["O"], c["K"]) * 0.02
        # a serving program keeps the weights in 8 bits; a training one their fp32 master
        s["W"] = _store(W, c["type"], True) if kind == "linear" else W
        if kind == "train":
            s["dY"] = _bf16(_randn(g, T, c["O"]) * 1e-3 * torch.exp(_randn(g, T, 1)))
    elif kind == "norm":
        s["X"], s["dU"] = _acts(g, T, c["K"]), _bf16(_randn(g, T, c["K"]) * 1e-3)
        s["gains"] = _bf16(1 + 0.1 * _randn(g, c["K"])) if c["gains"] else None
        s["dR"] = _bf16(_randn(g, T, c["K"]) * 1e-3) if c["residual"] else None
    else:
        G, U = _acts(g, T, c["F"]), _acts(g, T, c["F"]) if c["gated"] else None
        if kind == "glu_fwd":
            s["G"], s["U"] = G, U
        else:
            s["G8"], s["U8"] = _store(G.float(), c["type"]), _store(U.float(), c["type"]) if c["gated"] else None
            s["dH"] = _bf16(_randn(g, T, c["F"]) * 1e-3)
    s["kept"] = {}
    return s


def _buffers(s):
    """The outputs, workspaces and descriptors that a program allocates once and keeps."""
    from sparsity_sbl_quantize_b200 import sbl
    c, k = s["case"], s["kept"]
    if k:
        return sbl, k
    T, kind = c["T"], c["kind"]

    def empty(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device="cuda")

    def stored(m):
        d, b = _b8(sbl, m["codes"].shape[0], m["cols"], m["type"])
        return d, sbl.Block8(codes=m["codes"], scales=m["scales"])

    if kind == "linear":
        k["x"] = _b8(sbl, T, c["K"], c["type"])
        k["w"] = stored(s["W"])
        k["Y"] = empty(T, c["O"])
    elif kind == "train":
        k["x"], k["w"], k["wt"] = (_b8(sbl, *n, c["type"]) for n in ((T, c["K"]), (c["O"], c["K"]), (c["K"], c["O"])))
        k["gt"] = {"e4m3": sbl.SBL_B8_E4M3, "e5m2": sbl.SBL_B8_E5M2}[c["gtype"]]
        k["Y"], k["dX"], k["dW"] = empty(T, c["O"]), empty(T, c["K"]), empty(c["O"], c["K"], dtype=torch.float32)
        k["ws"] = sbl.alloc_workspace(sbl.sbl_b8_linear_workspace_bytes(k["w"][0], T))
    elif kind == "glu_fwd":
        k["g"], k["u"] = _b8(sbl, T, c["F"], c["type"]), _b8(sbl, T, c["F"], c["type"]) if c["gated"] else (None, None)
        k["H"] = empty(T, c["F"])
    elif kind == "glu_bwd":
        k["g"], k["u"] = stored(s["G8"]), stored(s["U8"]) if c["gated"] else (None, None)
        k["dG"], k["dU"] = empty(T, c["F"]), empty(T, c["F"]) if c["gated"] else None
    else:
        k["x"] = _b8(sbl, T, c["K"], c["type"])
        k["Xq"], k["d"], k["dX"] = empty(T, c["K"], dtype=torch.int8), empty(T, dtype=torch.float32), empty(T, c["K"])
        k["dgain"] = empty(c["K"], dtype=torch.float32) if c["gains"] else None
        k["ws"] = sbl.alloc_workspace(sbl.sbl_rmsnorm_backward_workspace_bytes(T, c["K"]))
    k["act"] = {"silu": sbl.SBL_ACT_SILU, "relu2": sbl.SBL_ACT_RELU2}.get(c.get("act"))
    return sbl, k


def _library(s):
    sbl, k = _buffers(s)
    c, view = s["case"], _TORCH[s["case"]["type"]]
    kind = c["kind"]
    if kind == "linear":
        (wd, w), (_, x) = k["w"], k["x"]
        sbl.sbl_b8_linear_forward(wd, w, s["X"], c["T"], x, k["Y"])
        return {"Y": k["Y"], "codes": x.codes.view(view), "scales": x.scales}
    if kind == "train":
        (wd, w), (_, wt), (_, x) = k["w"], k["wt"], k["x"]
        sbl.sbl_b8_quantize(wd, s["W"], w, wt, blocks=sbl.SBL_B8_TILES)
        sbl.sbl_b8_linear_forward(wd, w, s["X"], c["T"], x, k["Y"])
        sbl.sbl_b8_linear_backward(wd, wt, x, s["dY"], c["T"], k["dX"], k["dW"], k["ws"], g_type=k["gt"])
        return {"Y": k["Y"], "dX": k["dX"], "dW": k["dW"]}
    if kind == "glu_fwd":
        (gd, g), (_, u) = k["g"], k["u"]
        sbl.sbl_glu_forward(gd, k["act"], s["G"], s["U"], k["H"], g, u)
        out = {"H": k["H"], "g_codes": g.codes.view(view), "g_scales": g.scales}
        if c["gated"]:
            out |= {"u_codes": u.codes.view(view), "u_scales": u.scales}
        return out
    if kind == "glu_bwd":
        (gd, g), (_, u) = k["g"], k["u"]
        sbl.sbl_glu_backward(gd, k["act"], g, u, s["dH"], k["dG"], k["dU"])
        return {"dG": k["dG"], "dU": k["dU"]} if c["gated"] else {"dG": k["dG"]}
    xd, x = k["x"]
    sbl.sbl_quantize_act_rmsnorm_checkpoint(xd, s["X"], s["gains"], s["eps"], k["Xq"], k["d"], x)
    sbl.sbl_rmsnorm_backward(xd, x, s["gains"], s["eps"], s["dU"], s["dR"], k["dX"], k["dgain"], k["ws"])
    out = {"Xq": k["Xq"], "d": k["d"], "codes": x.codes.view(view), "scales": x.scales, "dX": k["dX"]}
    if c["gains"]:
        out["dgain"] = k["dgain"]
    return out


def run(state):
    return _library(state) if own else _plain(state)


def work(case):
    c, T = case, case["T"]
    if c["kind"] == "linear":
        K, O = c["K"], c["O"]
        return {"bytes": 2 * T * K + T * K + O * K + 2 * T * O + (T * K + O * K) / 128, "flops": 2 * T * K * O}
    if c["kind"] == "train":
        K, O = c["K"], c["O"]
        return {"bytes": 4 * O * K + 2 * T * K + 2 * T * O + 2 * T * O + 2 * T * K + 4 * O * K, "flops": 6 * T * K * O}
    if c["kind"] == "norm":
        n = T * c["K"]
        return {"bytes": n * (2 + 1 + 1 + 2 + 2 + (2 if c["residual"] else 0)) + 4 * T, "flops": 20 * n}
    n = T * c["F"]
    per = 8 if c["gated"] else 5
    return {"bytes": n * per + n * (2 if c["gated"] else 1) / 128, "flops": 12 * n}


# ------------------------------------------------------------------ values in 64 bits

def _grid64(x, typ, tile=False):
    """x (64-bit) rounded to the b8 grid: (codes, exponents), each code as its value."""
    largest = {"e4m3": 448.0, "e5m2": 57344.0, "i8": 127.0}[typ]
    bits, lowest = {"e4m3": (3, -6), "e5m2": (2, -14), "i8": (0, 0)}[typ]
    rows, cols = x.shape
    e = torch.empty(rows, -(-cols // 128), dtype=torch.float64, device=x.device)
    for j in range(e.shape[1]):
        a = x[:, 128 * j:128 * (j + 1)].abs().amax(1)
        if tile:
            a = torch.cat([p.amax().expand(p.numel()) for p in a.split(128)])
        f = torch.ceil(torch.log2(a / largest))
        f = torch.where(a > largest * torch.exp2(f), f + 1, f)
        f = torch.where(a <= largest * torch.exp2(f - 1), f - 1, f)
        e[:, j] = torch.where(a > 0, f.clamp(min=-126.0), torch.zeros_like(f))
    y = x / torch.exp2(e.repeat_interleave(128, 1)[:, :cols])
    if typ == "i8":
        return torch.round(y), e
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** lowest))) - bits)
    return torch.round(y / step) * step, e


def _value64(codes, e):
    return codes * torch.exp2(e.repeat_interleave(128, 1)[:, :codes.shape[1]])


def _kept64(m):
    rows, cols = m["codes"].shape[0], m["cols"]
    nb = -(-cols // 128)
    rp = -(-rows // 128) * 128
    r = torch.arange(rows, device="cuda").view(-1, 1)
    j = torch.arange(nb, device="cuda").view(1, -1)
    at = 4 * ((j // 4) * rp + 128 * (r // 128) + 4 * (r % 32) + (r % 128) // 32) + j % 4
    return _value64(m["codes"].view(_TORCH[m["type"]])[:, :cols].double(), m["scales"][at].double() - 127)


def _bytes64(e):
    rows, nb = e.shape
    rp = -(-rows // 128) * 128
    out = torch.full((rp * -(-nb // 4) * 4,), 127, dtype=torch.uint8, device="cuda")
    r = torch.arange(rows, device="cuda").view(-1, 1)
    j = torch.arange(nb, device="cuda").view(1, -1)
    out[4 * ((j // 4) * rp + 128 * (r // 128) + 4 * (r % 32) + (r % 128) // 32) + j % 4] = (e + 127).to(torch.uint8)
    return out


def _silu64(g):
    p = torch.special.expit(g)
    return g * p, p + g * p * torch.special.expit(-g)


def exact(case, seed):
    s, c = prepare(case, seed), case
    kind = c["kind"]
    if kind == "linear":
        q, e = _grid64(s["X"].double(), c["type"])
        return {"Y": _value64(q, e) @ _kept64(s["W"]).t(), "codes": q, "scales": _bytes64(e)}
    if kind == "train":
        W = _value64(*_grid64(s["W"].double(), c["type"], True))
        X = _value64(*_grid64(s["X"].double(), c["type"]))
        Y = X @ W.t()
        dX = _value64(*_grid64(s["dY"].double(), c["gtype"])) @ W
        del W
        dY = _value64(*_grid64(s["dY"].double().t().contiguous(), c["gtype"]))
        return {"Y": Y, "dX": dX, "dW": dY @ _value64(*_grid64(X.t().contiguous(), c["type"])).t()}
    if kind in ("glu_fwd", "glu_bwd"):
        g = s["G"].double() if kind == "glu_fwd" else _kept64(s["G8"])
        if c["act"] == "relu2":
            a, da = g.clamp(min=0).square(), 2 * g.clamp(min=0)
        else:
            a, da = _silu64(g)
        if kind == "glu_bwd":
            dh = s["dH"].double()
            return {"dG": dh * da * _kept64(s["U8"]), "dU": dh * a} if c["gated"] else {"dG": dh * da}
        q, e = _grid64(g, c["type"])
        out = {"H": a * s["U"].double() if c["gated"] else a, "g_codes": q, "g_scales": _bytes64(e)}
        if c["gated"]:
            q, e = _grid64(s["U"].double(), c["type"])
            out |= {"u_codes": q, "u_scales": _bytes64(e)}
        return out
    x, du, K, eps = s["X"].double(), s["dU"].double(), c["K"], s["eps"]
    gain = s["gains"].double() if c["gains"] else torch.ones(K, dtype=torch.float64, device=x.device)
    top = (x * gain).abs().amax(1) / torch.sqrt(x.square().sum(1) / K + eps)
    q, e = _grid64(x, c["type"])
    x8 = _value64(q, e)
    inv = 1 / torch.sqrt(x8.square().sum(1, keepdim=True) / K + eps)
    n = x8 * inv
    v = du * gain
    dx = inv * (v - n * (v * n).sum(1, keepdim=True) / K)
    if c["residual"]:
        dx = dx + s["dR"].double()
    # the int8 activations are defined by their roundings to 32 bits: no value of their own in 64
    out = {"Xq": None, "d": top / 127, "codes": q, "scales": _bytes64(e), "dX": dx}
    if c["gains"]:
        out["dgain"] = (du * n).sum(0)
    return out
