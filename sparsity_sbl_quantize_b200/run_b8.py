"""Time the 8-bit block operators on the GPU.

    python -m sparsity_sbl_quantize_b200.run_b8 OP T K [O] [--type e4m3|e5m2|i8] [--act silu|relu2]
                                                [--iters 20] [--warmup 3]

OP: quantize (row blocks), both (row blocks and the transposed copy), transpose
(of a checkpoint), linear (the forward through W [O, K]), linear_backward, glu,
glu_backward (K = the MLP's width), rmsnorm (the quantiser with a checkpoint),
rmsnorm_backward.  Inputs are seeded activations X ~ N(0, 1) (the generator of
``workloads``).  Each of ``warmup + iters`` calls is timed with CUDA events on the
launching stream after an L2 flush by a 512 MiB write; one JSON line gives the
mean and the algorithmic rates (each input read once, each output written once;
2 T K O operations a product), against the measured HBM copy bandwidth and twice
the measured sustained bf16 rate when MEASURED_PEAKS.json is present.
"""
import argparse
import json
import os

import numpy as np
import torch

from . import sbl
from . import workloads as wl

TYPES = {"e4m3": sbl.SBL_B8_E4M3, "e5m2": sbl.SBL_B8_E5M2, "i8": sbl.SBL_B8_I8}
ACTS = {"silu": sbl.SBL_ACT_SILU, "relu2": sbl.SBL_ACT_RELU2}


def activations(T: int, K: int, seed: int) -> torch.Tensor:
    return torch.from_numpy(wl.activations(T, K, seed).view(np.int16)).view(torch.bfloat16).cuda()


def operator(op: str, T: int, K: int, O: int, typ: int, act: int):
    """(one call, its algorithmic bytes, its operations)"""
    d = sbl.b8_desc(T, K, typ)
    x = activations(T, K, 1)
    n = T * K

    def empty(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device="cuda")

    if op in ("quantize", "both", "transpose"):
        q, qt = sbl.alloc_b8(d), sbl.alloc_b8(sbl.b8_desc(K, T, typ))
        sbl.sbl_b8_quantize(d, x, q)
        if op == "transpose":
            return lambda: sbl.sbl_b8_transpose(d, q, qt), 2 * n, 0
        return lambda: sbl.sbl_b8_quantize(d, x, q, qt if op == "both" else None), (4 if op == "both" else 3) * n, 0
    if op in ("linear", "linear_backward"):
        wd = sbl.b8_desc(O, K, typ)
        w, wt, xq = sbl.alloc_b8(wd), sbl.alloc_b8(sbl.b8_desc(K, O, typ)), sbl.alloc_b8(d)
        sbl.sbl_b8_quantize(wd, torch.from_numpy(wl.master_weights(O, K, 1)).cuda(), w, wt, sbl.SBL_B8_TILES)
        y = empty(T, O)
        sbl.sbl_b8_linear_forward(wd, w, x, T, xq, y, x_type=typ)
        if op == "linear":
            return lambda: sbl.sbl_b8_linear_forward(wd, w, x, T, xq, y, x_type=typ), 3 * n + O * K + 2 * T * O, 2 * n * O
        dy, dx, dw = activations(T, O, 2), empty(T, K), empty(O, K, dtype=torch.float32)
        ws = sbl.alloc_workspace(sbl.sbl_b8_linear_workspace_bytes(wd, T))
        return (lambda: sbl.sbl_b8_linear_backward(wd, wt, xq, dy, T, dx, dw, ws, x_type=typ, g_type=typ),
                2 * T * O + n + O * K + 2 * n + 4 * O * K, 4 * n * O)
    if op in ("glu", "glu_backward"):
        u, h, dg, du = activations(T, K, 2), empty(T, K), empty(T, K), empty(T, K)
        g8, u8 = sbl.alloc_b8(d), sbl.alloc_b8(d)
        sbl.sbl_glu_forward(d, act, x, u, h, g8, u8)
        if op == "glu":
            return lambda: sbl.sbl_glu_forward(d, act, x, u, h, g8, u8), 8 * n, 0
        return lambda: sbl.sbl_glu_backward(d, act, g8, u8, h, dg, du), 8 * n, 0
    g = empty(K).fill_(1.0)
    xq, s, x8 = empty(T, K, dtype=torch.int8), empty(T, dtype=torch.float32), sbl.alloc_b8(d)
    sbl.sbl_quantize_act_rmsnorm_checkpoint(d, x, g, 1e-6, xq, s, x8)
    if op == "rmsnorm":
        return lambda: sbl.sbl_quantize_act_rmsnorm_checkpoint(d, x, g, 1e-6, xq, s, x8), 4 * n + 4 * T, 0
    du, dx, dgain = activations(T, K, 2), empty(T, K), empty(K, dtype=torch.float32)
    ws = sbl.alloc_workspace(sbl.sbl_rmsnorm_backward_workspace_bytes(T, K))
    return lambda: sbl.sbl_rmsnorm_backward(d, x8, g, 1e-6, du, x, dx, dgain, ws), 7 * n, 0


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("op", choices=["quantize", "both", "transpose", "linear", "linear_backward", "glu", "glu_backward",
                                   "rmsnorm", "rmsnorm_backward"])
    ap.add_argument("T", type=int)
    ap.add_argument("K", type=int)
    ap.add_argument("O", type=int, nargs="?", default=0)
    ap.add_argument("--type", choices=sorted(TYPES), default="e4m3")
    ap.add_argument("--act", choices=sorted(ACTS), default="silu")
    ap.add_argument("--iters", type=int, default=20)
    ap.add_argument("--warmup", type=int, default=3)
    args = ap.parse_args()
    if args.op.startswith("linear") and args.O < 16:
        ap.error("a linear needs O")
    call, nbytes, flops = operator(args.op, args.T, args.K, args.O, TYPES[args.type], ACTS[args.act])
    flush = torch.empty(512 << 20, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream()
    times = []
    for i in range(args.warmup + args.iters):
        flush.fill_(i & 0xFF)
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record(stream)
        call()
        e1.record(stream)
        e1.synchronize()
        if i >= args.warmup:
            times.append(e0.elapsed_time(e1))
    err = sbl.sbl_device_error(clear=True)
    if err:
        raise SystemExit(f"device error flag {err:#x}")
    ms = sum(times) / max(len(times), 1)
    line = {"op": args.op, "T": args.T, "K": args.K, "O": args.O or None, "type": args.type, "iters": len(times),
            "ms_per_call": round(ms, 5), "gbs": round(nbytes / (ms * 1e-3) / 1e9, 1)}
    if flops:
        line["tflops"] = round(flops / (ms * 1e-3) / 1e12, 1)
    peaks = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "MEASURED_PEAKS.json")
    if os.path.exists(peaks):
        with open(peaks) as f:
            p = json.load(f)
        if p.get("hbm_gbs"):
            line["frac_of_measured_hbm"] = round(line["gbs"] / p["hbm_gbs"], 3)
        if flops and p.get("bf16_tflops_sustained"):
            line["frac_of_twice_measured_bf16"] = round(line["tflops"] / (2 * p["bf16_tflops_sustained"]), 3)
    print(json.dumps(line), flush=True)


if __name__ == "__main__":
    main()
