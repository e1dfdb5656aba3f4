"""The 8-bit block operators as a training step uses them together: RMSNorm
with a checkpoint, ternary gate / up, gated activation with checkpoints,
ternary down with the residual, an un-ternarised b8 head, and back.  Every
stage is compared with its definition in 64 bits on the values the stage
before it produced, so each tolerance is one operator's own; then the whole
step is captured in a graph, on another stream, and replayed on new inputs."""
import numpy as np
import pytest
import torch

import b8_ref as ref
from gpu_case import bf16_dev, sbl_mod, to_dev
from sparsity_sbl_quantize_b200 import workloads as wl

pytestmark = pytest.mark.gpu

T, K, F, V, EPS = 200, 256, 512, 272, 2.0 ** -16
ACT = 0  # silu


class Step:
    """Weights, buffers and the calls of one step."""

    def __init__(self, seed):
        self.sbl = sbl = sbl_mod()
        self.layers = {}
        for i, (name, o, k) in enumerate((("gate", F, K), ("up", F, K), ("down", K, F))):
            d = sbl.desc(o, k, 6, 8)
            p = sbl.alloc_packed(d, sbl.SBL_FMT_I8 | sbl.SBL_FMT_BF16T)
            w = to_dev(wl.master_weights(o, k, seed, i, std=0.1))
            ws = sbl.alloc_workspace(sbl.sbl_workspace_bytes(d, 0, sbl.SBL_OP_QUANTIZE_MASK_PACK))
            sbl.sbl_quantize_mask_pack(d, w, sbl.SBL_FMT_I8 | sbl.SBL_FMT_BF16T, p, ws)
            self.layers[name] = (d, p)
        r = np.random.Generator(np.random.PCG64(seed))
        self.head = torch.from_numpy((r.standard_normal((V, K)) * 0.05).astype(np.float32)).cuda()
        self.gain = torch.from_numpy((1 + 0.1 * r.standard_normal(K)).astype(np.float32)).to(torch.bfloat16).cuda()
        e = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
        f32, i8 = torch.float32, torch.int8
        self.x, self.dz = e(T, K), e(T, V)
        self.xq, self.xd, self.gu = e(T, K, dt=i8), e(T, dt=f32), e(T, 2 * F)
        self.h, self.hq, self.hd, self.y, self.z = e(T, F), e(T, F, dt=i8), e(T, dt=f32), e(T, K), e(T, V)
        self.g, self.u = e(T, F), e(T, F)
        self.nd, self.fd = sbl.b8_desc(T, K, sbl.SBL_B8_I8), sbl.b8_desc(T, F, sbl.SBL_B8_I8)
        self.x8, self.g8, self.u8 = sbl.alloc_b8(self.nd), sbl.alloc_b8(self.fd), sbl.alloc_b8(self.fd)
        self.wd = sbl.b8_desc(V, K)
        self.w8, self.w8t = sbl.alloc_b8(self.wd), sbl.alloc_b8(sbl.b8_desc(K, V))
        self.y8 = sbl.alloc_b8(sbl.b8_desc(T, K))
        self.dy, self.dh, self.dgu = e(T, K), e(T, F), e(T, 2 * F)
        self.dhead, self.dgain = e(V, K, dt=f32), e(K, dt=f32)
        self.dw = {n: e(d.out_features, d.in_features, dt=f32) for n, (d, _) in self.layers.items()}
        self.dn, self.dnu, self.dnb, self.dx = e(T, K, dt=f32), e(T, K, dt=f32), e(T, K), e(T, K)
        self.ws = sbl.alloc_workspace(max([sbl.sbl_workspace_bytes(d, T, sbl.SBL_OP_BACKWARD) for d, _ in self.layers.values()] +
                                          [sbl.sbl_b8_linear_workspace_bytes(self.wd, T), sbl.sbl_rmsnorm_backward_workspace_bytes(T, K)]))

    def set_inputs(self, seed):
        self.x.copy_(bf16_dev(wl.activations(T, K, seed, outlier_frac=0.02)))
        self.dz.copy_(bf16_dev(wl.output_grad(T, V, seed)))

    def run(self):
        s, L = self.sbl, self.layers
        s.sbl_b8_quantize(self.wd, self.head, self.w8, self.w8t, s.SBL_B8_TILES)
        s.sbl_quantize_act_rmsnorm_checkpoint(self.nd, self.x, self.gain, EPS, self.xq, self.xd, self.x8)
        s.sbl_forward_group([L["gate"][0], L["up"][0]], self.xq, self.xd, T, [L["gate"][1], L["up"][1]], [self.g, self.u])
        self.gu[:, :F].copy_(self.g)
        self.gu[:, F:].copy_(self.u)
        s.sbl_glu_forward(self.fd, ACT, self.gu[:, :F], self.gu[:, F:], self.h, self.g8, self.u8)
        s.sbl_quantize_act(self.h, T, F, self.hq, self.hd)
        s.sbl_forward_ex(L["down"][0], self.hq, self.hd, T, L["down"][1], s.SBL_FMT_I8, self.y, residual=self.x)
        s.sbl_b8_linear_forward(self.wd, self.w8, self.y, T, self.y8, self.z)
        # backward
        s.sbl_b8_linear_backward(self.wd, self.w8t, self.y8, self.dz, T, self.dy, self.dhead, self.ws)
        s.sbl_backward_dual_ste(L["down"][0], self.dy, self.hq, self.hd, T, L["down"][1], self.dh, False, self.dw["down"], self.ws)
        s.sbl_glu_backward(self.fd, ACT, self.g8, self.u8, self.dh, self.dgu[:, :F], self.dgu[:, F:])
        for n, half, out in (("gate", self.dgu[:, :F], self.dn), ("up", self.dgu[:, F:], self.dnu)):
            s.sbl_backward_dual_ste(L[n][0], half.contiguous(), self.xq, self.xd, T, L[n][1], out, True, self.dw[n], self.ws)
        self.dnb.copy_(self.dn + self.dnu)
        s.sbl_rmsnorm_backward(self.nd, self.x8, self.gain, EPS, self.dnb, self.dy, self.dx, self.dgain, self.ws)

    def results(self):
        return {"z": self.z, "y": self.y, "h": self.h, "dy": self.dy, "dh": self.dh, "dgu": self.dgu, "dx": self.dx, "dhead": self.dhead,
                "dgain": self.dgain, **{"dw_" + n: t for n, t in self.dw.items()}}


def d64(t):
    return t.double().cpu().numpy()


def close(got, want, half, slack=0.0):
    got = d64(got)
    tol = half * np.abs(want) + slack
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) - tol).max())


def sum_bound(a, b):
    """fp32 accumulation of a @ b.T as in test_gpu_b8.py."""
    return (-(-a.shape[1] // 32) + 5) * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T)


def test_training_step_stage_by_stage():
    st = Step(3)
    st.set_inputs(5)
    st.run()
    torch.cuda.synchronize()
    assert st.sbl.sbl_device_error() == 0
    x, dz, gain = d64(st.x), d64(st.dz), d64(st.gain)[None]
    # head forward and backward
    y = d64(st.y)
    w, y8 = ref.value(d64(st.head), ref.E4M3, True), ref.value(y, ref.E4M3)
    close(st.z, y8 @ w.T, 2.0 ** -8, 1.01 * sum_bound(y8, w))
    a = ref.value(dz, ref.E4M3)
    close(st.dy, a @ w, 2.0 ** -8, 1.01 * sum_bound(a, np.ascontiguousarray(w.T)))
    a, b = ref.value(np.ascontiguousarray(dz.T), ref.E4M3), ref.value(np.ascontiguousarray(y8.T), ref.E4M3)
    close(st.dhead, a @ b.T, 2.0 ** -24, 1.01 * sum_bound(a, b))
    # gated activation, from the bf16 gate and up forward, from their checkpoints backward
    g, u = d64(st.g), d64(st.u)
    act, _ = ref.act(g, ACT)
    close(st.h, act * u, 2.0 ** -8 + 2.0 ** -15, 2.0 ** -126)
    g8, u8, dh = ref.value(g, ref.I8), ref.value(u, ref.I8), d64(st.dh)
    act, da = ref.act(g8, ACT)
    sg = 1 / (1 + np.exp(-g8))
    close(st.dgu[:, :F], dh * u8 * da, 2.0 ** -8, 2.0 ** -14 * np.abs(dh * u8) * (np.abs(da) + sg * (1 + np.abs(g8))))
    close(st.dgu[:, F:], dh * act, 2.0 ** -8 + 2.0 ** -15, 2.0 ** -126)
    # norm backward at the checkpointed input, with the residual gradient
    x8, dn, dy = ref.value(x, ref.I8), d64(st.dnb), d64(st.dy)
    dx, dg = ref.rmsnorm_backward(x8, gain, EPS, dn, dy)
    r = 1 / np.sqrt((x8 * x8).mean(1, keepdims=True) + EPS)
    slack = 2.0 ** -24 * 180 * (np.abs(x8) * r ** 3 * (np.abs(dn * gain) * np.abs(x8)).mean(1, keepdims=True) + np.abs(r * dn * gain) + np.abs(dx))
    close(st.dx, dx, 2.0 ** -8, slack)
    close(st.dgain, dg, 0.0, 2.0 ** -24 * (T + 90) * np.abs(dn * x8 * r).sum(0))


def test_training_step_gradient_against_differences():
    """d loss / d x of the un-quantised function near the step's input: the step's gradient points along it.
    The quantisers (ternary weights are kept) move the gradient by their half steps: int8 activations and
    checkpoints 2^-7, e4m3 operands 2^-4 a value at most, with random signs over T K entries; the cosine of
    two vectors whose relative distance is r is at least sqrt(1 - r^2), and r = 3 * 2^-4 bounds the largest of
    them met three times (head, its backward, and all the smaller ones together)."""
    st = Step(7)
    st.set_inputs(8)
    st.run()
    x, dz, gain, head = d64(st.x), d64(st.dz), d64(st.gain)[None], d64(st.head)
    eff = {n: d64(p.i8.float()) * float(p.gamma[0]) for n, (_, p) in st.layers.items()}

    def loss(v):
        n = v / np.sqrt((v * v).mean(1, keepdims=True) + EPS) * gain
        g, u = n @ eff["gate"].T, n @ eff["up"].T
        y = v + (ref.act(g, ACT)[0] * u) @ eff["down"].T
        return (dz * (y @ head.T)).sum()

    got = d64(st.dx)
    r = np.random.Generator(np.random.PCG64(1))
    h, dirs = 1e-5, r.standard_normal((24, T, K))
    num = np.array([(loss(x + h * d) - loss(x - h * d)) / (2 * h) for d in dirs])
    ana = np.array([(got * d).sum() for d in dirs])
    cos = (num * ana).sum() / np.sqrt((num * num).sum() * (ana * ana).sum())
    assert cos >= np.sqrt(1 - (3 * 2.0 ** -4) ** 2), cos


def test_captured_on_another_stream_and_replayed():
    """Eager on the default stream, then captured on a side stream and replayed on two other inputs: the same bits."""
    st = Step(11)
    want = {}
    for seed in (1, 2):
        st.set_inputs(seed)
        st.run()
        torch.cuda.synchronize()
        want[seed] = {k: v.clone() for k, v in st.results().items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        st.run()  # first use on this stream before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        st.run()
    for seed in (2, 1, 2):
        st.set_inputs(seed)
        for v in st.results().values():
            v.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, v in st.results().items():
            assert torch.equal(v, want[seed][k]), k
    assert st.sbl.sbl_device_error() == 0


@pytest.mark.parametrize("t", [1, 40, 300])
def test_two_streams_at_once(t):
    """Two programs on two streams with the same weights and buffers of their own: what each gets alone."""
    sbl = sbl_mod()
    r = np.random.Generator(np.random.PCG64(t))
    o, k = 1040, 2064
    wd = sbl.b8_desc(o, k)
    w = sbl.alloc_b8(wd)
    sbl.sbl_b8_quantize(wd, torch.from_numpy(r.standard_normal((o, k)).astype(np.float32)).cuda(), w, None, sbl.SBL_B8_TILES)
    xs = [torch.from_numpy(r.standard_normal((t, k)).astype(np.float32)).to(torch.bfloat16).cuda() for _ in range(2)]
    xq = [sbl.alloc_b8(sbl.b8_desc(t, k)) for _ in range(2)]
    want = []
    for i in range(2):
        y = torch.empty((t, o), dtype=torch.bfloat16, device="cuda")
        sbl.sbl_b8_linear_forward(wd, w, xs[i], t, xq[i], y)
        want.append(y)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ys = [[torch.empty((t, o), dtype=torch.bfloat16, device="cuda") for _ in range(12)] for _ in range(2)]
    torch.cuda.synchronize()
    for j in range(12):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                sbl.sbl_b8_linear_forward(wd, w, xs[i], t, xq[i], ys[i][j])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in ys[i])
    assert sbl.sbl_device_error() == 0


def test_weights_quantised_right_before_the_product():
    """The product that follows a quantiser on the same stream sees its result: weights rewritten before every call."""
    sbl = sbl_mod()
    r = np.random.Generator(np.random.PCG64(9))
    o, k = 512, 1024
    wd = sbl.b8_desc(o, k)
    w = sbl.alloc_b8(wd)
    ws = [torch.from_numpy(r.standard_normal((o, k)).astype(np.float32)).cuda() for _ in range(6)]
    for t in (1, 20, 100, 400):
        x = torch.from_numpy(r.standard_normal((t, k)).astype(np.float32)).to(torch.bfloat16).cuda()
        xq = sbl.alloc_b8(sbl.b8_desc(t, k))
        alone = []
        for m in ws:
            sbl.sbl_b8_quantize(wd, m, w, None, sbl.SBL_B8_TILES)
            torch.cuda.synchronize()
            y = torch.empty((t, o), dtype=torch.bfloat16, device="cuda")
            sbl.sbl_b8_linear_forward(wd, w, x, t, xq, y)
            torch.cuda.synchronize()
            alone.append(y)
        run = [torch.empty_like(alone[0]) for _ in ws]
        torch.cuda.synchronize()
        for m, y in zip(ws, run):
            sbl.sbl_b8_quantize(wd, m, w, None, sbl.SBL_B8_TILES)
            sbl.sbl_b8_linear_forward(wd, w, x, t, xq, y)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(alone, run))


@pytest.mark.parametrize("op", ["quantize", "both", "transpose", "linear", "linear_backward", "glu", "glu_backward", "rmsnorm",
                                "rmsnorm_backward"])
def test_timing_command(op):
    import json
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "-m", "sparsity_sbl_quantize_b200.run_b8", op, "96", "256", "144", "--iters", "2", "--warmup", "1"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    line = json.loads(r.stdout)
    assert line["op"] == op and line["iters"] == 2 and line["ms_per_call"] > 0


@pytest.mark.parametrize("t,k,o", [(40, 512, 1040), (200, 1040, 272), (777, 1536, 1536), (2500, 2048, 1536)])
def test_backward_calls_back_to_back(t, k, o):
    """Calls that share weights and workspace, nothing waiting between them: each gets what it gets alone (the kernels of
    one call start beside one another, and those of the next behind them)."""
    sbl = sbl_mod()
    gen = torch.Generator(device="cuda").manual_seed(t)
    wd = sbl.b8_desc(o, k)
    w, wt = sbl.alloc_b8(wd), sbl.alloc_b8(sbl.b8_desc(k, o))
    sbl.sbl_b8_quantize(wd, torch.randn(o, k, generator=gen, device="cuda"), w, wt, sbl.SBL_B8_TILES)
    ws = sbl.alloc_workspace(sbl.sbl_b8_linear_workspace_bytes(wd, t))
    xs = [torch.randn(t, k, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(3)]
    dys = [torch.randn(t, o, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(3)]
    xq, y = sbl.alloc_b8(sbl.b8_desc(t, k)), torch.empty(t, o, dtype=torch.bfloat16, device="cuda")

    def call(i, dx, dw):
        sbl.sbl_b8_linear_forward(wd, w, xs[i], t, xq, y)
        sbl.sbl_b8_linear_backward(wd, wt, xq, dys[i], t, dx, dw, ws)

    def buffers():
        return torch.full((t, k), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((o, k), 7.0, device="cuda")

    want = []
    for i in range(3):
        b = buffers()
        torch.cuda.synchronize()
        call(i, *b)
        torch.cuda.synchronize()
        want.append(b)
    got = [buffers() for _ in range(24)]
    torch.cuda.synchronize()
    for j, b in enumerate(got):
        call(j % 3, *b)
    torch.cuda.synchronize()
    for j, b in enumerate(got):
        assert torch.equal(b[0], want[j % 3][0]) and torch.equal(b[1], want[j % 3][1]), j
    assert sbl.sbl_device_error() == 0
