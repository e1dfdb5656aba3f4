"""What the Python binding of the 8-bit block operators refuses before the library sees a pointer: tensors that the
C arguments cannot describe.  No device is needed, and none may be present: a call let through would hand host
pointers to kernels."""
import sys

import pytest
import torch

T, K, O = 4, 64, 32
BF, F32, I8 = torch.bfloat16, torch.float32, torch.int8


@pytest.fixture(scope="module")
def sbl():
    from sparsity_sbl_quantize_b200 import build
    build.build()
    from sparsity_sbl_quantize_b200 import sbl as m
    if torch.cuda.is_available():
        pytest.skip("a device is present: host pointers must not reach kernels")
    return m


@pytest.fixture
def placed(sbl, monkeypatch):
    """The host's tensors pass for tensors of device 0, the current one."""
    monkeypatch.setattr(sbl, "_device", lambda: 0)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)


def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def calls(sbl):
    """name -> (call taking its tensors, the tensors by name with their type)."""
    d, wd = sbl.b8_desc(T, K), sbl.b8_desc(O, K)
    m, w, wt = (sbl.alloc_b8(x, device="cpu") for x in (d, wd, sbl.b8_desc(K, O)))
    ws = z(1 << 20, dtype=torch.uint8)
    return {
        "quantize": (lambda X: sbl.sbl_b8_quantize(d, X, m), {"X": z(T, K)}),
        "dequantize": (lambda X: sbl.sbl_b8_dequantize(d, m, X), {"X": z(T, K)}),
        "gemm": (lambda D: sbl.sbl_b8_gemm(d, m, wd, w, D), {"D": z(T, O)}),
        "linear_forward": (lambda X, Y: sbl.sbl_b8_linear_forward(wd, w, X, T, m, Y), {"X": z(T, K), "Y": z(T, O)}),
        "linear_backward": (lambda dY, dX, dW: sbl.sbl_b8_linear_backward(wd, wt, m, dY, T, dX, dW, ws),
                            {"dY": z(T, O), "dX": z(T, K), "dW": z(O, K, dtype=F32)}),
        "glu_forward": (lambda G, U, H: sbl.sbl_glu_forward(d, 0, G, U, H, m, m), {"G": z(T, K), "U": z(T, K), "H": z(T, K)}),
        "glu_backward": (lambda dH, dG, dU: sbl.sbl_glu_backward(d, 0, m, m, dH, dG, dU),
                         {"dH": z(T, K), "dG": z(T, K), "dU": z(T, K)}),
        "rmsnorm_checkpoint": (lambda X, g, Xq, s: sbl.sbl_quantize_act_rmsnorm_checkpoint(d, X, g, 1e-5, Xq, s, m),
                               {"X": z(T, K), "g": z(K), "Xq": z(T, K, dtype=I8), "s": z(T, dtype=F32)}),
        "rmsnorm_backward": (lambda g, dU, dR, dX, dg: sbl.sbl_rmsnorm_backward(d, m, g, 1e-5, dU, dR, dX, dg, ws),
                             {"g": z(K), "dU": z(T, K), "dR": z(T, K), "dX": z(T, K), "dg": z(K, dtype=F32)}),
    }


EITHER = {("quantize", "X"), ("gemm", "D"), ("linear_forward", "Y"), ("linear_backward", "dX")}  # bf16 or fp32
ARGUMENTS = [(c, a) for c, names in (
    ("quantize", "X"), ("dequantize", "X"), ("gemm", "D"), ("linear_forward", "X Y"), ("linear_backward", "dY dX dW"),
    ("glu_forward", "G U H"), ("glu_backward", "dH dG dU"), ("rmsnorm_checkpoint", "X g Xq s"),
    ("rmsnorm_backward", "g dU dR dX dg")) for a in names.split()]


@pytest.mark.parametrize("call,name", ARGUMENTS)
def test_other_element_types_are_refused(sbl, placed, call, name):
    f, args = calls(sbl)[call]
    right = {BF, F32} if (call, name) in EITHER else {args[name].dtype}
    for dtype in (torch.float16, torch.float64, torch.int16, torch.uint8, BF, F32, I8):
        if dtype not in right:
            with pytest.raises(ValueError, match="tensor is needed"):
                f(**{**args, name: args[name].to(dtype)})


STRIDED = {("quantize", "X"), ("dequantize", "X"), ("gemm", "D"), ("linear_forward", "X"), ("linear_forward", "Y"), ("linear_backward", "dY"),
           ("glu_forward", "G"), ("glu_forward", "U"), ("glu_forward", "H"), ("glu_backward", "dH"), ("glu_backward", "dG"),
           ("glu_backward", "dU")}  # these have a row stride in the ABI


@pytest.mark.parametrize("call,name", [x for x in ARGUMENTS if x not in STRIDED])
def test_slices_of_wider_buffers_are_refused_where_there_is_no_stride(sbl, placed, call, name):
    f, args = calls(sbl)[call]
    t = args[name]
    wide = torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype)
    for bad in (wide[..., :t.shape[-1]], wide[..., ::2]):
        if bad.is_contiguous():
            continue  # the first half of a vector
        with pytest.raises(ValueError, match="contiguous"):
            f(**{**args, name: bad})


@pytest.mark.parametrize("call,name", sorted(STRIDED))
def test_rows_themselves_have_to_be_contiguous(sbl, placed, call, name):
    f, args = calls(sbl)[call]
    t = args[name]
    with pytest.raises(ValueError, match="contiguous rows"):
        f(**{**args, name: torch.zeros(t.shape[0], 2 * t.shape[1], dtype=t.dtype)[:, ::2]})


def test_workspaces_and_stored_matrices_are_contiguous(sbl, placed):
    d, wd = sbl.b8_desc(T, K), sbl.b8_desc(O, K)
    m = sbl.alloc_b8(d, device="cpu")
    gaps = torch.zeros(1 << 21, dtype=torch.uint8)[::2]
    with pytest.raises(ValueError, match="contiguous"):
        sbl.sbl_b8_linear_backward(wd, None, m, z(T, O), T, None, z(O, K, dtype=F32), gaps)
    with pytest.raises(ValueError, match="contiguous"):
        sbl.sbl_rmsnorm_backward(d, m, z(K), 1e-5, z(T, K), None, z(T, K), z(K, dtype=F32), gaps)
    for codes, scales in ((torch.zeros(T, 2 * K, dtype=torch.uint8)[:, :K], m.scales), (m.codes, gaps), (m.codes.short(), m.scales)):
        with pytest.raises(ValueError, match="contiguous tensors of bytes"):
            sbl.Block8(codes=codes, scales=scales)


@pytest.mark.parametrize("missing", ["_cuda_getDevice", "_cuda_getCurrentRawStream"])
def test_stream_without_torchs_private_names(sbl, monkeypatch, missing):
    """The binding loaded again where torch lacks one of them."""
    import importlib.util

    class Stream:
        cuda_stream = 0x5EED

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev: Stream if dev == 3 else None)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 3, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0x1000 + dev, raising=False)

    def load():
        spec = importlib.util.spec_from_file_location("sbl_again", sbl.__file__)
        m = importlib.util.module_from_spec(spec)
        monkeypatch.setitem(sys.modules, "sbl_again", m)
        spec.loader.exec_module(m)
        return m

    assert load()._stream() == 0x1003
    monkeypatch.delattr(torch._C, missing)
    assert load()._stream() == (0x1003 if missing == "_cuda_getDevice" else 0x5EED)


@pytest.mark.parametrize("call", sorted({c for c, _ in ARGUMENTS}))
def test_host_tensors_are_refused(sbl, call, monkeypatch):
    monkeypatch.setattr(sbl, "_device", lambda: 0)
    f, args = calls(sbl)[call]
    with pytest.raises(ValueError, match="device"):
        f(**args)


@pytest.mark.parametrize("call,name", ARGUMENTS)
def test_tensors_of_another_device_are_refused(sbl, call, name, monkeypatch):
    """Every tensor on device 0 but one: the calls that name it are refused, and only those reach the stream."""
    f, args = calls(sbl)[call]
    odd = args[name]

    class Reached(Exception):
        pass

    def stream(device):
        raise Reached

    monkeypatch.setattr(sbl, "_device", lambda: 0)
    monkeypatch.setattr(sbl, "_stream_of", stream)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 1 if self is odd else 0)
    with pytest.raises(ValueError, match="a tensor of device 1"):
        f(**args)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    with pytest.raises(Reached):
        f(**args)


def test_stored_matrices_of_another_device_are_refused(sbl, monkeypatch):
    d, wd = sbl.b8_desc(T, K), sbl.b8_desc(O, K)
    m, w, wt = (sbl.alloc_b8(x, device="cpu") for x in (d, wd, sbl.b8_desc(K, O)))
    with pytest.raises(ValueError, match="one device"):
        sbl.Block8(codes=m.codes, scales=m.scales.to("meta"))
    monkeypatch.setattr(sbl, "_device", lambda: 0)
    for odd in (m, w, wt):
        monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 1 if self is odd.codes else 0)
        with pytest.raises(ValueError, match="a tensor of device 1"):
            if odd is wt:
                sbl.sbl_b8_linear_backward(wd, wt, m, z(T, O), T, z(T, K), None, z(1 << 20))
            else:
                sbl.sbl_b8_linear_forward(wd, w, z(T, K), T, m, z(T, O))
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 1 if self is m.codes else 0)
    for f in (lambda: sbl.sbl_b8_transpose(d, w, m), lambda: sbl.sbl_b8_transpose(d, m, w), lambda: sbl.sbl_b8_dequantize(d, m, z(T, K)),
              lambda: sbl.sbl_b8_quantize(d, z(T, K), None, m), lambda: sbl.sbl_b8_gemm(d, m, wd, w, z(T, O)),
              lambda: sbl.sbl_glu_forward(d, 0, z(T, K), z(T, K), None, w, m), lambda: sbl.sbl_glu_backward(d, 0, w, m, z(T, K), z(T, K), z(T, K)),
              lambda: sbl.sbl_quantize_act_rmsnorm_checkpoint(d, z(T, K), None, 0.0, z(T, K, dtype=I8), z(T, dtype=F32), m),
              lambda: sbl.sbl_rmsnorm_backward(d, m, None, 0.0, z(T, K), None, z(T, K), None, None)):
        with pytest.raises(ValueError, match="a tensor of device 1"):
            f()
