"""What the MXFP4 calls and the block norm refuse, on the host and before
anything is enqueued: no GPU is needed, the addresses are never read."""
import ctypes

import pytest
import torch

import nvfp4_razer_w4a16_amd as rz
from nvfp4_razer_w4a16_amd.mx import razer_mx, razer_norm

X, Y, WS = 0x40000, 0x50000, 0x60000
INVALID, UNSUPPORTED, OK = rz.RAZER_E_INVALID, rz.RAZER_E_UNSUPPORTED, rz.RAZER_OK


def _mx(rows=4, cols=64, codes=0x10000, scales=0x20000):
    return razer_mx(rows, cols, codes, scales)


def test_struct_layouts_match_the_header():
    assert ctypes.sizeof(razer_mx) == 32
    assert ctypes.sizeof(razer_norm) == 15 * 8 and razer_norm.residual_scale.offset == 11 * 8
    assert razer_norm.flags.offset == 20 and razer_norm.packed.offset == 14 * 8


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(cols=48)),
    (INVALID, dict(rows=-1)),
    (INVALID, dict(rows=1 << 62)),
    (INVALID, dict(codes=0)),
    (INVALID, dict(scales=0)),
    (INVALID, dict(codes=0x10008)),
    (INVALID, dict(dt=3)),
    (INVALID, dict(x=0)),
    (INVALID, dict(x=X + 8)),
    (INVALID, dict(stride=32)),            # shorter than a row
    (INVALID, dict(stride=130)),           # rows not on 16 bytes
    (INVALID, dict(out=None)),
    (UNSUPPORTED, dict(rows=(1 << 28) + 1)),
    (OK, dict(rows=0, codes=0, scales=0, x=0)),
])
@pytest.mark.parametrize("gated", [False, True])
def test_encoders_refuse(want, kw, gated):
    a = dict(rows=4, cols=64, codes=0x10000, scales=0x20000, dt=rz.RAZER_BF16, x=X, stride=128)
    a.update(kw)
    t = _mx(a["rows"], a["cols"], a["codes"], a["scales"])
    L = rz.lib()
    f = L.razer_mx_quantize_gated if gated else L.razer_mx_quantize
    assert f(a["x"], a["dt"], a["stride"], None if "out" in kw else ctypes.byref(t), None) == want


def test_gated_rows_hold_both_halves():
    t = _mx()
    assert rz.lib().razer_mx_quantize_gated(X, rz.RAZER_F16, 64, ctypes.byref(t), None) == INVALID


@pytest.mark.parametrize("want,t,out,dt", [
    (INVALID, dict(cols=16), Y, 0), (INVALID, dict(codes=0), Y, 0), (INVALID, {}, 0, 0), (INVALID, {}, Y + 4, 0),
    (INVALID, {}, Y, 5), (UNSUPPORTED, dict(rows=1 << 29), Y, 0), (OK, dict(cols=0), 0, 0)])
def test_decoder_refuses(want, t, out, dt):
    s = _mx(**t)
    assert rz.lib().razer_mx_dequant(ctypes.byref(s), out, dt, None) == want


@pytest.mark.parametrize("want,x,w,kw", [
    (INVALID, dict(cols=96), {}, {}),
    (INVALID, dict(codes=0), {}, {}),
    (INVALID, {}, dict(rows=-2), {}),
    (INVALID, {}, {}, dict(y=0)),
    (INVALID, {}, {}, dict(y=Y + 2)),
    (INVALID, {}, {}, dict(dt=7)),
    (UNSUPPORTED, dict(cols=0), dict(cols=0), {}),
    (UNSUPPORTED, {}, dict(rows=(1 << 30) + 1), {}),
    (OK, dict(rows=0), {}, dict(y=0)),
    (OK, {}, dict(rows=0), dict(y=0)),
])
def test_product_refuses(want, x, w, kw):
    a = dict(y=Y, dt=rz.RAZER_F32)
    a.update(kw)
    sx, sw = _mx(**x), _mx(**w)
    L = rz.lib()
    assert L.razer_mx_gemm(ctypes.byref(sx), ctypes.byref(sw), a["y"], a["dt"], WS, 1 << 40, None) == want
    if want == INVALID:
        assert L.razer_mx_gemm(None, ctypes.byref(sw), Y, 0, WS, 1 << 40, None) == INVALID


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(experts=0)),
    (INVALID, dict(experts=3)),                       # 4 weight rows
    (INVALID, dict(experts=rz.RAZER_MX_MAX_EXPERTS * 2, wrows=rz.RAZER_MX_MAX_EXPERTS * 2)),
    (INVALID, dict(off=0)),
    (INVALID, dict(off=0x70002)),
    (INVALID, dict(rows=0x80001)),
    (INVALID, dict(rows=0, m=5)),                     # without row numbers M is x's
    (INVALID, dict(m=-1)),
    (INVALID, dict(xrows=0)),                         # row numbers of no rows
    (INVALID, dict(y=0)),
    (INVALID, dict(y=Y + 4)),
    (UNSUPPORTED, dict(m=(1 << 30) + 1)),
    (OK, dict(m=0)),
    (OK, dict(wrows=0)),
])
def test_grouped_refuses(want, kw):
    a = dict(experts=2, off=0x70000, rows=0x80000, m=6, y=Y, xrows=4, wrows=4)
    a.update(kw)
    sx, sw = _mx(rows=a["xrows"]), _mx(rows=a["wrows"])
    assert rz.lib().razer_mx_gemm_grouped(ctypes.byref(sx), ctypes.byref(sw), a["off"], a["experts"], a["rows"], a["m"],
                                          a["y"], rz.RAZER_BF16, WS, 1 << 40, None) == want


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(cols=40)), (INVALID, dict(rows=-1)), (INVALID, dict(dtype=4)), (INVALID, dict(flags=2)),
    (INVALID, dict(h=0)), (INVALID, dict(h=X + 8)), (INVALID, dict(h_stride=32)), (INVALID, dict(h_stride=65)),
    (INVALID, dict(y=X + 4)), (INVALID, dict(y_stride=8)), (INVALID, dict(y=0)),       # a norm of no y
    (INVALID, dict(y=0, flags=0, gate=X, gate_rows=1)),
    (INVALID, dict(gate=X, gate_rows=3)), (INVALID, dict(gate=X, gate_rows=0)), (INVALID, dict(gate=X + 2, gate_rows=1)),
    (INVALID, dict(post_weight=X + 8)), (INVALID, dict(pre_weight=X + 8)),
    (INVALID, dict(h_out=0, x_out=0)), (INVALID, dict(h_out=Y + 8)), (INVALID, dict(x_out=Y + 8)),
    (INVALID, dict(packed=(4, 32))), (INVALID, dict(packed=(3, 64))),
    (UNSUPPORTED, dict(cols=32800, y_stride=32800, h_stride=32800)),
    (OK, dict(rows=0, h=0, y=0, h_out=0, x_out=0)),
])
def test_block_norm_refuses(want, kw):
    a = razer_norm(rows=4, cols=64, dtype=rz.RAZER_BF16, flags=rz.RAZER_NORM_POST, y=X, h=X, y_stride=64, h_stride=64,
                   residual_scale=1.0, eps=1e-5, h_out=Y, x_out=Y)
    for k, v in kw.items():
        if k == "packed":
            t = _mx(*v)
            a.packed = ctypes.pointer(t)
        else:
            setattr(a, k, v)
    assert rz.lib().razer_block_norm(ctypes.byref(a), None) == want
    assert rz.lib().razer_block_norm(None, None) == INVALID


def test_workspace_bytes():
    for a in ((0, 8, 64, 0), (8, 0, 64, 0), (8, 8, 0, 2), (-1, 8, 64, 0), (8, 8, 64, -1)):
        assert rz.razer_mx_workspace_bytes(*a) == 0


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    t = rz.MxTensor(4, 64, "cpu")
    x = torch.zeros(4, 64)
    for call in (lambda: rz.razer_mx_quantize(x), lambda: rz.razer_mx_quantize_gated(x), lambda: rz.razer_mx_dequant(t),
                 lambda: rz.razer_mx_gemm(t, t), lambda: rz.razer_block_norm(x, x),
                 lambda: rz.razer_mx_gemm_grouped(t, t, torch.zeros(3, dtype=torch.int32))):
        with pytest.raises(ValueError, match="must be on a GPU"):
            call()
    with pytest.raises(ValueError, match="multiple of 32"):
        rz.MxTensor(4, 48, "cpu")
    with pytest.raises(ValueError, match="no contiguous uint8"):
        rz.MxTensor.of(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 3, dtype=torch.uint8))
    t.codes = torch.zeros(4, 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="no contiguous uint8"):
        t.check()
    with pytest.raises(TypeError, match="MxTensor"):
        rz.razer_mx_gemm(x, t)


@pytest.mark.gpu
def test_binding_refuses_before_it_writes():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bf = torch.bfloat16
    w, x = rz.razer_mx_quantize(torch.ones(6, 64, device="cuda")), rz.razer_mx_quantize(torch.ones(4, 64, device="cuda"))
    k = rz.razer_mx_quantize(torch.ones(6, 96, device="cuda"))
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    h = torch.ones(4, 64, dtype=bf, device="cuda")
    out = torch.full((4, 6), 7.0, device="cuda")
    for call in (lambda: rz.razer_mx_gemm(x, k), lambda: rz.razer_mx_gemm(x, w, out=out[:3]),
                 lambda: rz.razer_mx_gemm(x, w, out=out.t()), lambda: rz.razer_mx_gemm_grouped(x, w, off.long()),
                 lambda: rz.razer_mx_gemm_grouped(x, w, off[:0]), lambda: rz.razer_mx_gemm_grouped(x, w, off.cpu()),
                 lambda: rz.razer_mx_gemm_grouped(x, k, off), lambda: rz.razer_mx_quantize(h, out=w),
                 lambda: rz.razer_mx_quantize(h[:, :40]), lambda: rz.razer_mx_quantize_gated(h[:, :32]),
                 lambda: rz.razer_mx_dequant(x, out=out), lambda: rz.razer_block_norm(h[:2], h),
                 lambda: rz.razer_block_norm(h.float(), h), lambda: rz.razer_block_norm(h, h, gate=h[:, :32]),
                 lambda: rz.razer_block_norm(None, h, post_weight=h[0]), lambda: rz.razer_block_norm(h, h, x_out=out),
                 lambda: rz.razer_block_norm(h, h, pre_weight=h[0].float())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(rz.RazerError):  # three gates for four rows
        rz.razer_block_norm(h, h, gate=h[:3])
    for bad in (torch.float64, torch.int32):
        with pytest.raises(TypeError):
            rz.razer_mx_quantize(h.to(bad))
    torch.cuda.synchronize()
    assert (out == 7.0).all()


def test_workspace_bytes_of_refused_sizes():
    for a in ((2 ** 30 + 1, 8, 64, 0), (8, 2 ** 62, 64, 0), (8, 8, 2 ** 23 + 32, 0), (8, 8, 64, rz.RAZER_MX_MAX_EXPERTS + 1),
              (2 ** 63 - 1, 2 ** 63 - 1, 2 ** 63 - 1, 2 ** 63 - 1)):
        assert rz.razer_mx_workspace_bytes(*a) == 0
    for a in ((2 ** 30, 2 ** 30, 2 ** 23, 0), (2 ** 30, 2 ** 30, 2 ** 23, 4096), (1, 2 ** 30, 32, 0)):
        assert rz.razer_mx_workspace_bytes(*a) >= 0
