"""What the 8-bit integer calls, the routing and the combination refuse, on the host and
before anything is enqueued: no GPU is needed, the addresses are never read."""
import ctypes

import pytest
import torch

import nvfp4_razer_w4a16_amd as rz
from nvfp4_razer_w4a16_amd.i8 import razer_i8
from nvfp4_razer_w4a16_amd.moe import razer_combine, razer_route

X, Y, WS = 0x40000, 0x50000, 0x60000
INVALID, UNSUPPORTED, OK = rz.RAZER_E_INVALID, rz.RAZER_E_UNSUPPORTED, rz.RAZER_OK


def _i8(rows=4, cols=64, codes=0x10000, scales=0x20000):
    return razer_i8(rows, cols, codes, scales)


def test_struct_layouts_match_the_header():
    assert ctypes.sizeof(razer_i8) == 32
    assert razer_route.scale.offset == 48 and razer_route.logits.offset == 56 and ctypes.sizeof(razer_route) == 112
    assert razer_combine.dtype.offset == 48 and razer_combine.y.offset == 56 and ctypes.sizeof(razer_combine) == 96


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(cols=40)), (INVALID, dict(rows=-1)), (INVALID, dict(rows=1 << 60)), (INVALID, dict(codes=0)),
    (INVALID, dict(scales=0)), (INVALID, dict(codes=0x10008)), (INVALID, dict(scales=0x20002)), (INVALID, dict(dt=3)),
    (INVALID, dict(x=0)), (INVALID, dict(x=X + 8)), (INVALID, dict(stride=32)), (INVALID, dict(stride=130)),
    (INVALID, dict(out=None)), (UNSUPPORTED, dict(rows=(1 << 28) + 1)), (UNSUPPORTED, dict(cols=0)),
    (OK, dict(rows=0, codes=0, scales=0, x=0)),
])
@pytest.mark.parametrize("gated", [False, True])
def test_encoders_refuse(want, kw, gated):
    a = dict(rows=4, cols=64, codes=0x10000, scales=0x20000, dt=rz.RAZER_BF16, x=X, stride=128)
    a.update(kw)
    t = _i8(a["rows"], a["cols"], a["codes"], a["scales"])
    f = rz.lib().razer_i8_quantize_gated if gated else rz.lib().razer_i8_quantize
    assert f(a["x"], a["dt"], a["stride"], None if "out" in kw else ctypes.byref(t), None) == want


def test_gated_rows_hold_both_halves():
    t = _i8()
    assert rz.lib().razer_i8_quantize_gated(X, rz.RAZER_F16, 64, ctypes.byref(t), None) == INVALID


@pytest.mark.parametrize("want,t,out,dt", [
    (INVALID, {}, 0, 0), (INVALID, {}, Y + 8, 0), (INVALID, {}, Y, 5), (INVALID, dict(cols=8), Y, 0),
    (UNSUPPORTED, dict(rows=1 << 31), Y, 0), (OK, dict(rows=0), 0, 1), (OK, dict(cols=0), 0, 1)])
def test_decoder_refuses(want, t, out, dt):
    s = _i8(**t)
    assert rz.lib().razer_i8_dequant(ctypes.byref(s), out, dt, None) == want


@pytest.mark.parametrize("want,x,w,kw", [
    (INVALID, dict(cols=80), {}, {}), (INVALID, dict(codes=0), {}, {}), (INVALID, {}, dict(rows=-2), {}),
    (INVALID, {}, dict(scales=0), {}), (INVALID, {}, {}, dict(y=0)), (INVALID, {}, {}, dict(y=Y + 2)),
    (INVALID, {}, {}, dict(dt=7)), (UNSUPPORTED, dict(cols=0), dict(cols=0), {}),
    (UNSUPPORTED, dict(cols=rz.RAZER_I8_MAX_K + 16), dict(cols=rz.RAZER_I8_MAX_K + 16), {}),
    (UNSUPPORTED, {}, dict(rows=(1 << 30) + 1), {}), (OK, dict(rows=0), {}, dict(y=0)), (OK, {}, dict(rows=0), dict(y=0)),
])
def test_product_refuses(want, x, w, kw):
    a = dict(y=Y, dt=rz.RAZER_F32)
    a.update(kw)
    sx, sw = _i8(**x), _i8(**w)
    L = rz.lib()
    assert L.razer_i8_gemm(ctypes.byref(sx), ctypes.byref(sw), a["y"], a["dt"], WS, 1 << 40, None) == want
    assert L.razer_i8_gemm(None, ctypes.byref(sw), Y, 0, WS, 1 << 40, None) == INVALID


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(experts=0)), (INVALID, dict(experts=3)),
    (INVALID, dict(experts=rz.RAZER_MX_MAX_EXPERTS * 2, wrows=rz.RAZER_MX_MAX_EXPERTS * 2)), (INVALID, dict(off=0)),
    (INVALID, dict(off=0x70002)), (INVALID, dict(rows=0x80001)), (INVALID, dict(rows=0, m=5)), (INVALID, dict(m=-1)),
    (INVALID, dict(xrows=0)), (INVALID, dict(y=0)), (INVALID, dict(y=Y + 4)), (UNSUPPORTED, dict(m=(1 << 30) + 1)),
    (UNSUPPORTED, dict(xrows=1 << 26)), (OK, dict(m=0)), (OK, dict(wrows=0))])
def test_grouped_refuses(want, kw):
    a = dict(experts=2, off=0x70000, rows=0x80000, m=6, y=Y, xrows=4, wrows=4)
    a.update(kw)
    sx, sw = _i8(rows=a["xrows"]), _i8(rows=a["wrows"])
    assert rz.lib().razer_i8_gemm_grouped(ctypes.byref(sx), ctypes.byref(sw), a["off"], a["experts"], a["rows"], a["m"],
                                          a["y"], rz.RAZER_BF16, WS, 1 << 40, None) == want


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(tokens=-1)), (INVALID, dict(experts=0)), (INVALID, dict(top=0)),
    (INVALID, dict(groups=0)), (INVALID, dict(groups=5)), (INVALID, dict(groups=128, experts=128)),
    (INVALID, dict(groups_kept=0)), (INVALID, dict(groups_kept=5)), (INVALID, dict(top=17)),
    (INVALID, dict(group_best=0)), (INVALID, dict(group_best=3)), (INVALID, dict(score=2)), (INVALID, dict(score=-1)),
    (INVALID, dict(dtype=3)), (INVALID, dict(flags=2)), (INVALID, dict(logits=0)), (INVALID, dict(logits=X + 2)),
    (INVALID, dict(stride=31)), (INVALID, dict(stride=1 << 62)), (INVALID, dict(chosen=0)), (INVALID, dict(weights=0)),
    (INVALID, dict(weights=Y + 2)), (INVALID, dict(bias=Y + 1)), (INVALID, dict(rows=0)), (INVALID, dict(slots=0)),
    (INVALID, dict(offsets=0)), (INVALID, dict(slots=Y + 3)), (INVALID, dict(space=0, tokens=40)), (INVALID, dict(ws=0, tokens=40)),
    (INVALID, dict(ws=WS + 4, tokens=40)),
    (UNSUPPORTED, dict(experts=1025, groups=1, groups_kept=1, stride=2000)), (UNSUPPORTED, dict(top=33)),
    (UNSUPPORTED, dict(tokens=1 << 29)), (UNSUPPORTED, dict(tokens=(1 << 20) + 1)),
    (UNSUPPORTED, dict(tokens=(1 << 26) + 1, offsets=0, rows=0, slots=0)), (OK, dict(tokens=0, offsets=0, rows=0, slots=0, logits=0, chosen=0, weights=0))])
def test_route_refuses(want, kw):
    ws = dict(ws=WS, space=1 << 40)
    ws.update({k: kw[k] for k in kw if k in ws})
    a = razer_route(tokens=4, stride=32, experts=32, top=2, groups=4, groups_kept=2, group_best=2, score=1,
                    dtype=rz.RAZER_F32, flags=1, scale=1.0, logits=X, bias=Y, chosen=Y, weights=Y, offsets=Y, rows=Y,
                    slots=Y)
    for k, v in kw.items():
        if k not in ws:
            setattr(a, k, v)
    L = rz.lib()
    assert L.razer_moe_route(ctypes.byref(a), ws["ws"], ws["space"], None) == want
    assert L.razer_moe_route(None, WS, 1 << 40, None) == INVALID


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(tokens=-1)), (INVALID, dict(cols=-1)), (INVALID, dict(top=0)), (INVALID, dict(dtype=4)),
    (INVALID, dict(y_rows=-1)), (INVALID, dict(y=0)), (INVALID, dict(y=X + 1)), (INVALID, dict(y_stride=63)),
    (INVALID, dict(add_stride=63)), (INVALID, dict(add=X + 1)), (INVALID, dict(slots=0)), (INVALID, dict(slots=X + 2)),
    (INVALID, dict(weights=0)), (INVALID, dict(out=0)), (INVALID, dict(out=Y + 1)), (INVALID, dict(tokens=1 << 60)),
    (UNSUPPORTED, dict(top=33)), (UNSUPPORTED, dict(tokens=1 << 29, add=0)), (UNSUPPORTED, dict(y_rows=1 << 31)),
    (OK, dict(tokens=0, slots=0, out=0)), (OK, dict(cols=0))])
def test_combine_refuses(want, kw):
    a = razer_combine(tokens=4, top=2, cols=64, y_rows=8, y_stride=64, add_stride=64, dtype=rz.RAZER_BF16, y=X, slots=X,
                      weights=X, add=X, out=Y)
    for k, v in kw.items():
        setattr(a, k, v)
    assert rz.lib().razer_moe_combine(ctypes.byref(a), None) == want
    assert rz.lib().razer_moe_combine(None, None) == INVALID


def test_workspace_bytes():
    for a in ((0, 8, 64, 0), (8, 0, 64, 0), (8, 8, 0, 2), (-1, 8, 64, 0), (8, 8, 64, -1), (2 ** 30 + 1, 8, 64, 0),
              (8, 2 ** 62, 64, 0), (8, 8, rz.RAZER_I8_MAX_K + 16, 0), (8, 8, 64, rz.RAZER_MX_MAX_EXPERTS + 1)):
        assert rz.razer_i8_workspace_bytes(*a) == 0
    for a in ((-1, 8, 2), (8, 0, 2), (8, 8, 0), (8, 1025, 2), (8, 64, 33), (2 ** 20 + 1, 8, 1), (2 ** 62, 8, 1)):
        assert rz.razer_moe_workspace_bytes(*a) == 0
    for a in ((2 ** 30, 2 ** 30, 131056, 0), (2 ** 30, 2 ** 30, 131056, 4096), (1, 2 ** 30, 16, 0)):
        assert rz.razer_i8_workspace_bytes(*a) >= 0
    assert rz.razer_moe_workspace_bytes(1 << 20, 1024, 32) > 0


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    t = rz.I8Tensor(4, 64, "cpu")
    x = torch.zeros(4, 64)
    for call in (lambda: rz.razer_i8_quantize(x), lambda: rz.razer_i8_quantize_gated(x), lambda: rz.razer_i8_dequant(t),
                 lambda: rz.razer_i8_gemm(t, t), lambda: rz.razer_moe_route(x, 2),
                 lambda: rz.razer_i8_gemm_grouped(t, t, torch.zeros(3, dtype=torch.int32)),
                 lambda: rz.razer_moe_combine(x, torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2))):
        with pytest.raises(ValueError, match="must be on a GPU"):
            call()
    with pytest.raises(ValueError, match="multiple of 16"):
        rz.I8Tensor(4, 40, "cpu")
    codes, scales = torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4)
    for c, s in ((codes.view(torch.uint8), scales), (codes, scales.half()), (codes, scales[:3]),
                 (codes[:, :16], scales), (codes[:, :24].contiguous(), scales)):
        with pytest.raises(ValueError, match="no contiguous 8-bit tensor"):
            rz.I8Tensor.of(c, s)
    with pytest.raises(TypeError, match="I8Tensor"):
        rz.razer_i8_gemm(x, t)


def test_tensor_keeps_its_shape_and_buffers_together():
    t = rz.I8Tensor(4, 32, "cpu")
    assert t.codes.shape == (4, 32) and t.scales.shape == (4,) and t.nbytes() == 4 * 36
    t.codes.fill_(3), t.scales.fill_(0.5)
    assert t.check() == torch.device("cpu")
    stack = rz.I8Tensor.of(t.codes.view(2, 2, 32), t.scales.view(2, 2))
    assert stack.shape == (4, 32) and stack.codes.data_ptr() == t.codes.data_ptr()
    for change in (lambda s: setattr(s, "rows", 3), lambda s: setattr(s, "cols", 16),
                   lambda s: setattr(s, "codes", torch.zeros(4, 16, dtype=torch.int8)),
                   lambda s: setattr(s, "scales", torch.zeros(5)), lambda s: s.scales.resize_(3)):
        s = rz.I8Tensor.of(t.codes.clone(), t.scales.clone())
        change(s)
        with pytest.raises(ValueError, match="no contiguous 8-bit tensor"):
            s.check()
    own = rz.I8Tensor(2, 16, "cpu")
    own.rows = 3
    with pytest.raises(ValueError, match="no contiguous 8-bit tensor"):
        own.check()


@pytest.mark.gpu
def test_binding_refuses_before_it_writes():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    w, x = rz.razer_i8_quantize(torch.ones(6, 64, device="cuda")), rz.razer_i8_quantize(torch.ones(4, 64, device="cuda"))
    k = rz.razer_i8_quantize(torch.ones(6, 96, device="cuda"))
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    h = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.full((4, 6), 7.0, device="cuda")
    r = rz.razer_moe_route(h, 2)
    for call in (lambda: rz.razer_i8_gemm(x, k), lambda: rz.razer_i8_gemm(x, w, out=out[:3]),
                 lambda: rz.razer_i8_gemm(x, w, out=out.t()), lambda: rz.razer_i8_gemm_grouped(x, w, off.long()),
                 lambda: rz.razer_i8_gemm_grouped(x, w, off[:0]), lambda: rz.razer_i8_gemm_grouped(x, w, off.cpu()),
                 lambda: rz.razer_i8_gemm_grouped(x, k, off), lambda: rz.razer_i8_gemm_grouped(x, w, off, off[None]),
                 lambda: rz.razer_i8_quantize(h, out=w), lambda: rz.razer_i8_quantize(h[:, :40]),
                 lambda: rz.razer_i8_quantize_gated(h[:, :16]), lambda: rz.razer_i8_dequant(x, out=out),
                 lambda: rz.razer_moe_route(h[0], 2), lambda: rz.razer_moe_route(h, 0), lambda: rz.razer_moe_route(h, 65),
                 lambda: rz.razer_moe_route(h, 2, score="max"), lambda: rz.razer_moe_route(h, 2, groups=5),
                 lambda: rz.razer_moe_route(h, 9, groups=8, groups_kept=1), lambda: rz.razer_moe_route(h, 2, bias=h[0]),
                 lambda: rz.razer_moe_route(h, 2, bias=torch.zeros(63, device="cuda")),
                 lambda: rz.razer_moe_route(h, 3, out=r), lambda: rz.razer_moe_route(h[:3], 2, out=r),
                 lambda: rz.razer_moe_combine(h, r.slots, r.weights.half()),
                 lambda: rz.razer_moe_combine(h, r.slots.long(), r.weights),
                 lambda: rz.razer_moe_combine(h, r.slots[:2], r.weights),
                 lambda: rz.razer_moe_combine(h, r.slots, r.weights, add=h[:3]),
                 lambda: rz.razer_moe_combine(h, r.slots, r.weights, add=h.float()),
                 lambda: rz.razer_moe_combine(h, r.slots, r.weights, out=out)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: rz.razer_moe_route(h, 33), lambda: rz.razer_moe_route(h, 2, group_best=3),
                 lambda: rz.razer_moe_route(h.repeat(9, 1), 2, workspace=off[:1]),
                 lambda: rz.razer_moe_route(torch.zeros(2, 1025, device="cuda"), 2)):
        with pytest.raises(rz.RazerError):
            call()
    for bad in (torch.float64, torch.int32):
        for call in (lambda: rz.razer_i8_quantize(h.to(bad)), lambda: rz.razer_moe_route(h.to(bad), 2),
                     lambda: rz.razer_moe_combine(h.to(bad), r.slots, r.weights)):
            with pytest.raises(TypeError):
                call()
    torch.cuda.synchronize()
    assert (out == 7.0).all()


@pytest.mark.gpu
def test_backward_raises():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    l = torch.randn(5, 16, device="cuda", requires_grad=True)
    want = rz.razer_moe_route(l.detach(), 3)
    r = rz.razer_moe_route(l, 3)
    assert torch.equal(r.weights.detach(), want.weights) and torch.equal(r.experts, want.experts)
    with pytest.raises(RuntimeError, match="razer_moe_route has no backward"):
        r.weights.sum().backward()
    for which in range(3):
        t = [torch.randn(15, 8, device="cuda"), want.weights.clone(), torch.randn(5, 8, device="cuda")]
        plain = rz.razer_moe_combine(t[0], want.slots, t[1], t[2])
        t[which].requires_grad_()
        got = rz.razer_moe_combine(t[0], want.slots, t[1], t[2])
        assert torch.equal(got.detach(), plain)
        with pytest.raises(RuntimeError, match="razer_moe_combine has no backward"):
            got.sum().backward()
        with torch.no_grad():
            assert not rz.razer_moe_combine(t[0], want.slots, t[1], t[2]).requires_grad


@pytest.mark.parametrize("owned", [True, False])
def test_a_copy_is_where_its_buffers_are(owned):
    """A tensor copied whole, or saved and loaded, is taken from its own buffers."""
    import copy
    import pickle

    t = rz.I8Tensor(3, 32, "cpu")
    t.codes.copy_(torch.arange(96).view(3, 32))
    t.scales.fill_(2.0)
    if not owned:
        t = rz.I8Tensor.of(t.codes.clone(), t.scales.clone())
    for other in (copy.deepcopy(t), pickle.loads(pickle.dumps(t))):
        packed = razer_i8.from_buffer_copy(other._checked("t"))
        assert (packed.rows, packed.cols) == (3, 32)
        assert packed.codes == other.codes.data_ptr() != t.codes.data_ptr()
        assert packed.scales == other.scales.data_ptr() != t.scales.data_ptr()
        assert torch.equal(other.codes, t.codes) and torch.equal(other.scales, t.scales)
        other.codes[0, 0] = 9
        other.scales[1] = 3.0
        assert ctypes.string_at(packed.codes, 1) == b"\x09" and t.codes[0, 0] == 0
        assert ctypes.c_float.from_address(packed.scales + 4).value == 3.0 and t.scales[1] == 2.0
    assert razer_i8.from_buffer_copy(t._checked("t")).codes == t.codes.data_ptr()
