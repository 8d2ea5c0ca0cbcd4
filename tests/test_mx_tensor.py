"""An MxTensor whose shape or buffers were changed after it was made: the kernels
would read past its buffers, so it is refused, until shape and buffers agree again."""
import copy
import pickle

import pytest
import torch

import nvfp4_razer_w4a16_amd as rz

U8 = torch.uint8
DEVICES = ["cpu", pytest.param("cuda", marks=[pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")])]


def _given(device="cpu", rows=4, cols=64):
    return rz.MxTensor.of(torch.zeros(rows, cols // 2, dtype=U8, device=device),
                          torch.zeros(rows, cols // 32, dtype=U8, device=device))


def _own(device="cpu", rows=4, cols=64):
    t = rz.MxTensor(rows, cols, device)
    t.codes.zero_(), t.scales.zero_()
    return t


def _set(name, value):
    return lambda t: setattr(t, name, value)


CHANGES = {
    "rows": _set("rows", 100), "cols": _set("cols", 4096), "fewer rows": _set("rows", 2), "fewer cols": _set("cols", 32),
    "codes": _set("codes", torch.zeros(4, 16, dtype=U8)), "scales": _set("scales", torch.zeros(3, 2, dtype=U8)),
    "type": _set("codes", torch.zeros(4, 32, dtype=torch.int8)), "odd cols": _set("cols", 40),
}
IN_PLACE = {
    "smaller codes": lambda t: t.codes.resize_(2, 8), "smaller scales": lambda t: t.scales.resize_(1, 1),
    "no codes": lambda t: t.codes.resize_(0), "larger codes": lambda t: t.codes.resize_(8, 32),
    "other scales": lambda t: t.scales.set_(torch.zeros(2, 4, dtype=U8, device=t.device)),
    "other codes": lambda t: t.codes.set_(torch.zeros(2, 8, dtype=U8, device=t.device)),
}


def _refused(t):
    with pytest.raises(ValueError, match="no contiguous uint8"):
        t.check()
    if t.device.type == "cpu":
        with pytest.raises(ValueError, match="no contiguous uint8"):
            rz.mx._operand(t, "x")
        return
    good = _given("cuda")
    for call in (lambda: rz.razer_mx_dequant(t), lambda: rz.razer_mx_gemm(t, good), lambda: rz.razer_mx_gemm(good, t),
                 lambda: rz.razer_mx_gemm_grouped(t, good, torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")),
                 lambda: rz.razer_mx_quantize(torch.ones(4, 64, device="cuda"), out=t),
                 lambda: rz.razer_block_norm(None, torch.ones(4, 64, device="cuda"), packed=True, x_out=t)):
        with pytest.raises(ValueError, match="no contiguous uint8"):
            call()
    torch.cuda.synchronize()


@pytest.mark.parametrize("device", DEVICES)
@pytest.mark.parametrize("what", CHANGES)
@pytest.mark.parametrize("make", [_given, _own])
def test_replaced(make, what, device):
    t = make(device)
    assert t.check() == t.codes.device
    CHANGES[what](t)
    _refused(t)


@pytest.mark.parametrize("device", DEVICES)
@pytest.mark.parametrize("what", IN_PLACE)
def test_changed_in_place(what, device):
    t = _given(device)
    t.check()
    IN_PLACE[what](t)
    _refused(t)


@pytest.mark.parametrize("what", IN_PLACE)
def test_own_buffer_outlives_changes_of_its_views(what):
    """Its addresses come from the one buffer that it keeps."""
    t = _own()
    before = t.struct()
    IN_PLACE[what](t)
    t.check()
    s = t.struct()
    assert (s.rows, s.cols, s.scales - s.codes) == (4, 64, 128)
    assert t._buf.untyped_storage().nbytes() >= 136
    if what != "larger codes":  # which moves the memory of both
        assert s.codes == before.codes


@pytest.mark.parametrize("make", [_given, _own])
def test_shape_and_buffers_replaced_together(make):
    t = make()
    t.rows, t.cols = 2, 96
    t.codes, t.scales = torch.zeros(2, 48, dtype=U8), torch.zeros(2, 3, dtype=U8)
    t.check()
    s = t.struct()
    assert t.shape == (2, 96) and t.nbytes() == 102
    assert (s.rows, s.cols, s.codes, s.scales) == (2, 96, t.codes.data_ptr(), t.scales.data_ptr())
    t.rows = 2  # what it is already
    t.check()


def test_device_is_that_of_the_buffers():
    t = _given()
    with pytest.raises(AttributeError):
        t.device = torch.device("cuda", 0)
    assert t.device.type == "cpu"


@pytest.mark.parametrize("codes,scales", [((4, 32), (4, 3)), ((4, 32), (2, 2)), ((4, 40), (4, 2)), ((2, 2, 32), (2, 3, 2))])
def test_of_refuses(codes, scales):
    with pytest.raises((ValueError, RuntimeError)):
        rz.MxTensor.of(torch.zeros(codes, dtype=U8), torch.zeros(scales, dtype=U8))
    with pytest.raises(ValueError, match="no contiguous uint8"):
        rz.MxTensor.of(torch.zeros(32, 4, dtype=U8).t(), torch.zeros(4, 2, dtype=U8))
    with pytest.raises(ValueError, match="no contiguous uint8"):
        rz.MxTensor.of(torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4, 2, dtype=U8))


def test_copies_and_pickles():
    t = _given()
    t.codes.fill_(3)
    for u in (copy.copy(t), copy.deepcopy(t), pickle.loads(pickle.dumps(t))):
        assert u.check().type == "cpu" and u.shape == (4, 64)
        assert torch.equal(u.codes, t.codes) and torch.equal(u.scales, t.scales)
        assert u.struct().codes == u.codes.data_ptr() and u.struct().scales == u.scales.data_ptr()
