"""An I8Tensor whose buffers were changed in place: a call takes what codes and scales show,
or refuses them."""
import pytest
import torch

import nvfp4_razer_w4a16_amd as rz
from nvfp4_razer_w4a16_amd.i8 import razer_i8

DEVICES = ["cpu", pytest.param("cuda", marks=[pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")])]


def _given(device="cpu", rows=4, cols=32):
    return rz.I8Tensor.of(torch.ones(rows, cols, dtype=torch.int8, device=device), torch.ones(rows, device=device))


def _own(device="cpu", rows=4, cols=32):
    t = rz.I8Tensor(rows, cols, device)
    t.codes.fill_(1), t.scales.fill_(1.0)
    return t


def _own_checked(device="cpu"):
    t = _own(device)
    t.check()
    return t


def _data(name, make):
    def change(t):
        getattr(t, name).data = make().to(t.device)
    return change


UNFIT = {
    "turned codes": lambda t: t.codes.t_(), "codes of another shape": lambda t: t.codes.resize_(8, 16),
    "flat codes": lambda t: t.codes.resize_(128), "fewer codes": lambda t: t.codes.resize_(2, 32),
    "codes apart": lambda t: t.codes.as_strided_((4, 32), (1, 4)),
    "codes of bits": _data("codes", lambda: torch.ones(4, 32, dtype=torch.uint8)),
    "bits of the same memory": lambda t: setattr(t.codes, "data", t.codes.view(torch.uint8)),
    "fewer scales": _data("scales", lambda: torch.zeros(3)), "more scales": _data("scales", lambda: torch.zeros(7)),
    "scales of another shape": lambda t: t.scales.resize_(2, 2),
    "scales apart": lambda t: t.scales.as_strided_((4,), (0,)),
    "whole scales": lambda t: setattr(t.scales, "data", t.scales.view(torch.int32)),
}
FIT = {
    "scales": _data("scales", lambda: torch.arange(4) + 5.0), "codes": _data("codes", lambda: torch.full((4, 32), 7, dtype=torch.int8)),
    "set scales": lambda t: t.scales.set_(torch.full((4,), 3.0, device=t.device)),
    "written": lambda t: (t.codes.fill_(2), t.scales.fill_(0.5)),
}
MAKE = [_given, _own, _own_checked]


@pytest.mark.parametrize("device", DEVICES)
@pytest.mark.parametrize("what", UNFIT)
@pytest.mark.parametrize("make", MAKE)
def test_refused(make, what, device):
    t = make(device)
    UNFIT[what](t)
    for _ in range(2):
        with pytest.raises(ValueError, match="no contiguous 8-bit tensor"):
            t.check()
    if device == "cpu":
        return
    good = _given("cuda")
    for call in (lambda: rz.razer_i8_dequant(t), lambda: rz.razer_i8_gemm(t, good), lambda: rz.razer_i8_gemm(good, t),
                 lambda: rz.razer_i8_gemm_grouped(good, t, torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")),
                 lambda: rz.razer_i8_quantize(torch.ones(4, 32, device="cuda"), out=t)):
        with pytest.raises(ValueError, match="no contiguous 8-bit tensor"):
            call()
    torch.cuda.synchronize()


@pytest.mark.parametrize("device", DEVICES)
@pytest.mark.parametrize("what", FIT)
@pytest.mark.parametrize("make", MAKE)
def test_taken_as_shown(make, what, device):
    t = make(device)
    FIT[what](t)
    packed = razer_i8.from_buffer_copy(t._checked("t"))
    assert (packed.rows, packed.cols) == (4, 32)
    assert (packed.codes, packed.scales) == (t.codes.data_ptr(), t.scales.data_ptr())
    if device == "cuda":
        assert torch.equal(rz.razer_i8_dequant(t), t.codes.float() * t.scales[:, None])
        out = rz.razer_i8_quantize(torch.full((4, 32), -127.0, device="cuda"), out=t)
        assert out is t and (t.codes == -127).all() and (t.scales == 1).all()


def test_changed_back():
    t = _given()
    t.codes.t_()
    with pytest.raises(ValueError, match="no contiguous 8-bit tensor"):
        t.check()
    t.codes.t_()
    assert t.check() == torch.device("cpu")
