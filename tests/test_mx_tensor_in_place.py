"""Buffers given to an MxTensor and changed in place, at the same address and length: their
bytes would be read in another layout than they show, so the tensor is refused until they
fit again."""
import pytest
import torch

import nvfp4_razer_w4a16_amd as rz
from test_mx_tensor import DEVICES, U8, _given, _refused

UNFIT = {
    "turned codes": lambda t: t.codes.t_(), "turned scales": lambda t: t.scales.t_(),
    "codes of another shape": lambda t: t.codes.resize_(8, 16), "flat scales": lambda t: t.scales.resize_(8),
    "codes apart": lambda t: t.codes.as_strided_((4, 32), (1, 4)),
    "codes with a sign": lambda t: setattr(t.codes, "data", t.codes.view(torch.int8)),
    "scales with a sign": lambda t: setattr(t.scales, "data", t.scales.view(torch.int8)),
}


@pytest.mark.parametrize("device", DEVICES)
@pytest.mark.parametrize("what", UNFIT)
def test_refused(what, device):
    t = _given(device)
    t.check()
    UNFIT[what](t)
    for _ in range(2):
        _refused(t)


def test_changed_back():
    t = _given()
    t.codes.t_()
    with pytest.raises(ValueError, match="no contiguous uint8"):
        t.check()
    t.codes.t_()
    assert t.check() == torch.device("cpu")


@pytest.mark.parametrize("device", DEVICES)
def test_replaced_by_others_that_fit(device):
    t = _given(device)
    t.check()
    t.codes.data = torch.full((4, 32), 0x22, dtype=U8, device=device)  # codes of 1.0
    t.scales.data = torch.full((4, 2), 128, dtype=U8, device=device)   # times 2
    s = rz.mx._operand(t, "t") if device == "cuda" else t._checked("t")
    assert (s.rows, s.cols, s.codes, s.scales) == (4, 64, t.codes.data_ptr(), t.scales.data_ptr())
    if device == "cuda":
        assert (rz.razer_mx_dequant(t) == 2.0).all()
