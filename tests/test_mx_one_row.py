"""One row of a wider buffer (a decoded token beside other states) as the input of
the MXFP4 encoders and the block norm: torch counts it as contiguous whatever its
stride, which then need not be whole 16 bytes."""
import numpy as np
import pytest
import torch

import mx_common as mx
import nvfp4_razer_w4a16_amd as rz

DT = mx.DT
# (columns of the buffer, row, first column) of a row of 512: strides and addresses on 16 bytes and not
VIEWS = [(516, 0, 0), (516, 1, 0), (516, 1, 4), (515, 0, 0), (515, 2, 3), (520, 2, 8), (520, 0, 1), (512, 1, 0)]


def _view(buf, row, first, cols=512):
    return buf[row:row + 1, first:first + cols]


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("wide,row,first", VIEWS)
def test_stride_of_one_row(wide, row, first, dt):
    """What goes to the library: the row's values, at 16 bytes, with a stride it takes."""
    buf = torch.randn(3, wide).to(DT[dt])
    v = _view(buf, row, first)
    x, ptr, ld = rz.mx._rows_of(v, 512)
    assert torch.equal(x, v) and ptr == x.data_ptr() and ptr % 16 == 0
    assert ld >= 512 and ld * x.element_size() % 16 == 0


@pytest.mark.parametrize("dt", DT)
def test_strides_of_rows(dt):
    """More rows than one keep their stride where it is whole 16 bytes, and are copied where not."""
    buf = torch.randn(5, 1032).to(DT[dt])
    for v, kept in ((buf[:, :512], True), (buf[::2, 8:520], True), (buf[:2, 1:513], False), (buf.t()[:512].t(), True),
                    (buf[:, ::2][:, :512], False), (buf[:1].expand(5, 1032)[:, :512], False), (buf[1:, 4:516], dt == "f32")):
        x, ptr, ld = rz.mx._rows_of(v, 512)
        assert torch.equal(x, v) and ptr % 16 == 0 and ld * x.element_size() % 16 == 0
        assert (ptr == v.data_ptr()) == kept
        assert ld == x.stride(0) >= 512


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("wide,row,first", VIEWS)
def test_one_row_through_the_calls(wide, row, first, dt):
    rng = np.random.default_rng(wide + row)
    a, b = (torch.from_numpy(rng.standard_normal((3, wide))).to(DT[dt]).cuda() for _ in range(2))
    v, u = _view(a, row, first), _view(b, row, first)
    code, byte = mx.encode(v.double().cpu().numpy())
    t = rz.razer_mx_quantize(v)
    assert np.array_equal(t.scales.cpu().numpy(), byte) and np.array_equal(t.codes.cpu().numpy(), mx.pack(code))
    own_v, own_u = (torch.stack([w[0]]) for w in (v, u))  # rows of their own
    got, want = rz.razer_mx_quantize_gated(v), rz.razer_mx_quantize_gated(own_v)
    assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)
    for y, h in ((v, u), (own_v, u), (v, own_u)):
        for g, w in zip(rz.razer_block_norm(y, h, post_norm=True), rz.razer_block_norm(own_v, own_u, post_norm=True)):
            assert torch.equal(g, w)
