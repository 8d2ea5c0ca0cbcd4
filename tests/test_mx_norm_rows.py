"""The block norm's number of rows: a launch has fewer than 2^32 threads, 64 of them a
row (up to 1024 columns), 256 (up to 8192) or 1024."""
import ctypes

import pytest
import torch

import nvfp4_razer_w4a16_amd as rz
from nvfp4_razer_w4a16_amd.mx import razer_norm

MOST = {32: 2 ** 26 - 4, 1024: 2 ** 26 - 4, 1056: 2 ** 24 - 1, 8192: 2 ** 24 - 1, 8224: 2 ** 22 - 1, 32768: 2 ** 22 - 1}


@pytest.mark.parametrize("cols", MOST)
@pytest.mark.parametrize("over", [1, 4, 2 ** 20, 2 ** 40])
def test_more_rows_than_a_launch_holds_are_refused(cols, over):
    """On the host, before anything is enqueued: the addresses are never read."""
    a = razer_norm(rows=MOST[cols] + over, cols=cols, dtype=rz.RAZER_BF16, h=0x40000, h_stride=cols, h_out=0x50000,
                   residual_scale=1.0, eps=1e-5)
    assert rz.lib().razer_block_norm(ctypes.byref(a), None) == rz.RAZER_E_UNSUPPORTED


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")
def test_as_many_rows_as_a_launch_holds():
    """Rows at both ends and where a row's offset passes 2^31 bytes, against the same
    rows by themselves."""
    cols, rows = 32, MOST[32]
    h = torch.empty(rows, cols, dtype=torch.float16, device="cuda").normal_()
    w = torch.linspace(0.5, 2.0, cols, device="cuda").half()
    h_out, x = rz.razer_block_norm(None, h, pre_weight=w, packed=True)
    for first in (0, 2 ** 25 - 50, rows // 3, rows - 100):
        part = h[first:first + 100].clone()
        want_h, want = rz.razer_block_norm(None, part, pre_weight=w, packed=True)
        assert torch.equal(h_out[first:first + 100], want_h)
        assert torch.equal(x.codes[first:first + 100], want.codes)
        assert torch.equal(x.scales[first:first + 100], want.scales)
    assert torch.equal(h_out, h)
