"""The MXFP4 layer of ``examples/mx_block.py``, dense and of experts, and the calls
on a stream that is not the current one."""
import importlib.util
import os

import pytest
import torch

import nvfp4_razer_w4a16_amd as rz

pytestmark = pytest.mark.gpu

_path = os.path.join(os.path.dirname(os.path.abspath(__file__)), os.pardir, "examples", "mx_block.py")
_spec = importlib.util.spec_from_file_location("mx_block", _path)
block = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(block)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,hidden,inner,experts,top", [(1, 512, 1056, 0, 2), (70, 256, 544, 0, 2),
                                                             (5, 256, 320, 4, 2), (90, 512, 544, 16, 3)])
def test_layer(tokens, hidden, inner, experts, top, dtype):
    """Packing x and silu(g) * u to 4 bits errs by some 0.11 of their size each (an
    element's rounding is uniform in steps of a quarter to a third of it: 0.29 * 0.3,
    and a little more where a block's largest saturates), g and u each carry x's, so y
    is off by about 0.11 * sqrt(1 + 1 + 1) = 0.2.  A wrong layer is off by 1 or more."""
    torch.manual_seed(tokens)
    us, error = block.run(tokens, hidden, inner, 2, experts, top, dtype)
    assert us > 0
    assert error < 0.4


def test_given_stream():
    """A call on a given stream orders the copies and the workspace it makes with its
    launch, behind work that stream still has to do."""
    torch.manual_seed(0)
    rows, hidden, k = 300, 256, 16384
    wide = torch.randn(rows, k + 1, device="cuda")
    x = wide[:, 1:]  # rows that the call has to copy
    w = rz.razer_mx_quantize(torch.randn(hidden, k, device="cuda"))
    want_t = rz.razer_mx_quantize(x)
    want_y = rz.razer_mx_gemm(want_t, w)
    assert rz.razer_mx_workspace_bytes(rows, hidden, k) > 0
    offsets = torch.tensor([0, 100, rows], dtype=torch.int32, device="cuda")
    stack = rz.razer_mx_quantize(torch.randn(2 * hidden, k, device="cuda"))
    want_g = rz.razer_mx_gemm_grouped(want_t, stack, offsets)
    h = torch.randn(rows, hidden, device="cuda", dtype=torch.bfloat16)
    want_h, want_n = rz.razer_block_norm(want_y, h)
    want_q = rz.razer_mx_quantize_gated(h)
    late = torch.zeros_like(wide)
    torch.cuda.synchronize()
    for stream in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        with rz.mx._entered(stream):
            late.zero_()
            busy = torch.randn(4096, 4096, device="cuda")
            for _ in range(10):
                busy = (busy @ busy).clamp_(-1, 1)
            late.copy_(wide)
        t = rz.razer_mx_quantize(late[:, 1:], stream=stream)
        y = rz.razer_mx_gemm(t, w, stream=stream)
        g = rz.razer_mx_gemm_grouped(t, stack, offsets, stream=stream)
        q = rz.razer_mx_quantize_gated(h, stream=stream)
        v = rz.razer_mx_dequant(t, stream=stream)
        gh, gn = rz.razer_block_norm(y, h, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(t.codes, want_t.codes) and torch.equal(t.scales, want_t.scales)
        assert torch.equal(y, want_y) and torch.equal(g, want_g)
        assert torch.equal(q.codes, want_q.codes) and torch.equal(q.scales, want_q.scales)
        assert torch.equal(v, rz.razer_mx_dequant(want_t))
        assert torch.equal(gh, want_h) and torch.equal(gn, want_n)
