"""The 8-bit operators and the routing have no backward.  Their values are the same for
inputs that require a gradient, and a backward pass that reaches them raises instead of
passing them by, also by way of a packed tensor."""
import pytest
import torch

import nvfp4_razer_w4a16_amd as rz

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")]


def _randn(*shape, seed=0, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).cuda().to(dtype)


def _uses(t, w, stack, offsets):
    """What a packed x [6, 64] ends in."""
    return {"dequant": rz.razer_i8_dequant(t), "gemm": rz.razer_i8_gemm(t, w), "weight": rz.razer_i8_gemm(w, t),
            "grouped": rz.razer_i8_gemm_grouped(t, stack, offsets),
            "given": rz.razer_i8_gemm(rz.I8Tensor.of(t.codes.view(2, 3, 64), t.scales.view(2, 3)), w)}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_gradients_do_not_pass_an_encoder_unseen(gated, apart, dtype):
    call, name = ((rz.razer_i8_quantize_gated, "razer_i8_quantize_gated") if gated
                  else (rz.razer_i8_quantize, "razer_i8_quantize"))
    x = _randn(6, 128 if gated else 64, dtype=dtype)
    if apart:  # rows that the call copies
        x = torch.cat([x[:, :1], x], 1)[:, 1:]
    w, stack = rz.razer_i8_quantize(_randn(48, 64, seed=1)), rz.razer_i8_quantize(_randn(96, 64, seed=2))
    offsets = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    want_t = call(x)
    assert not want_t.scales.requires_grad
    want = _uses(want_t, w, stack, offsets)
    x = x.detach().requires_grad_()
    t = call(x)
    assert torch.equal(t.codes, want_t.codes) and torch.equal(t.scales, want_t.scales)
    got = _uses(t, w, stack, offsets)
    for k, y in got.items():
        assert torch.equal(y, want[k]) and y.requires_grad and not want[k].requires_grad, k
        other = _randn(*y.shape, seed=3).requires_grad_()  # something else that learns
        with pytest.raises(RuntimeError, match="has no backward"):
            (y.float() + other).sum().backward()
        assert x.grad is None
    with pytest.raises(RuntimeError, match=f"{name} has no backward"):
        t.scales.sum().backward()
    down = rz.razer_i8_quantize(_randn(8, 48, seed=4))
    chain = rz.razer_i8_gemm(rz.razer_i8_quantize(rz.razer_i8_gemm(t, w)), down)
    with pytest.raises(RuntimeError, match="has no backward"):
        (chain.sum() + x.sum()).backward()


def test_outside_a_graph():
    """Nothing is recorded where none is asked for, and in a caller's own tensor."""
    x = _randn(6, 64).requires_grad_()
    with torch.no_grad():
        t = rz.razer_i8_quantize(x)
        assert not t.scales.requires_grad
    with torch.inference_mode():
        assert not rz.razer_i8_quantize(x).scales.requires_grad
    out = rz.I8Tensor(6, 64, "cuda")
    assert rz.razer_i8_quantize(x, out=out) is out and not out.scales.requires_grad
    assert not rz.razer_i8_gemm(out, t).requires_grad
    assert not rz.razer_i8_gemm(rz.razer_i8_quantize(x.detach()), t).requires_grad


def test_packed_again_and_on_a_stream():
    """The tensor stays good for calls whatever graph it stands in."""
    x = _randn(6, 64).requires_grad_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    t = rz.razer_i8_quantize(x, stream=s)
    y = rz.razer_i8_dequant(t, stream=s)
    s.synchronize()
    assert t.check() == x.device and y.requires_grad and torch.equal(y, rz.razer_i8_dequant(rz.razer_i8_quantize(x.detach())))
    with torch.no_grad():
        rz.razer_i8_quantize(x * 2, out=t)
    assert torch.equal(rz.razer_i8_dequant(t), rz.razer_i8_dequant(rz.razer_i8_quantize(x.detach() * 2)))
