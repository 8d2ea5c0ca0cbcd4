"""The block norm has no backward.  Its values are the same for inputs that require a
gradient, and a backward pass that reaches them raises instead of passing them by."""
import pytest
import torch

import nvfp4_razer_w4a16_amd as rz

gpu = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")]


def _gpu(f):
    for m in gpu:
        f = m(f)
    return f


def _inputs(**grad):
    g = torch.Generator().manual_seed(1)
    t = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    a = dict(y=t(4, 64), h=t(4, 64), post_weight=t(64), pre_weight=t(64), gate=t(2, 64))
    for k in grad:
        a[k].requires_grad_()
    return a


def _norm(a, **kw):
    return rz.razer_block_norm(a["y"], a["h"], **{k: a[k] for k in ("post_weight", "pre_weight", "gate")}, **kw)


@_gpu
@pytest.mark.parametrize("which", ["y", "h", "post_weight", "pre_weight", "gate"])
def test_backward_raises(which):
    want = _norm(_inputs())
    assert not any(t.requires_grad for t in want)
    a = _inputs(**{which: True})
    got = _norm(a)
    for g, w in zip(got, want):
        assert torch.equal(g, w)
    for part in got:
        assert part.requires_grad
        with pytest.raises(RuntimeError, match="razer_block_norm has no backward"):
            (part * 2 + a["h"]).sum().backward()
    h, _ = _norm(_inputs(**{which: True}), packed=True)
    with pytest.raises(RuntimeError, match="razer_block_norm has no backward"):
        h.sum().backward()


@_gpu
def test_results_without_gradients():
    """None is recorded where none is asked for, and a caller's own buffers stay plain."""
    a = _inputs(h=True, pre_weight=True)
    want = _norm(_inputs())
    with torch.no_grad():
        assert not any(t.requires_grad for t in _norm(a))
    with torch.inference_mode():
        assert all(torch.equal(g, w) for g, w in zip(_norm(a), want))
    outs = [torch.empty(4, 64, device="cuda") for _ in range(2)]
    for _ in range(2):
        assert all(g is o for g, o in zip(_norm(a, h_out=outs[0], x_out=outs[1]), outs))
        assert all(torch.equal(o, w) and not o.requires_grad for o, w in zip(outs, want))
    h, x = _norm(a)
    assert torch.equal(h.add_(1), want[0] + 1) and torch.equal(x.detach(), want[1])


def test_backward_of_what_has_none():
    w = torch.ones(3, requires_grad=True)
    a, b = rz.mx._without_backward("a call", (torch.zeros(2), torch.ones(2)), (None, w, torch.ones(1)))
    assert a.requires_grad and b.requires_grad and torch.equal(b.detach(), torch.ones(2))
    for t in (a, b):
        with pytest.raises(RuntimeError, match="a call has no backward"):
            (t.sum() + w.sum()).backward()
