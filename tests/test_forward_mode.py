"""No call has a derivative in forward mode: a tangent among its inputs raises, with and
without a graph, instead of being lost."""
import pytest
import torch
from torch.autograd import forward_ad

import nvfp4_razer_w4a16_amd as rz


def _randn(*shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(sum(shape))).cuda()


def _inputs():
    w = rz.razer_i8_quantize(_randn(32, 64))
    return dict(x=_randn(4, 64), codes=w.codes, scales=w.scales, offsets=torch.tensor([0, 1, 4], dtype=torch.int32, device="cuda"),
                logits=_randn(4, 8), bias=_randn(8), rows=_randn(8, 64), weights=_randn(4, 2), add=_randn(4, 64),
                slots=torch.arange(8, dtype=torch.int32, device="cuda").view(4, 2), y=_randn(4, 64), h=_randn(4, 64),
                post=_randn(64), pre=_randn(64), gate=_randn(64))


def _weight(a):
    return rz.I8Tensor.of(a["codes"], a["scales"])


# call, its inputs that can carry a tangent, the same into a caller's own results
CALLS = {
    "razer_i8_quantize": (lambda a, **k: rz.razer_i8_quantize(a["x"], **k), ["x"], lambda: dict(out=rz.I8Tensor(4, 64, "cuda"))),
    "razer_i8_quantize_gated": (lambda a, **k: rz.razer_i8_quantize_gated(a["x"], **k), ["x"],
                                lambda: dict(out=rz.I8Tensor(4, 32, "cuda"))),
    "razer_i8_dequant": (lambda a, **k: rz.razer_i8_dequant(_weight(a), **k), ["scales"],
                         lambda: dict(out=torch.empty(32, 64, device="cuda"))),
    "razer_i8_gemm": (lambda a, **k: rz.razer_i8_gemm(rz.razer_i8_quantize(a["x"].detach()), _weight(a), torch.float32, **k), ["scales"],
                      lambda: dict(out=torch.empty(4, 32, device="cuda"))),
    "razer_i8_gemm_grouped": (lambda a, **k: rz.razer_i8_gemm_grouped(rz.razer_i8_quantize(a["x"].detach()), _weight(a),
                                                                      a["offsets"], out_dtype=torch.float32, **k),
                              ["scales"], lambda: dict(out=torch.empty(4, 16, device="cuda"))),
    "razer_moe_route": (lambda a, **k: rz.razer_moe_route(a["logits"], 2, bias=a["bias"], **k), ["logits", "bias"],
                        lambda: dict(out=rz.razer_moe_route(_randn(4, 8), 2))),
    "razer_moe_combine": (lambda a, **k: rz.razer_moe_combine(a["rows"], a["slots"], a["weights"], add=a["add"], **k),
                          ["rows", "weights", "add"], lambda: dict(out=torch.empty(4, 64, device="cuda"))),
    "razer_block_norm": (lambda a, **k: rz.razer_block_norm(a["y"], a["h"], post_weight=a["post"], pre_weight=a["pre"],
                                                            gate=a["gate"], **k), ["y", "h", "post", "pre", "gate"],
                         lambda: dict(h_out=torch.empty(4, 64, device="cuda"), x_out=torch.empty(4, 64, device="cuda"))),
}


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")
@pytest.mark.parametrize("name", CALLS)
def test_tangents_raise(name):
    call, inputs, own = CALLS[name]
    a = _inputs()
    want = call(a)
    with forward_ad.dual_level():
        for got in (call(a), call(a, **own())):  # no tangent: as ever
            for g, w in zip(*(t if isinstance(t, tuple) else (t,) for t in (got, want))):
                if isinstance(g, rz.I8Tensor):
                    g, w = rz.razer_i8_dequant(g), rz.razer_i8_dequant(w)
                assert torch.equal(g.float(), w.float())
        for which in inputs:
            b = dict(a, **{which: forward_ad.make_dual(a[which], torch.ones_like(a[which]))})
            for record in (True, False):
                with torch.set_grad_enabled(record):
                    with pytest.raises(RuntimeError, match=f"{name} has no derivative in forward mode"):
                        call(b)
            call(b, **own())  # a caller's own results stand outside any graph
            b[which] = b[which].detach()
            call(b)


def test_what_carries_no_tangent():
    t = torch.ones(3)
    rz.mx._no_tangents("a call", (None, t))
    with forward_ad.dual_level():
        rz.mx._no_tangents("a call", (None, t))
        with pytest.raises(RuntimeError, match="a call has no derivative"):
            rz.mx._no_tangents("a call", (t, forward_ad.make_dual(t, t)))
