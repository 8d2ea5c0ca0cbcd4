"""The feed-forward half of a transformer block with weights and activations in MXFP4 or
in 8-bit integers, dense or as a mixture of experts:

    python examples/mx_block.py [--form mx] [--tokens 1] [--hidden 4096] [--inner 14336]
                                [--layers 4] [--experts 0] [--top 2]

``y`` is what the block's attention gave, ``h`` the residual.  A layer of the dense form
is residual and both norms with the packing of x (in MXFP4 one launch, in 8-bit integers
two), the gate and up projections as one product, silu(gate) * up with its packing, the
down projection.  A layer of experts routes its tokens and joins the experts' rows again
on the GPU, without a wait.  The layers are captured in a graph and replayed; the last
layer is compared with the same layer in 32-bit torch on the decoded weights.
"""
import argparse
import os
import sys
from types import SimpleNamespace

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), os.pardir))
import nvfp4_razer_w4a16_amd as rz  # noqa: E402


# the calls of each form
FORMS = {"mx": SimpleNamespace(pack=rz.razer_mx_quantize, gated=rz.razer_mx_quantize_gated, values=rz.razer_mx_dequant,
                               gemm=rz.razer_mx_gemm, grouped=rz.razer_mx_gemm_grouped),
         "i8": SimpleNamespace(pack=rz.razer_i8_quantize, gated=rz.razer_i8_quantize_gated, values=rz.razer_i8_dequant,
                               gemm=rz.razer_i8_gemm, grouped=rz.razer_i8_gemm_grouped)}


class Layer:
    """Random weights of one layer, packed once; experts' weights are stacked by rows."""

    def __init__(self, hidden, inner, experts=0, dtype=torch.bfloat16, device="cuda", form="mx"):
        self.form = FORMS[form]

        def packed(rows, cols):
            w = torch.randn(max(experts, 1) * rows, cols, device=device) * cols ** -0.5
            return self.form.pack(w)

        self.gate_up, self.down = packed(2 * inner, hidden), packed(hidden, inner)
        self.post, self.pre = (torch.rand(hidden, device=device, dtype=dtype) + 0.5 for _ in range(2))
        self.router = torch.randn(hidden, experts, device=device, dtype=dtype) * hidden ** -0.5 if experts else None
        self.experts = experts


def norms(layer, y, h):
    """(h', packed x)"""
    if layer.form is FORMS["mx"]:
        return rz.razer_block_norm(y, h, post_weight=layer.post, pre_weight=layer.pre, packed=True)
    h, x = rz.razer_block_norm(y, h, post_weight=layer.post, pre_weight=layer.pre)
    return h, layer.form.pack(x)


def dense(layer, y, h):
    """(h', y') of one layer."""
    f = layer.form
    h, x = norms(layer, y, h)
    return h, f.gemm(f.gated(f.gemm(x, layer.gate_up, h.dtype)), layer.down, h.dtype)


def route(layer, x, top):
    """The experts of packed x."""
    logits = layer.form.values(x, layer.router.dtype) @ layer.router
    return rz.razer_moe_route(logits, top, renormalise=True)


def mixture(layer, y, h, top):
    """(h', y') of one layer of experts."""
    f = layer.form
    h, x = norms(layer, y, h)
    r = route(layer, x, top)
    gu = f.grouped(x, layer.gate_up, r.offsets, r.rows, h.dtype)
    rows = f.grouped(f.gated(gu), layer.down, r.offsets, None, torch.float32)
    return h, rz.razer_moe_combine(rows, r.slots, r.weights).to(h.dtype)


def plain(layer, y, h, top=0):
    """The layer in 32-bit torch on the decoded weights; activations are not packed,
    but for the router, whose choices would differ."""
    def rms(v, w):
        return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-5) * w.float()

    if layer.experts:
        r = route(layer, norms(layer, y, h)[1], top)
    h = h.float() + rms(y.float(), layer.post)
    x = rms(h, layer.pre)
    w1, w2 = layer.form.values(layer.gate_up), layer.form.values(layer.down)

    def feed(x, w1, w2):
        g, u = (x @ w1.T).chunk(2, -1)
        return (torch.nn.functional.silu(g) * u) @ w2.T

    if not layer.experts:
        return h, feed(x, w1, w2)
    w1, w2 = w1.view(layer.experts, -1, w1.shape[1]), w2.view(layer.experts, -1, w2.shape[1])
    out, at = torch.zeros_like(h), r.offsets.tolist()
    for e in range(layer.experts):
        s = slice(at[e], at[e + 1])
        token = r.rows[s].long()
        weight = r.weights[r.experts == e]  # in the order of tokens, as the rows are
        out.index_add_(0, token, feed(x[token], w1[e], w2[e]) * weight[:, None])
    return h, out


def run(tokens, hidden, inner, layers, experts=0, top=2, dtype=torch.bfloat16, device="cuda", form="mx"):
    """(us a layer, error of the last layer's y relative to the plain form's size)."""
    stack = [Layer(hidden, inner, experts, dtype, device, form) for _ in range(layers)]
    y0, h0 = (torch.randn(tokens, hidden, device=device, dtype=dtype) for _ in range(2))

    def step():
        y, h = y0, h0
        for layer in stack:
            last = y, h
            h, y = mixture(layer, y, h, top) if experts else dense(layer, y, h)
        return last, y

    (y_in, h_in), y = step()
    _, want = plain(stack[-1], y_in, h_in, top)
    error = float((y.float() - want).norm() / want.norm())

    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        graph.replay()
    start.record()
    for _ in range(10):
        graph.replay()
    end.record()
    end.synchronize()
    return start.elapsed_time(end) * 100 / layers, error


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("tokens", 1), ("hidden", 4096), ("inner", 14336), ("layers", 4), ("experts", 0), ("top", 2)):
        p.add_argument(f"--{name}", type=int, default=value)
    p.add_argument("--form", choices=sorted(FORMS), default="mx")
    a = p.parse_args()
    us, error = run(a.tokens, a.hidden, a.inner, a.layers, a.experts, a.top, form=a.form)
    print(f"{a.form}: {a.tokens} tokens, {a.hidden} -> {a.inner}, {a.experts or 'no'} experts: {us:.1f} us a layer, "
          f"error {error:.3f} of the 32-bit layer with unpacked activations")
