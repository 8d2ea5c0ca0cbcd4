"""The feed-forward half of a transformer block with MXFP4 weights and activations,
dense or as a mixture of experts:

    python examples/mx_block.py [--tokens 1] [--hidden 4096] [--inner 14336] [--layers 4]
                                [--experts 0] [--top 2]

``y`` is what the block's attention gave, ``h`` the residual.  A layer is four
launches for the dense form: residual and both norms with the packing of x, the gate
and up projections as one product, silu(gate) * up with its packing, the down
projection.  The layers are captured in a graph and replayed; the last layer is
compared with the same layer in 32-bit torch on the decoded weights.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), os.pardir))
import nvfp4_razer_w4a16_amd as rz  # noqa: E402


class Layer:
    """Random weights of one layer, packed once; experts' weights are stacked by rows."""

    def __init__(self, hidden, inner, experts=0, dtype=torch.bfloat16, device="cuda"):
        def packed(rows, cols):
            w = torch.randn(max(experts, 1) * rows, cols, device=device) * cols ** -0.5
            return rz.razer_mx_quantize(w)

        self.gate_up, self.down = packed(2 * inner, hidden), packed(hidden, inner)
        self.post, self.pre = (torch.rand(hidden, device=device, dtype=dtype) + 0.5 for _ in range(2))
        self.router = torch.randn(hidden, experts, device=device, dtype=dtype) * hidden ** -0.5 if experts else None
        self.experts = experts


def dense(layer, y, h):
    """(h', y') of one layer."""
    h, x = rz.razer_block_norm(y, h, post_weight=layer.post, pre_weight=layer.pre, packed=True)
    gu = rz.razer_mx_gemm(x, layer.gate_up, h.dtype)
    return h, rz.razer_mx_gemm(rz.razer_mx_quantize_gated(gu), layer.down, h.dtype)


def route(layer, x, top):
    """(offsets, token of every sorted row, its weight): rows sorted by expert."""
    p, e = torch.topk(torch.softmax(x @ layer.router, -1, dtype=torch.float32), top)
    order = torch.argsort(e.reshape(-1), stable=True)
    offsets = torch.searchsorted(e.reshape(-1)[order].contiguous(),
                                 torch.arange(layer.experts + 1, device=x.device)).int()
    return offsets, (order // top).int(), (p / p.sum(-1, keepdim=True)).reshape(-1)[order]


def mixture(layer, y, h, top):
    """(h', y') of one layer of experts."""
    h, x = rz.razer_block_norm(y, h, post_weight=layer.post, pre_weight=layer.pre, packed=True)
    offsets, token, weight = route(layer, rz.razer_mx_dequant(x, h.dtype), top)
    gu = rz.razer_mx_gemm_grouped(x, layer.gate_up, offsets, token, h.dtype)
    rows = rz.razer_mx_gemm_grouped(rz.razer_mx_quantize_gated(gu), layer.down, offsets, None, torch.float32)
    y = torch.zeros(h.shape, device=h.device).index_add_(0, token, rows * weight[:, None])
    return h, y.to(h.dtype)


def plain(layer, y, h, top=0):
    """The layer in 32-bit torch on the decoded weights; activations are not packed,
    but for the router, whose choices would differ."""
    def rms(v, w):
        return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-5) * w.float()

    if layer.experts:
        _, x = rz.razer_block_norm(y, h, post_weight=layer.post, pre_weight=layer.pre, packed=True)
        offsets, token, weight = route(layer, rz.razer_mx_dequant(x, h.dtype), top)
    h = h.float() + rms(y.float(), layer.post)
    x = rms(h, layer.pre)
    w1, w2 = rz.razer_mx_dequant(layer.gate_up), rz.razer_mx_dequant(layer.down)

    def feed(x, w1, w2):
        g, u = (x @ w1.T).chunk(2, -1)
        return (torch.nn.functional.silu(g) * u) @ w2.T

    if not layer.experts:
        return h, feed(x, w1, w2)
    w1, w2 = w1.view(layer.experts, -1, w1.shape[1]), w2.view(layer.experts, -1, w2.shape[1])
    out, at = torch.zeros_like(h), offsets.tolist()
    for e in range(layer.experts):
        s = slice(at[e], at[e + 1])
        out.index_add_(0, token[s], feed(x[token[s].long()], w1[e], w2[e]) * weight[s, None])
    return h, out


def run(tokens, hidden, inner, layers, experts=0, top=2, dtype=torch.bfloat16, device="cuda"):
    """(us a layer, error of the last layer's y relative to the plain form's size)."""
    stack = [Layer(hidden, inner, experts, dtype, device) for _ in range(layers)]
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
    replay = step
    if not experts:  # the router's sort is torch's
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        replay = graph.replay
    for _ in range(3):
        replay()
    start.record()
    for _ in range(10):
        replay()
    end.record()
    end.synchronize()
    return start.elapsed_time(end) * 100 / layers, error


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("tokens", 1), ("hidden", 4096), ("inner", 14336), ("layers", 4), ("experts", 0), ("top", 2)):
        p.add_argument(f"--{name}", type=int, default=value)
    a = p.parse_args()
    us, error = run(a.tokens, a.hidden, a.inner, a.layers, a.experts, a.top)
    print(f"{a.tokens} tokens, {a.hidden} -> {a.inner}, {a.experts or 'no'} experts: {us:.1f} us a layer, "
          f"error {error:.3f} of the 32-bit layer with unpacked activations")
