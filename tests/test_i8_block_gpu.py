"""The layers of ``examples/mx_block.py`` in 8-bit integers and with the library's routing,
and the calls as a program makes them: captured and replayed, on another stream, at once."""
import pytest
import torch

import nvfp4_razer_w4a16_amd as rz
from test_mx_block_gpu import block

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,hidden,inner,experts,top", [(1, 512, 1056, 0, 2), (70, 256, 544, 0, 2),
                                                             (5, 256, 320, 4, 2), (90, 512, 544, 16, 3),
                                                             (700, 256, 272, 4, 2)])
def test_layer(tokens, hidden, inner, experts, top, dtype):
    """Rounding a normal row to 8 bits errs by 0.29 of a step of its largest element / 127,
    3.1 to 3.5 standard deviations here: 0.008.  Of x it reaches g and u, of silu(g) * u, whose
    largest element lies further out, some 0.02: together below 0.03.  The fp types between
    add 2^-8 a few times.  A wrong layer is off by 1 or more."""
    torch.manual_seed(tokens)
    us, error = block.run(tokens, hidden, inner, 2, experts, top, dtype, form="i8")
    assert us > 0
    assert error < 0.06


def _layer(x, logits, w1, w2, h, top):
    r = rz.razer_moe_route(logits, top, score="sigmoid", renormalise=True)
    gu = rz.razer_i8_gemm_grouped(rz.razer_i8_quantize(x), w1, r.offsets, r.rows, x.dtype)
    rows = rz.razer_i8_gemm_grouped(rz.razer_i8_quantize_gated(gu), w2, r.offsets, None, x.dtype)
    return [*r, rz.razer_moe_combine(rows, r.slots, r.weights, add=h)]


def _data(tokens, experts, hidden, inner, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    w1 = rz.razer_i8_quantize(n(experts * 2 * inner, hidden) * hidden ** -0.5)
    w2 = rz.razer_i8_quantize(n(experts * hidden, inner) * inner ** -0.5)
    return n(tokens, hidden).bfloat16(), n(tokens, experts), w1, w2, n(tokens, hidden).bfloat16()


# one workgroup's route and streamed products; routes by blocks, tiles; rows of K slices
@pytest.mark.parametrize("tokens,experts,top,hidden,inner", [(1, 8, 2, 256, 272), (37, 8, 2, 512, 96),
                                                             (1500, 4, 2, 256, 512)])
def test_captured_and_replayed(tokens, experts, top, hidden, inner):
    """Every replay on new inputs gives what the eager calls give, also with eager work and
    other replays between them; two graphs have workspaces of their own."""
    data = [_data(tokens, experts, hidden, inner, i) for i in range(3)]
    want = [_layer(*d, top) for d in data]
    graphs = []
    for _ in range(2):
        held = [t.clone() if isinstance(t, torch.Tensor) else rz.I8Tensor.of(t.codes.clone(), t.scales.clone())
                for t in data[0]]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = _layer(*held, top)
        graphs.append((graph, held, out))
    streams = [torch.cuda.Stream() for _ in graphs]
    for turn in range(4):
        torch.cuda.synchronize()
        for i, (graph, held, out) in enumerate(graphs):
            d = data[(turn + i) % 3]
            with torch.cuda.stream(streams[i]):
                for at in (0, 1, 4):
                    held[at].copy_(d[at])
                for at in (2, 3):
                    held[at].codes.copy_(d[at].codes), held[at].scales.copy_(d[at].scales)
                graph.replay()
        _layer(*data[turn % 3], top)  # eager, beside them
        torch.cuda.synchronize()
        for i, (_, _, out) in enumerate(graphs):
            assert all(torch.equal(a, b) for a, b in zip(out, want[(turn + i) % 3])), (turn, i)


@pytest.mark.parametrize("m,n,k", [(1, 500, 4096), (300, 2000, 640), (260, 300, 16384), (2048, 3600, 512)])
def test_products_at_once(m, n, k):
    """The same product on several streams at once, each with its own workspace."""
    g = torch.Generator(device="cuda").manual_seed(m)
    x = rz.razer_i8_quantize(torch.randn(m, k, generator=g, device="cuda"))
    w = rz.razer_i8_quantize(torch.randn(n, k, generator=g, device="cuda"))
    want = rz.razer_i8_gemm(x, w)
    torch.cuda.synchronize()
    got = []
    for s in [torch.cuda.Stream() for _ in range(4)]:
        for _ in range(3):
            got.append(rz.razer_i8_gemm(x, w, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(t, want) for t in got)


def test_given_stream():
    """A call on a given stream orders the copies and the workspace it makes with its
    launch, behind work that stream still has to do."""
    tokens, experts, cols = 300, 16, 4096
    g = torch.Generator(device="cuda").manual_seed(0)
    wide = torch.randn(tokens, cols + 1, generator=g, device="cuda")
    x = wide[:, 1:]  # rows that the call has to copy
    want_t, want_r = rz.razer_i8_quantize(x), rz.razer_moe_route(x[:, :experts], 3)
    want_g = rz.razer_i8_quantize_gated(x)
    w = rz.razer_i8_quantize(torch.randn(200, cols, generator=g, device="cuda"))
    want_y = rz.razer_i8_gemm(want_t, w)
    want_c = rz.razer_moe_combine(want_y.repeat(3, 1), want_r.slots, want_r.weights)
    stack = rz.razer_i8_quantize(torch.randn(experts * 32, cols, generator=g, device="cuda"))
    want_e = rz.razer_i8_gemm_grouped(want_t, stack, want_r.offsets, want_r.rows)
    late = torch.zeros_like(wide)
    torch.cuda.synchronize()
    for stream in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        with rz.mx._entered(stream):
            late.zero_()
            busy = torch.randn(4096, 4096, device="cuda")
            for _ in range(10):
                busy = (busy @ busy).clamp_(-1, 1)
            late.copy_(wide)
        t = rz.razer_i8_quantize(late[:, 1:], stream=stream)
        q = rz.razer_i8_quantize_gated(late[:, 1:], stream=stream)
        r = rz.razer_moe_route(late[:, 1:experts + 1], 3, stream=stream)
        y = rz.razer_i8_gemm(t, w, stream=stream)
        e = rz.razer_i8_gemm_grouped(t, stack, r.offsets, r.rows, stream=stream)
        v = rz.razer_i8_dequant(t, stream=stream)
        with rz.mx._entered(stream):
            rows = y.repeat(3, 1)
        c = rz.razer_moe_combine(rows, r.slots, r.weights, stream=stream)
        torch.cuda.synchronize()
        for a, b in ((t, want_t), (q, want_g)):
            assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
        assert all(torch.equal(a, b) for a, b in zip(r, want_r))
        assert torch.equal(y, want_y) and torch.equal(e, want_e) and torch.equal(c, want_c)
        assert torch.equal(v, rz.razer_i8_dequant(want_t))
