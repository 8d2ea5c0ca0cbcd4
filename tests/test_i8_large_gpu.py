"""Tensors of more than 2^32 bytes or elements: what lies behind that many is read and
written where it belongs."""
import pytest
import torch

import i8_common as ref
import nvfp4_razer_w4a16_amd as rz

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


def _codes(rows, cols, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c = torch.randint(-128, 128, (rows, cols), generator=gen, device="cuda", dtype=torch.int8).clamp_(-127)
    return c, torch.exp(torch.randn(rows, generator=gen, device="cuda") - 5)


def _product(x, sx, w, sw, dtype):
    return ((x.double() @ w.double().t()).float() * sx[:, None] * sw).to(dtype)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("tokens", [24, 3000])  # streamed, and on tiles
def test_weights(tokens, gather):
    n, k, experts = 70000, 8192, 8  # 4.6 GB of codes
    w, sw = _codes(experts * n, k, 1)
    x, sx = _codes(tokens, k, 2)
    off = [0, tokens // 3, tokens // 3, tokens // 3, tokens // 2, tokens // 2, tokens // 2, tokens // 2, tokens]
    rows = torch.arange(tokens - 1, -1, -1, device="cuda") if gather else torch.arange(tokens, device="cuda")
    y = rz.razer_i8_gemm_grouped(rz.I8Tensor.of(x, sx), rz.I8Tensor.of(w, sw), torch.tensor(off, dtype=torch.int32).cuda(),
                                 rows.int() if gather else None, torch.float16)
    for e in (0, 3, 7):
        for a, b in ((0, 300), (n - 300, n)):  # the first columns and the last
            s, c = slice(off[e], off[e + 1]), slice(e * n + a, e * n + b)
            ref.same(y[s, a:b], _product(x[rows[s]], sx[rows[s]], w[c], sw[c], torch.float16))


@pytest.mark.parametrize("n", [20, 3000])  # streamed, and on tiles
def test_rows(n):
    m, k = 300000, 16384  # 4.9 GB of codes
    x, sx = _codes(m, k, 3)
    w, sw = _codes(n, k, 4)
    y = rz.razer_i8_gemm(rz.I8Tensor.of(x, sx), rz.I8Tensor.of(w, sw))
    for s in (slice(0, 200), slice(m - 200, m)):
        ref.same(y[s], _product(x[s], sx[s], w, sw, torch.bfloat16))


def test_results():
    m, n, k = 70000, 65600, 32  # 2^32 results and more
    (x, sx), (w, sw) = _codes(m, k, 5), _codes(n, k, 6)
    y = rz.razer_i8_gemm(rz.I8Tensor.of(x, sx), rz.I8Tensor.of(w, sw))
    for s in (slice(0, 100), slice(m - 100, m)):
        ref.same(y[s], _product(x[s], sx[s], w, sw, torch.bfloat16))


def test_encode_and_decode():
    rows, cols = 70000, 65536
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    for s in (slice(0, 2), slice(rows - 2, rows)):
        x[s] = torch.randn(2, cols, device="cuda")
    t = rz.razer_i8_quantize(x)
    v = rz.razer_i8_dequant(t, torch.bfloat16)
    for s in (slice(0, 2), slice(rows - 2, rows)):
        codes, scales = ref.encode(x[s])
        ref.same(t.codes[s], torch.from_numpy(codes))
        ref.same(t.scales[s], torch.from_numpy(scales))
        ref.same(v[s], (t.codes[s].float() * t.scales[s, None]).bfloat16())


def test_combine():
    rows, cols = 70000, 65536
    y = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    y[-3:] = torch.randn(3, cols, device="cuda")
    slots = torch.tensor([[rows - 1, rows - 3], [rows - 2, -1]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, 0.25], [1.0, 3.0]], device="cuda")
    got = rz.razer_moe_combine(y, slots, w)
    ref.same(got[1], y[rows - 2])
    ref.same(got[0], (0.5 * y[-1].float() + 0.25 * y[-3].float()).bfloat16())


@pytest.mark.parametrize("tokens,experts,top", [(1 << 20, 8, 2), (600000, 256, 8)])
def test_route(tokens, experts, top):
    gen = torch.Generator(device="cuda").manual_seed(7)
    l = torch.randn(tokens, experts, generator=gen, device="cuda")
    r = rz.razer_moe_route(l, top)
    chosen = r.experts.reshape(-1).long()
    at = torch.argsort(chosen, stable=True)
    assert torch.equal(r.rows.long(), at // top)
    slots = torch.empty_like(at)
    slots[at] = torch.arange(tokens * top, device="cuda")
    assert torch.equal(r.slots.reshape(-1).long(), slots)
    assert torch.equal(r.offsets.long(), torch.searchsorted(chosen[at].contiguous(), torch.arange(experts + 1, device="cuda")))
    best = torch.sort(l, dim=1, descending=True, stable=True)[1][:, :top]
    assert torch.equal(r.experts.long(), best)
