"""The 8-bit integer encoder, decoder and products against their definitions: codes,
scales and results bit for bit."""
import numpy as np
import pytest
import torch

import i8_common as ref
import nvfp4_razer_w4a16_amd as rz

pytestmark = pytest.mark.gpu
DT = ref.DT


def _same_tensor(t, codes, scales):
    ref.same(t.codes, torch.from_numpy(codes))
    ref.same(t.scales, torch.from_numpy(scales))


def _input(rows, cols, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g)
    x[:, cols // 3] *= 30
    return x.to(dtype)


# every form of the encoder: rows within a wave, 256, 512 and 1024 lanes, and longer ones, whole and partly filled
@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 512), (5, 528), (2, 2048), (7, 2064), (1, 4096), (3, 8192),
                                       (2, 8208), (1, 16384), (2, 20000), (1, 32768), (2, 32784), (1, 131056),
                                       (333, 80)])
def test_encode(rows, cols, dtype):
    x = _input(rows, cols, rows + cols, DT[dtype])
    t = rz.razer_i8_quantize(x.cuda())
    codes, scales = ref.encode(x)
    _same_tensor(t, codes, scales)
    for out in DT.values():  # code * scale, rounded to fp32, then to the type
        want = torch.from_numpy(codes.astype(np.float32) * scales[:, None]).to(out)
        ref.same(rz.razer_i8_dequant(t, out), want)


def test_encode_of_rows_in_one_buffer():
    """Rows apart, a copy where they are not 16 bytes apart, one row of a column-major tensor."""
    x = _input(9, 256, 1, torch.bfloat16).cuda()
    for v in (x[:, 64:160], x[:, 3:19], x[::2, :64], x[:, :16].t().contiguous().t(), x[2:3, 1:33]):
        _same_tensor(rz.razer_i8_quantize(v), *ref.encode(v))


@pytest.mark.parametrize("cols", [64, 4096, 40000])
def test_encode_of_special_rows(cols):
    """Zeros, one value, infinities, NaN, the ends of fp32 and rows that lie between."""
    x = torch.zeros(14, cols)
    x[1, 5] = -3.0
    x[2, 7], x[3, 8], x[4, cols - 1] = float("inf"), float("-inf"), float("nan")
    x[5] = torch.linspace(-1, 1, cols) * 2.0 ** -149
    x[6] = torch.linspace(-1, 1, cols) * 3.0e38
    x[7] = torch.linspace(-1, 1, cols) * 2.0 ** -126
    x[8] = torch.linspace(-1, 1, cols) * 2.0 ** -64
    x[9] = torch.linspace(-1, 1, cols) * np.nextafter(np.float32(2.0 ** -64), np.float32(0))
    x[10], x[11] = 1e-45, -0.0
    x[12] = torch.arange(cols) % 128 - 0.5
    x[13] = (torch.arange(cols) % 255 - 127).float()  # 127 / amax = 1: halves do not occur
    codes, scales = ref.encode(x)
    t = rz.razer_i8_quantize(x.cuda())
    _same_tensor(t, codes, scales)
    v = rz.razer_i8_dequant(t)
    assert torch.isnan(v[2:5]).all() and not torch.isnan(v[5:]).any()
    assert (v[0] == 0).all() and (v[13].cpu() == x[13]).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (4, 1040), (2, 14336), (1, 40000)])
def test_gated(rows, cols, dtype):
    """A value differs from silu(g) * u by half a step of its row and what fp32 takes: the
    exponent g * log2(e) is off by 2^-24 of itself, which exp turns into |g| 2^-24, and
    some eight roundings follow (exp, sum, quotient, product, times 127 / amax, amax's own)."""
    g = torch.Generator().manual_seed(cols)
    gu = (torch.randn(rows, 2 * cols, generator=g) * 2).to(DT[dtype])
    a, b = gu[:, :cols].double(), gu[:, cols:].double()
    want = a / (1 + torch.exp(-a)) * b
    t = rz.razer_i8_quantize_gated(gu.cuda())
    rel = (float(a.abs().max()) + 10) * 2.0 ** -23
    amax = want.abs().amax(1)
    assert ((t.scales.cpu().double() * 127 - amax).abs() <= amax * rel).all()
    off = (t.codes.cpu().double() * t.scales.cpu().double()[:, None] - want).abs()
    assert (off <= (amax / 127 * (0.5 + 127 * rel) * (1 + rel))[:, None]).all()


def test_gated_far_from_zero():
    """exp(-g) overflows to infinity far below zero: silu is zero there."""
    gu = torch.zeros(2, 64)
    gu[:, :32] = torch.linspace(-500, 500, 32)
    gu[:, 32:] = 1.0
    t = rz.razer_i8_quantize_gated(gu.cuda())
    v = rz.razer_i8_dequant(t).cpu()
    assert torch.isfinite(v).all() and (v[:, :15] == 0).all() and (t.codes[:, 31] == 127).all()


SHAPES = [(1, 1, 16), (1, 64, 32), (1, 4096, 4096), (1, 77, 14336), (2, 100, 48), (3, 129, 2064), (16, 130, 1024),
          (17, 500, 528), (27, 1000, 4096), (32, 33, 8208), (33, 257, 2048), (64, 640, 96), (65, 300, 4112),
          (100, 4096, 256), (127, 255, 272), (128, 513, 640), (200, 700, 1008), (256, 256, 512), (300, 777, 4096),
          (513, 1025, 1040), (1000, 520, 144), (40, 96, 131056)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(m, n, k):
    rng = np.random.default_rng(m * 7 + n * 3 + k)
    (x, sx), (w, sw) = ref.random_i8(rng, m, k), ref.random_i8(rng, n, k)
    dx, dw = ref.device(x, sx), ref.device(w, sw)
    for name, dtype in DT.items():
        want = ref.product(x, sx, w, sw, dtype)
        ref.same(rz.razer_i8_gemm(dx, dw, dtype), want)
        out = torch.full((m + 1, n), 7.0, dtype=dtype, device="cuda")
        rz.razer_i8_gemm(dx, dw, out=out[:m])
        ref.same(out[:m], want)
        assert (out[m] == 7.0).all()


@pytest.mark.parametrize("m,n,k", [(1, 16, 131056), (5, 40, 65536), (300, 300, 131056)])
def test_largest_sums(m, n, k):
    """Codes of one sign and -128, which the encoder does not write: 2^14 * 131056 < 2^31."""
    x, w = np.full((m, k), -128, dtype=np.int8), np.full((n, k), -128, dtype=np.int8)
    w[1::2] = 127
    sx, sw = np.ones(m, dtype=np.float32), np.full(n, 2.0 ** -20, dtype=np.float32)
    ref.same(rz.razer_i8_gemm(ref.device(x, sx), ref.device(w, sw), torch.float32),
             ref.product(x, sx, w, sw, torch.float32))


@pytest.mark.parametrize("m,n,k", [(3, 40, 96), (20, 70, 1040), (300, 300, 1040)])
def test_scales_that_are_not_finite(m, n, k):
    rng = np.random.default_rng(m)
    (x, sx), (w, sw) = ref.random_i8(rng, m, k), ref.random_i8(rng, n, k)
    sx[0], sx[1], sx[2], sw[3], sw[5], sw[n - 1] = np.nan, 0.0, 1e38, np.nan, 1e-40, np.inf
    x[m - 1] = 0
    for dtype in DT.values():
        ref.same(rz.razer_i8_gemm(ref.device(x, sx), ref.device(w, sw), dtype), ref.product(x, sx, w, sw, dtype))


def test_product_of_nothing():
    x, w = rz.I8Tensor(0, 64, "cuda"), rz.razer_i8_quantize(torch.ones(5, 64, device="cuda"))
    assert rz.razer_i8_gemm(x, w).shape == (0, 5)
    assert rz.razer_i8_gemm(w, x).shape == (5, 0)
    t = rz.razer_i8_quantize(torch.empty(0, 64, device="cuda"))
    assert t.shape == (0, 64) and rz.razer_i8_dequant(t).shape == (0, 64)


def _grouped(sizes, n, k, seed, tokens=None, dtype=torch.bfloat16, gap=0):
    """Products of runs of `sizes` rows, `gap` rows behind the last; rows gathered from `tokens` tokens."""
    rng = np.random.default_rng(seed)
    e, total = len(sizes), sum(sizes)
    m = total + gap
    (x, sx), (w, sw) = ref.random_i8(rng, tokens or m, k), ref.random_i8(rng, e * n, k)
    offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    rows = None
    if tokens:
        rows = rng.integers(0, tokens, m).astype(np.int32)
        rows[rng.random(m) < 0.1] = -1
        rows[rng.random(m) < 0.05] = tokens + 3
    want = torch.full((m, n), 7.0, dtype=dtype)
    for i in range(e):
        a, b = offsets[i], offsets[i + 1]
        r = np.arange(a, b) if rows is None else rows[a:b]
        ok = (r >= 0) & (r < (tokens or m))
        part = ref.product(x[r * ok], sx[r * ok], w[i * n:(i + 1) * n], sw[i * n:(i + 1) * n], dtype)
        part[~torch.from_numpy(ok)] = 0.0
        want[a:b] = part
    out = torch.full((m, n), 7.0, dtype=dtype, device="cuda")
    rz.razer_i8_gemm_grouped(ref.device(x, sx), ref.device(w, sw), torch.from_numpy(offsets).cuda(),
                             None if rows is None else torch.from_numpy(rows).cuda(), out=out)
    ref.same(out, want)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("sizes,n,k", [
    ([1], 40, 32), ([0, 1, 0, 0, 2], 33, 528), ([3, 0, 5, 1, 0, 0, 7], 300, 2064), ([1] * 70, 64, 96),
    ([2, 2, 3, 1, 0, 4, 2, 2], 1000, 4096), ([100, 0, 31, 65, 1], 257, 1040), ([0, 0, 0], 8, 64),
    ([300, 200, 0, 129], 520, 640), ([17] * 100, 96, 208), ([700, 1, 600], 256, 4096), ([5] * 130, 24, 48)])
def test_experts(sizes, n, k, gather):
    for i, (name, dtype) in enumerate(DT.items()):
        _grouped(sizes, n, k, i + n, tokens=37 if gather else None, dtype=dtype, gap=3)


def test_experts_with_offsets_that_do_not_ascend():
    """Offsets outside [0, M], or that go back: clamped; nothing outside y is written."""
    rng = np.random.default_rng(3)
    n, k, m = 40, 64, 20
    (x, sx), (w, sw) = ref.random_i8(rng, m, k), ref.random_i8(rng, 3 * n, k)
    for offsets in ([-5, 4, 9, 99], [6, 2, 2, 20], [30, 40, 50, 60], [-9, -8, -7, -6]):
        out = torch.full((m + 8, n), 7.0, device="cuda")
        rz.razer_i8_gemm_grouped(ref.device(x, sx), ref.device(w, sw), torch.tensor(offsets, dtype=torch.int32).cuda(),
                                 out=out[4:m + 4])
        lo = [min(max(o, 0), m) for o in offsets]
        want = torch.full((m, n), 7.0)
        for e in range(3):
            if lo[e + 1] > lo[e]:
                want[lo[e]:lo[e + 1]] = ref.product(x[lo[e]:lo[e + 1]], sx[lo[e]:lo[e + 1]], w[e * n:(e + 1) * n],
                                                    sw[e * n:(e + 1) * n], torch.float32)
        ref.same(out[4:m + 4], want)
        assert (out[:4] == 7.0).all() and (out[m + 4:] == 7.0).all()


def test_scales_of_the_first_token_do_not_reach_padding():
    """A padding row is zero also where the rows that stand in for it are NaN."""
    rng = np.random.default_rng(4)
    (x, sx), (w, sw) = ref.random_i8(rng, 4, 64), ref.random_i8(rng, 24, 64)
    sx[:] = np.nan
    sw[3] = np.inf
    for copies in (3, 300):
        rows = torch.full((copies,), -1, dtype=torch.int32).cuda()
        y = rz.razer_i8_gemm_grouped(ref.device(x, sx), ref.device(w, sw),
                                     torch.tensor([0, copies], dtype=torch.int32).cuda(), rows)
        assert (y == 0).all()


def test_scales_that_require_a_gradient():
    """There is no backward: results are in the graph of such scales, and raise there."""
    x, w = rz.razer_i8_quantize(torch.randn(6, 64, device="cuda")), rz.razer_i8_quantize(torch.randn(48, 64, device="cuda"))
    offsets = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    leaf = rz.I8Tensor.of(w.codes, w.scales.clone().requires_grad_())
    for result, want in ((rz.razer_i8_gemm(x, leaf), rz.razer_i8_gemm(x, w)),
                         (rz.razer_i8_gemm_grouped(x, leaf, offsets), rz.razer_i8_gemm_grouped(x, w, offsets)),
                         (rz.razer_i8_dequant(leaf), rz.razer_i8_dequant(w))):
        assert torch.equal(result, want) and result.requires_grad and not want.requires_grad
        with pytest.raises(RuntimeError, match="no backward"):
            result.sum().backward()
    out = torch.empty(6, 48, dtype=torch.bfloat16, device="cuda")
    assert not rz.razer_i8_gemm(x, leaf, out=out).requires_grad
    with torch.no_grad():
        assert not rz.razer_i8_gemm(x, leaf).requires_grad
