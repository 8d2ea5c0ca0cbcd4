"""MXFP4 operators and the block norm on the GPU, against their definitions in
64 bits (mx_common)."""
import numpy as np
import pytest
import torch

import mx_common as mx
import nvfp4_razer_w4a16_amd as rz

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")]
DT = mx.DT


def assert_encoded(t, code, byte):
    assert np.array_equal(t.scales.cpu().numpy(), byte)
    assert np.array_equal(t.codes.cpu().numpy(), mx.pack(code))


def values(rng, rows, cols, dt):
    """Normal values whose blocks spread over the type's exponents, some blocks zero."""
    lo, hi = {"f32": (-140, 120), "f16": (-20, 12), "bf16": (-125, 120)}[dt]
    e = rng.integers(lo, hi, (rows, cols // 32, 1))
    v = rng.standard_normal((rows, cols // 32, 32)) * np.exp2(e * 1.0)
    v[rng.random(v.shape[:2]) < 0.05] = 0.0
    return torch.from_numpy(v.reshape(rows, cols)).to(DT[dt])


# ---- encode / decode ---------------------------------------------------------

@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 4096), (3, 96), (7, 2080), (129, 1504), (1000, 64)])
def test_encode_bytes(rows, cols, dt):
    x = values(np.random.default_rng(rows * cols), rows, cols, dt)
    code, byte = mx.encode(x.double().numpy())
    t = rz.razer_mx_quantize(x.cuda())
    assert_encoded(t, code, byte)
    for out in DT.values():
        want = torch.from_numpy(mx.decode(code, byte)).to(out)
        assert torch.equal(rz.razer_mx_dequant(t, out).cpu(), want)


@pytest.mark.parametrize("dt", DT)
def test_encode_every_16_bit_value(dt):
    """Every 16-bit value (for f32, every value with those upper bits) beside block
    maxima of every relevant size: all roundings, ties, subnormals and signs."""
    bits = torch.arange(65536, dtype=torch.int32)
    if dt == "f32":
        v = (bits << 16).view(torch.float32)
    else:
        v = bits.to(torch.int16).view(DT[dt])
    v = v[torch.isfinite(v.float())]
    keep = v.shape[0] // 31 * 31
    rows = []
    for shift in range(0, 6):  # the block's largest magnitude, up to 32 times its other values
        b = v[:keep].reshape(-1, 31).double()
        top = b.abs().amax(1, keepdim=True) * 2.0 ** shift
        rows.append(torch.cat([b, top], 1).to(DT[dt]))
    x = torch.cat(rows)
    x = x[torch.isfinite(x.float()).all(1)]
    code, byte = mx.encode(x.double().numpy())
    assert_encoded(rz.razer_mx_quantize(x.cuda()), code, byte)


@pytest.mark.parametrize("dt", DT)
def test_encode_halfway_points(dt):
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.5])
    x = np.zeros((24, 32))
    for r in range(24):
        x[r, :9], x[r, 9:18] = mids, -mids
        x[r, 18] = 4.0 if r % 2 else 7.9375  # scale 1 in either case
        x[r] *= 2.0 ** (r - 12)
    x = torch.from_numpy(x).to(DT[dt])
    code, byte = mx.encode(x.double().numpy())
    assert_encoded(rz.razer_mx_quantize(x.cuda()), code, byte)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_encode_not_finite(dt, bad):
    x = values(np.random.default_rng(5), 4, 256, dt)
    x[1, 40], x[3, 255] = bad, bad
    code, byte = mx.encode(x.double().numpy())
    assert (byte == 255).sum() == 2
    t = rz.razer_mx_quantize(x.cuda())
    assert_encoded(t, code, byte)
    v = rz.razer_mx_dequant(t).cpu().numpy()
    assert np.isnan(v[1, 32:64]).all() and np.isnan(v[3, 224:]).all() and np.isfinite(v[0]).all()


def test_decode_every_byte():
    byte = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 1, 1)
    code = np.tile(np.arange(32, dtype=np.uint8) % 16, (256, 1))
    t = mx.device(code, byte)
    with np.errstate(over="ignore"):
        want = mx.decode(code, byte)
    for out in DT.values():
        got = rz.razer_mx_dequant(t, out).cpu()
        assert torch.equal(torch.nan_to_num(got, nan=123.0), torch.nan_to_num(torch.from_numpy(want).to(out), nan=123.0))


@pytest.mark.parametrize("dt", DT)
def test_encode_strides(dt):
    """A column slice is read in place; other orders are copied."""
    x = values(np.random.default_rng(9), 33, 320, dt).cuda()
    for v in (x[:, 64:192], x[::2, :], x[:, 4:36], x.t()[:, :32].t().contiguous().t().t()):
        code, byte = mx.encode(v.double().cpu().numpy())
        assert_encoded(rz.razer_mx_quantize(v), code, byte)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("rows,cols", [(1, 32), (5, 1056), (64, 4096)])
def test_gated_encode(rows, cols, dt):
    """silu(g) * u carries a few fp32 roundings, so a value may fall to the other
    side of a rounding point only where it is within 2^-20 of it."""
    rng = np.random.default_rng(rows)
    gu = torch.from_numpy(rng.standard_normal((rows, 2 * cols)) * 3).to(DT[dt])
    gu[0, :4] = torch.tensor([0.0, -80.0, 80.0, -30.0], dtype=DT[dt])
    g, u = gu.double().numpy()[:, :cols], gu.double().numpy()[:, cols:]
    p = g / (1 + np.exp(-g)) * u
    t = rz.razer_mx_quantize_gated(gu.cuda())
    got = rz.razer_mx_dequant(t).double().cpu().numpy()
    lo, hi = (mx.decode(*mx.encode(p * (1 + s * 2.0 ** -20))) for s in (-1, 1))
    code, byte = mx.encode(p)
    want = mx.decode(code, byte)
    assert ((got == want) | (got == lo) | (got == hi)).all()
    assert (got == want).mean() > 0.999


# ---- product -----------------------------------------------------------------

SHAPES = [(1, 1, 32), (1, 64, 4096), (1, 4097, 160), (2, 130, 96), (5, 33, 2080), (16, 256, 512), (17, 100, 1024),
          (31, 4096, 288), (33, 1503, 2080), (64, 512, 4128), (65, 31, 14336), (128, 128, 256), (129, 257, 320),
          (200, 1000, 8192), (257, 513, 736), (300, 2048, 1024), (512, 384, 4096), (700, 1100, 96)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(m, n, k):
    rng = np.random.default_rng(m + n + k)
    x, w = mx.random_mx(rng, m, k), mx.random_mx(rng, n, k)
    want, norm = mx.product(mx.decode(*x), mx.decode(*w))
    for dt in DT.values():
        got = rz.razer_mx_gemm(mx.device(*x), mx.device(*w), dt)
        mx.assert_product(got, want, norm, k, (m, n, k, dt))


@pytest.mark.parametrize("m", [1, 3, 40, 300])
def test_product_scale_range(m):
    """Scales at both ends of their range, whose products are ordinary numbers."""
    rng = np.random.default_rng(m)
    n, k = 96, 544
    x, w = mx.random_mx(rng, m, k, 0, 6), mx.random_mx(rng, n, k, 248, 255)
    want, norm = mx.product(mx.decode(*x), mx.decode(*w))
    got = rz.razer_mx_gemm(mx.device(*x), mx.device(*w), torch.float32)
    mx.assert_product(got, want, norm, k)


@pytest.mark.parametrize("m", [1, 20, 290])
def test_product_nan_scale(m):
    """A NaN block makes its row of x, or its column of y, NaN and nothing else."""
    rng = np.random.default_rng(m)
    n, k = 200, 1056
    (xc, xb), (wc, wb) = mx.random_mx(rng, m, k), mx.random_mx(rng, n, k)
    xb[m - 1, 32], wb[77, 5], wb[n - 1, 32] = 255, 255, 255
    want, norm = mx.product(mx.decode(xc, xb), mx.decode(wc, wb))
    got = rz.razer_mx_gemm(mx.device(xc, xb), mx.device(wc, wb), torch.float32)
    assert np.isnan(want).sum() == n + 2 * (m - 1)
    mx.assert_product(got, want, norm, k)


def test_product_guards():
    """Nothing past the output is written, at widths that end inside a tile."""
    rng = np.random.default_rng(1)
    for m, n, k in ((1, 33, 64), (19, 1001, 96), (130, 129, 288)):
        x, w = mx.random_mx(rng, m, k), mx.random_mx(rng, n, k)
        buf = torch.full((m * n + 4096,), 7.0, dtype=torch.bfloat16, device="cuda")
        rz.razer_mx_gemm(mx.device(*x), mx.device(*w), out=buf[:m * n].view(m, n))
        assert (buf[m * n:] == 7.0).all()


# ---- grouped product ---------------------------------------------------------

GROUPS = [
    (40, 128, [3]),
    (64, 160, [0, 0, 5, 0]),
    (33, 4096, [1, 0, 2, 1]),
    (130, 288, [17, 0, 1, 40, 6]),
    (96, 512, [0, 130, 3, 0, 260, 129]),
    (257, 1056, [200, 1, 90]),
    (31, 96, [i % 4 for i in range(130)]),
    (64, 2080, [64] * 9),
]


@pytest.mark.parametrize("n,k,sizes", GROUPS)
@pytest.mark.parametrize("gather", [False, True])
def test_grouped(n, k, sizes, gather):
    rng = np.random.default_rng(n + k)
    e, m = len(sizes), sum(sizes)
    tokens = max(1, m // 3) if gather else m
    x, w = mx.random_mx(rng, tokens, k), mx.random_mx(rng, e * n, k)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    rows = rng.integers(0, tokens, m).astype(np.int32)
    xv, wv = mx.decode(*x), mx.decode(*w)
    src = xv[rows] if gather else xv
    want, norm = np.zeros((m, n)), np.zeros((m, n))
    for i in range(e):
        s = slice(off[i], off[i + 1])
        want[s], norm[s] = mx.product(src[s], wv[i * n:(i + 1) * n])
    for dt in DT.values():
        got = rz.razer_mx_gemm_grouped(mx.device(*x), mx.device(*w), torch.from_numpy(off).cuda(),
                                       torch.from_numpy(rows).cuda() if gather else None, dt)
        mx.assert_product(got, want, norm, k, (n, k, dt))


@pytest.mark.parametrize("m", [8, 400])
def test_grouped_padding_and_open_rows(m):
    """Row numbers outside x give zero rows (whatever a NaN row of x holds), rows
    outside every run keep what they held, and offsets outside [0, M] are clamped."""
    rng = np.random.default_rng(m)
    n, k, tokens = 48, 320, 5
    (xc, xb), w = mx.random_mx(rng, tokens, k), mx.random_mx(rng, 3 * n, k)
    xb[0, 0] = xb[4, 3] = 255  # the rows that clamped numbers would read
    rows = rng.integers(1, 4, m).astype(np.int32)
    rows[::3], rows[1::7] = -1, 5
    last = m - 2
    off = np.array([-9, m // 2, m // 2, last], np.int32)
    want, norm = np.full((m, n), 7.0), np.zeros((m, n))
    xv, wv = mx.decode(xc, xb), mx.decode(*w)
    for i in range(last):
        ex = 0 if i < m // 2 else 2
        if rows[i] in (-1, 5):
            want[i] = 0
        else:
            a, b = mx.product(xv[rows[i]][None], wv[ex * n:(ex + 1) * n])
            want[i], norm[i] = a[0], b[0]
    out = torch.full((m, n), 7.0, device="cuda")
    rz.razer_mx_gemm_grouped(mx.device(xc, xb), mx.device(*w), torch.from_numpy(off).cuda(),
                             torch.from_numpy(rows).cuda(), out=out)
    mx.assert_product(out, want, norm, k)
    off[3] = m + 1000
    got = rz.razer_mx_gemm_grouped(mx.device(xc, xb), mx.device(*w), torch.from_numpy(off).cuda(),
                                   torch.from_numpy(rows).cuda(), torch.float32)
    assert torch.equal(got[:last], out[:last])


# ---- block norm --------------------------------------------------------------

def _norm_case(rng, rows, cols, dt, gates):
    t = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(DT[dt])  # noqa: E731
    return dict(y=t(rows, cols) * 4, h=t(rows, cols), post=t(cols), pre=t(cols), gate=t(gates, cols) if gates else None)


def _f64(t):
    return None if t is None else t.double().cpu().numpy()


def _close(got, want, size, dt):
    """64 roundings of fp32 (a lane's sums, the tree, the root and the products)
    against the magnitudes that were added, and the output's own rounding."""
    got = _f64(got)
    bound = 64 * 2.0 ** -24 * size + mx.HALF_ULP[dt] * np.abs(want) * 1.01 + mx.TINY[dt]
    assert (np.abs(got - want) <= bound).all(), np.abs(got - want).max()


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("rows,cols,gates", [(1, 32, 0), (1, 4096, 1), (3, 544, 3), (6, 1024, 2), (5, 1056, 0),
                                             (9, 2048, 9), (4, 4128, 2), (2, 8192, 0), (2, 8224, 1), (3, 16416, 0),
                                             (1, 32768, 1), (130, 512, 10)])
def test_block_norm(rows, cols, gates, dt):
    c = _norm_case(np.random.default_rng(cols), rows, cols, dt, gates)
    d = {k: None if v is None else v.cuda() for k, v in c.items()}
    y, h, post, pre, gate = (_f64(c[k]) for k in ("y", "h", "post", "pre", "gate"))
    for norm_y in (True, False):
        wh, wx = mx.block_norm(y, h, post, norm_y, gate, 0.75, pre, 1e-5)
        size = np.abs(h) + np.abs(wh - h)
        gh, gx = rz.razer_block_norm(d["y"], d["h"], post_weight=d["post"], post_norm=norm_y, gate=d["gate"],
                                     residual_scale=0.75, pre_weight=d["pre"])
        _close(gh, wh, size, DT[dt])
        root = np.sqrt((wh * wh).mean(-1, keepdims=True) + 1e-5)
        _close(gx, wx, (size + np.abs(wh) * (size / root).max(-1, keepdims=True) + np.abs(wh)) / root * np.abs(pre), DT[dt])


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("rows,cols", [(1, 32), (5, 1056), (3, 4096), (2, 16384)])
def test_block_norm_packed(rows, cols, dt):
    """The packed x is the encoding of the unrounded norm: values within 2^-16 of a
    rounding point may fall to either side, all others are equal."""
    c = _norm_case(np.random.default_rng(cols + rows), rows, cols, dt, 0)
    d = {k: None if v is None else v.cuda() for k, v in c.items()}
    gh, t = rz.razer_block_norm(d["y"], d["h"], post_weight=d["post"], pre_weight=d["pre"], packed=True)
    gh2, _ = rz.razer_block_norm(d["y"], d["h"], post_weight=d["post"], pre_weight=d["pre"])
    assert torch.equal(gh, gh2)
    _, x = mx.block_norm(_f64(c["y"]), _f64(c["h"]), _f64(c["post"]), True, None, 1.0, _f64(c["pre"]), 1e-5)
    got = rz.razer_mx_dequant(t).double().cpu().numpy()
    b = np.abs(x).reshape(rows, -1, 32).max(-1).repeat(32, -1) * 2.0 ** -16
    near = [mx.decode(*mx.encode(x + s * b)) for s in (-1, 0, 1)] + [mx.decode(*mx.encode(x * (1 + s * 2.0 ** -16))) for s in (-1, 1)]
    assert np.logical_or.reduce([got == v for v in near]).all()
    assert (got == near[1]).mean() > 0.99


@pytest.mark.parametrize("dt", DT)
def test_block_norm_parts(dt):
    """Without y, without weights, in place, from strided rows, of zero rows."""
    rng = np.random.default_rng(3)
    wide = torch.from_numpy(rng.standard_normal((6, 3 * 256))).to(DT[dt]).cuda()
    h, y = wide[:, 256:512], wide[:, 512:]
    gh, gx = rz.razer_block_norm(None, h)
    assert torch.equal(gh, h)
    wx = mx.rms(_f64(h), None, 1e-5)
    _close(gx, wx, np.abs(wx) + 1, DT[dt])
    wh, wx = mx.block_norm(_f64(y), _f64(h), None, True, None, -2.0, None, 0.5)
    gh, gx = rz.razer_block_norm(y, h, post_norm=True, residual_scale=-2.0, eps=0.5)
    _close(gh, wh, np.abs(_f64(h)) + np.abs(wh - _f64(h)), DT[dt])
    own = h.contiguous()
    g2, x2 = rz.razer_block_norm(y, own, post_norm=True, residual_scale=-2.0, eps=0.5, h_out=own)
    assert g2 is own and torch.equal(own, gh) and torch.equal(x2, gx)
    z = torch.zeros(3, 256, dtype=DT[dt], device="cuda")
    gh, t = rz.razer_block_norm(z, z, post_norm=True, packed=True)
    assert (gh == 0).all() and (t.codes == 0).all() and (t.scales == 0).all()
    nan = z.clone()
    nan[1, 7] = float("nan")
    _, t = rz.razer_block_norm(nan, z, post_norm=True, packed=True)
    assert (t.scales[1] == 255).all() and (t.scales[0] == 0).all() and (t.codes == 0).all()


def test_empty():
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    t = rz.razer_mx_quantize(e)
    assert t.shape == (0, 64) and rz.razer_mx_dequant(t).shape == (0, 64)
    w = rz.razer_mx_quantize(torch.ones(8, 64, device="cuda"))
    assert rz.razer_mx_gemm(t, w).shape == (0, 8) and rz.razer_mx_gemm(w, t).shape == (8, 0)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert rz.razer_mx_gemm_grouped(t, w, off).shape == (0, 4)
    assert rz.razer_mx_gemm_grouped(w, w, off, torch.empty(0, dtype=torch.int32, device="cuda")).shape == (0, 4)
    h, x = rz.razer_block_norm(e, e, post_norm=True)
    assert h.shape == x.shape == (0, 64)


# ---- streams and graphs ------------------------------------------------------

def test_other_stream_and_graph():
    """The calls run on the current stream, and a captured layer replays to the
    eager result."""
    rng = np.random.default_rng(2)
    d, i, m = 256, 384, 5
    t = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(torch.bfloat16).cuda()  # noqa: E731
    y, h, p, q = t(m, d), t(m, d), t(d), t(d)
    up, down = rz.razer_mx_quantize(t(2 * i, d)), rz.razer_mx_quantize(t(d, i))
    off = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda")

    def layer():
        a, x = rz.razer_block_norm(y, h, post_weight=p, pre_weight=q, packed=True)
        b = rz.razer_mx_gemm(rz.razer_mx_quantize_gated(rz.razer_mx_gemm(x, up)), down)
        return a, b, rz.razer_mx_gemm_grouped(x, up, off)

    want = layer()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = layer()
    s.synchronize()
    for u, v in zip(got, want):
        assert torch.equal(u, v)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = layer()
    for r in range(3):
        y.copy_(t(m, d))
        g.replay()
        torch.cuda.synchronize()
        for u, v in zip(got, layer()):
            assert torch.equal(u, v), r
        torch.cuda.synchronize()
