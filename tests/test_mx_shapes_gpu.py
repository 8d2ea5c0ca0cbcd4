"""MXFP4 products at the sizes where the kernels take another path: more tiles than
compute units, K cut into slices, K that ends inside a window or a chunk, jobs that
share a workgroup, scale bytes that start anywhere.  References in 64 bits; the
bound is that of ``mx_common.assert_product``."""
import numpy as np
import pytest
import torch

import mx_common as mx
import nvfp4_razer_w4a16_amd as rz

pytestmark = pytest.mark.gpu


def check(m, n, k, dts, seed=0, x=None, w=None):
    rng = np.random.default_rng(m + n + k + seed)
    x = x or mx.random_mx(rng, m, k)
    w = w or mx.random_mx(rng, n, k)
    want, norm = mx.product(mx.decode(*x), mx.decode(*w))
    dx, dw = mx.device(*x), mx.device(*w)
    for dt in dts:
        got = rz.razer_mx_gemm(dx, dw, dt)
        mx.assert_product(got, want, norm, k, (m, n, k, dt))
        again = rz.razer_mx_gemm(dx, dw, dt)  # the same bits, NaN included
        assert torch.equal(got.view(torch.uint8), again.view(torch.uint8)), (m, n, k, dt)


# many rows: tiles of 256 x 256, one window of 512 to many, K ending inside one
@pytest.mark.parametrize("m,n,k", [(1100, 1300, 512), (1030, 2300, 544), (2060, 1801, 1056), (1300, 2050, 2080),
                                   (900, 8300, 992)])
def test_tiles(m, n, k):
    check(m, n, k, mx.DT.values())


# more tiles than compute units: workgroups walk from tile to tile, with one window a
# tile, an odd number of them, and a last round that is cut along K
@pytest.mark.parametrize("m,n,k", [(4200, 4300, 512), (4113, 4357, 544), (4200, 4300, 1440), (4113, 4301, 7200)])
def test_rounds_of_tiles(m, n, k):
    check(m, n, k, [torch.bfloat16])


# few tiles and a long K: slices whose sums are added afterwards
@pytest.mark.parametrize("m,n,k", [(1, 300, 16384), (40, 257, 15392), (300, 260, 16416), (513, 770, 20000)])
def test_slices(m, n, k):
    if m == 1:
        assert rz.razer_mx_workspace_bytes(m, n, k) > 0
    check(m, n, k, mx.DT.values())


# few rows: one, two and four chunks of a row, jobs of 16, 32 and 64 rows, more row
# tiles of W than compute units; K ends inside a chunk, a product and a dword of scales
@pytest.mark.parametrize("k", [2048, 2080, 4096, 6176, 8192, 8224, 13152, 15360])
@pytest.mark.parametrize("m", [1, 16, 20, 50, 130, 250])
def test_few_rows(m, k):
    check(m, 4999, k, [torch.bfloat16, torch.float32] if m == 50 else [torch.bfloat16])


# W from memory where its scale bytes start on any byte, NaN bytes around them
@pytest.mark.parametrize("skew", [1, 2, 3])
@pytest.mark.parametrize("m,n,k", [(1, 100, 4096), (7, 33, 2080), (40, 100, 6176), (130, 70, 13184), (1200, 2100, 1056)])
def test_scale_alignment(m, n, k, skew):
    rng = np.random.default_rng(m + skew)
    x, w = mx.random_mx(rng, m, k), mx.random_mx(rng, n, k)

    def moved(t, by):
        code, byte = t
        buf = np.full(byte.size + 64, 255, np.uint8)
        buf[16 + by:16 + by + byte.size] = byte.ravel()
        s = torch.from_numpy(buf).cuda()[16 + by:16 + by + byte.size].view(byte.shape)
        return rz.MxTensor.of(torch.from_numpy(np.ascontiguousarray(mx.pack(code))).cuda(), s)

    want, norm = mx.product(mx.decode(*x), mx.decode(*w))
    got = rz.razer_mx_gemm(moved(x, 4 - skew), moved(w, skew), torch.float32)
    mx.assert_product(got, want, norm, k)


@pytest.mark.parametrize("m,n,k", [(1, 5000, 4096), (30, 4200, 8192), (60, 4200, 4128), (20, 4200, 13152), (1100, 2100, 1504)])
def test_nan_scale(m, n, k):
    """A NaN block makes its row of x, or its column of y, NaN and nothing else, in
    the last block of K, the last row and in between."""
    rng = np.random.default_rng(m + k)
    (xc, xb), (wc, wb) = mx.random_mx(rng, m, k), mx.random_mx(rng, n, k)
    xb[m - 1, -1] = wb[n - 1, -1] = wb[1700, 0] = wb[33, k // 64] = 255
    check(m, n, k, [torch.float32], x=(xc, xb), w=(wc, wb))


def grouped(n, k, sizes, gather, holes=False, dts=(torch.bfloat16,)):
    rng = np.random.default_rng(n + k + len(sizes))
    e, m = len(sizes), sum(sizes)
    tokens = max(1, m // 2) if gather else m
    x, w = mx.random_mx(rng, tokens, k), mx.random_mx(rng, e * n, k)
    if holes:
        x[1][0] = x[1][-1] = 255  # the rows that clamped numbers would read
    rows = rng.integers(1, max(2, tokens - 1), m).astype(np.int32) if holes else rng.integers(0, tokens, m).astype(np.int32)
    if holes:
        rows[::5], rows[3::7] = -1, tokens
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    xv, wv = mx.decode(*x), mx.decode(*w)
    none = (rows < 0) | (rows >= tokens) if gather else np.zeros(m, bool)
    src = xv[np.where(none, 1 % tokens, rows)] if gather else xv
    want, norm = np.zeros((m, n)), np.zeros((m, n))
    for i in range(e):
        s = slice(off[i], off[i + 1])
        want[s], norm[s] = mx.product(src[s], wv[i * n:(i + 1) * n])
    want[none], norm[none] = 0, 0
    for dt in dts:
        got = rz.razer_mx_gemm_grouped(mx.device(*x), mx.device(*w), torch.from_numpy(off).cuda(),
                                       torch.from_numpy(rows).cuda() if gather else None, dt)
        mx.assert_product(got, want, norm, k, (n, k, dt))


# experts of a few rows: a workgroup's piece of the line holds several of them
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("n,k,sizes", [(40, 2080, [i % 4 for i in range(600)]), (100, 6176, [(7 * i) % 30 for i in range(80)]),
                                       (33, 4096, [(11 * i) % 70 for i in range(90)]), (50, 13152, [i % 3 for i in range(70)]),
                                       (1000, 1056, [0] * 5 + [300] + [1] * 60), (24, 14336, [40, 0, 33, 1, 90])])
def test_small_experts(n, k, sizes, gather):
    grouped(n, k, sizes, gather)


# experts of many rows: tiles of 256 rows, more of them than compute units
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("n,k,sizes", [(2080, 576, [2600, 0, 5200]), (700, 1056, [1, 900, 257, 0, 1500]),
                                       (4100, 512, [1300, 255, 3000, 256, 257]), (300, 16384, [3, 0, 260])])
def test_large_experts(n, k, sizes, gather):
    grouped(n, k, sizes, gather, dts=[torch.float32] if n == 700 else [torch.bfloat16])


@pytest.mark.parametrize("n,k,sizes", [(64, 2080, [3, 0, 9, 16] * 12), (70, 6176, [30, 5, 41]), (90, 13152, [20] * 4),
                                       (1100, 1056, [1500, 3, 1200]), (50, 4096, [60] * 7)])
def test_open_rows(n, k, sizes):
    """Row numbers outside x give zero rows, whatever the rows at x's ends hold."""
    grouped(n, k, sizes, True, holes=True, dts=[torch.float32])
