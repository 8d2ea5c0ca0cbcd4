"""The products in 8-bit integers at sizes that reach every form of the kernels
(tests/test_i8_paths.py says which), with rows and columns that end inside a tile, bit for
bit.  The sums of the reference are whole numbers below 2^53, exact in fp64."""
import numpy as np
import pytest
import torch

import i8_common as ref
import nvfp4_razer_w4a16_amd as rz

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.float16, torch.bfloat16]


def _random(gen, rows, cols):
    codes = torch.randint(-127, 128, (rows, cols), generator=gen, device="cuda").to(torch.int8)
    return rz.I8Tensor.of(codes, torch.exp(torch.randn(rows, generator=gen, device="cuda") - 5))


def _product(x, sx, w, sw, dtype):
    return ((x.double() @ w.double().t()).float() * sx[:, None] * sw).to(dtype)


def _check(m, n, k, types=TYPES):
    gen = torch.Generator(device="cuda").manual_seed(m + n + k)
    x, w = _random(gen, m, k), _random(gen, n, k)
    for dtype in types:
        out = torch.full((m + 1, n), 7.0, dtype=dtype, device="cuda")
        rz.razer_i8_gemm(x, w, out=out[:m])
        ref.same(out[:m], _product(x.codes, x.scales, w.codes, w.scales, dtype))
        assert (out[m] == 7.0).all()


FEW = [(m, n, k) for m in (5, 20, 50)
       for n, k in ((20000, 512), (20000, 496), (9000, 1024), (9000, 560), (4999, 2048), (4999, 1872), (4999, 4096),
                    (4999, 2080), (4999, 8192), (4999, 5008), (4999, 16384), (4999, 9216))]


@pytest.mark.parametrize("m,n,k", FEW)
def test_few_rows(m, n, k):
    _check(m, n, k)


TILES = [(4096, 4096, 1040), (8192, 4111, 528), (4100, 4099, 528), (3000, 8000, 144), (2300, 8000, 16), (1500, 9000, 128),
         (6200, 3500, 1296), (5537, 8530, 1040), (2112, 7887, 1168), (1259, 5439, 5008), (600, 2000, 1008)]
HALVES = [(5700, 4000, 2000), (2600, 7168, 2048), (4907, 7097, 1296)]
SLICES = [(1024, 4096, 14336), (1000, 4090, 14336), (900, 2040, 16400), (1030, 3000, 9008), (100, 260, 16400),
          (299, 7026, 9360), (1361, 5987, 7376), (4161, 4018, 5664), (1450, 866, 8592)]


@pytest.mark.parametrize("m,n,k", TILES + HALVES + SLICES)
def test_tiles(m, n, k):
    _check(m, n, k)


def sizes_of(total, experts, seed):
    """`total` rows over the experts, a fifth of which get none."""
    rng = np.random.default_rng(seed)
    liking = np.exp(rng.normal(0, 0.5, experts)) * (rng.random(experts) > 0.2)
    liking[0] = max(liking[0], 0.5)
    return rng.multinomial(total, liking / liking.sum()).tolist()


GROUPS = [(40, 2000, 512, 8), (40, 2000, 480, 8), (100, 3000, 512, 8), (40, 2000, 1024, 8), (90, 2000, 1008, 5),
          (40, 2000, 2048, 8), (90, 2000, 2048, 5), (200, 2000, 2048, 8), (40, 900, 4096, 8), (90, 900, 4096, 5),
          (700, 300, 4096, 20), (40, 900, 8192, 8), (200, 900, 8192, 8), (40, 900, 16384, 8), (1000, 24, 64, 500),
          (9000, 3000, 656, 8), (9000, 3001, 656, 100), (3000, 2000, 528, 4), (12000, 1100, 528, 5), (700, 900, 16400, 4),
          (2304, 1323, 1232, 50), (2689, 3565, 1040, 4)]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("m,n,k,experts", GROUPS)
def test_experts(m, n, k, experts, gather):
    gen = torch.Generator(device="cuda").manual_seed(m + n + k)
    tokens = 77 if gather else m
    x, w = _random(gen, tokens, k), _random(gen, experts * n, k)
    offsets = np.concatenate([[0], np.cumsum(sizes_of(m - 3, experts, m))])  # the last three rows belong to none
    rows = torch.arange(m, device="cuda")
    if gather:
        rows = torch.randint(0, tokens, (m,), generator=gen, device="cuda")
        rows[torch.rand(m, generator=gen, device="cuda") < 0.1] = -1
    for dtype in TYPES:
        out = torch.full((m, n), 7.0, dtype=dtype, device="cuda")
        want = out.clone()
        rz.razer_i8_gemm_grouped(x, w, torch.from_numpy(offsets.astype(np.int32)).cuda(), rows.int() if gather else None,
                                 out=out)
        for e in range(experts):
            s, we = slice(int(offsets[e]), int(offsets[e + 1])), slice(e * n, (e + 1) * n)
            if s.start == s.stop:
                continue
            r = rows[s].clamp_min(0)
            want[s] = _product(x.codes[r], x.scales[r], w.codes[we], w.scales[we], dtype)
            want[s][rows[s] < 0] = 0.0
        ref.same(out, want)
