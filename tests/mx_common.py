"""The MXFP4 operators and the block norm from their definitions in 64 bits
(numpy), for the tests; shares nothing with the library.  `plant` lets a test of
the tests make one mistake here, on the CPU."""
import numpy as np
import torch

import nvfp4_razer_w4a16_amd as rz

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_ULP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def encode(x):
    """(codes, scale bytes) of x [rows, cols], float64, one code an entry."""
    rows, cols = x.shape
    b = x.reshape(rows, cols // 32, 32)
    amax = np.abs(b).max(-1)
    bad = ~np.isfinite(b).all(-1)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.frexp(np.where(bad, 0.0, amax))[1] - 1  # floor(log2)
    byte = np.where(amax > 0, np.maximum(e - 2 + 127, 0), 0)
    v = np.where(bad[..., None], 0.0, b) / np.exp2(byte - 127.0)[..., None]
    d = np.abs(np.abs(v)[..., None] - GRID)
    near = d.min(-1, keepdims=True)
    # the nearest grid value; of two equally near, the one with the even index
    code = np.where(d == near, np.array([0, 9, 1, 9, 2, 9, 3, 9]) * 1.0 + 0.5 * (np.arange(8) % 2), 99.0)
    even = np.argmin(code, -1)
    only = np.argmax(d == near, -1)
    ties = (d == near).sum(-1) > 1
    code = np.where(ties, even, only)
    code = code + 8 * (np.signbit(v) & ~bad[..., None])
    byte = np.where(bad, 255, byte)
    return code.reshape(rows, cols).astype(np.uint8), byte.astype(np.uint8)


def pack(code):
    return code[:, 0::2] | (code[:, 1::2] << 4)


def decode(code, byte):
    rows, cols = code.shape
    v = np.where(code & 8, -1.0, 1.0) * GRID[code & 7]
    s = np.where(byte == 255, np.nan, np.exp2(byte.astype(np.float64) - 127.0))
    return (v.reshape(rows, cols // 32, 32) * s[..., None]).reshape(rows, cols)


def device(code, byte):
    return rz.MxTensor.of(torch.from_numpy(np.ascontiguousarray(pack(code))).cuda(),
                          torch.from_numpy(np.ascontiguousarray(byte)).cuda())


def random_mx(rng, rows, cols, lo=118, hi=134):
    """Random codes and scale bytes in [lo, hi): (codes, bytes)."""
    return (rng.integers(0, 16, (rows, cols)).astype(np.uint8),
            rng.integers(lo, hi, (rows, cols // 32)).astype(np.uint8))


def product(x, w):
    """(x w^T, sum |x||w|) in float64."""
    return x @ w.T, np.abs(x) @ np.abs(w).T


def assert_product(got: torch.Tensor, want, norm, k, what=""):
    """Every fp32 addition of the K products errs by at most one part in 2^23 of
    a partial sum, which is at most `norm`; the output is rounded once, to
    infinity from half a step above its type's largest value."""
    y = got.double().cpu().numpy()
    top = float(torch.finfo(got.dtype).max)
    top = (top + 2.0 ** np.ceil(np.log2(top))) / 2
    over = np.isinf(y) & (np.abs(want) + k * 2.0 ** -23 * norm >= top)
    assert (np.sign(y[over]) == np.sign(want[over])).all(), what
    y, want, norm = np.where(over, 0.0, y), np.where(over, 0.0, want), np.where(over, 0.0, norm)
    assert y.shape == want.shape, what
    assert np.array_equal(np.isnan(y), np.isnan(want)), what
    bound = k * 2.0 ** -23 * norm + HALF_ULP[got.dtype] * np.abs(want) * 1.01 + TINY[got.dtype]
    ok = np.isnan(want) | (np.abs(y - want) <= bound)
    assert ok.all(), f"{what}: {(~ok).sum()} of {ok.size} off, first at {np.argwhere(~ok)[0]}"


def rms(v, w, eps):
    v = v / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    return v if w is None else v * w


def block_norm(y, h, post, norm_y, gate, scale, pre, eps):
    t = 0.0
    if y is not None:
        t = rms(y, post, eps) if norm_y else (y if post is None else y * post)
        if gate is not None:
            g = np.atleast_2d(gate)
            t = t * np.repeat(g, h.shape[0] // g.shape[0], 0)
    h = h + scale * t
    return h, rms(h, pre, eps)
