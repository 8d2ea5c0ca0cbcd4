"""The 8-bit integer operators from their definitions (numpy), for the tests; shares
nothing with the library."""
import numpy as np
import torch

import nvfp4_razer_w4a16_amd as rz

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def encode(x):
    """(codes, scales) of x [rows, cols] (a tensor), in fp32 with one rounding an operation."""
    x = x.float().cpu().numpy()
    amax = np.abs(x).max(1)
    bad = ~np.isfinite(x).all(1)
    amax = np.where(bad, np.float32(1), amax).astype(np.float32)
    pre = np.where(amax < np.float32(2.0 ** -64), np.float32(2.0 ** 64), np.float32(1))
    with np.errstate(divide="ignore", invalid="ignore"):
        inverse = np.where(amax > 0, np.float32(127) / (amax * pre), np.float32(0)).astype(np.float32)
        q = np.rint((x * pre[:, None]).astype(np.float32) * inverse[:, None])
    scales = np.where(bad, np.float32(np.nan), amax / np.float32(127)).astype(np.float32)
    q[bad] = 0
    return q.astype(np.int8), scales


def device(codes, scales):
    return rz.I8Tensor.of(torch.from_numpy(np.ascontiguousarray(codes)).cuda(),
                          torch.from_numpy(np.ascontiguousarray(scales, dtype=np.float32)).cuda())


def random_i8(rng, rows, cols, lo=-127, hi=127):
    """Random codes and scales (about 2^-8): (codes, scales)."""
    return (rng.integers(lo, hi + 1, (rows, cols)).astype(np.int8),
            np.exp(rng.normal(-5, 1, rows)).astype(np.float32))


def product(x, sx, w, sw, dtype):
    """The exact sum, rounded to fp32, times sx, times sw, rounded to dtype."""
    # sums of up to 2^17 products of up to 2^14 are whole numbers below 2^53
    total = np.rint(x.astype(np.float64) @ w.astype(np.float64).T).astype(np.float32)
    with np.errstate(over="ignore", under="ignore", invalid="ignore"):
        y = (total * sx[:, None].astype(np.float32)).astype(np.float32) * sw[None, :].astype(np.float32)
    return torch.from_numpy(y.astype(np.float32)).to(dtype)


def same(got, want):
    """Bit for bit, NaN for NaN."""
    got, want = got.cpu(), want.cpu()
    assert got.shape == want.shape and got.dtype == want.dtype
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    bad = (got != want) & ~nan
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} differ, first at {bad.nonzero()[0].tolist()}"
