"""Comparing a packed tensor with values that are known up to a bound."""
import numpy as np

import mx_common as mx


def scale_byte(amax):
    e = np.frexp(amax)[1] - 1  # floor(log2)
    return np.where(amax > 0, np.maximum(e - 2 + 127, 0), 0)


def rounded(v, byte):
    """v [rows, cols] on the grid of scale bytes [rows, cols // 32]; monotone in v."""
    unit = np.exp2(byte - 127.0).repeat(32, -1)
    a = np.abs(v) / unit
    step = np.where(a >= 4, 2.0, np.where(a >= 2, 1.0, 0.5))
    return np.copysign(np.minimum(np.rint(a / step) * step, 6.0), v) * unit


def assert_packed(code, byte, x, err, what=""):
    """codes (one an entry) and scale bytes are an encoding of some values within err of
    x: each byte that of a block maximum in its range, each code between the roundings,
    under that byte, of x - err and x + err."""
    blocks = lambda v: v.reshape(v.shape[0], -1, 32).max(-1)  # noqa: E731
    lo, hi = scale_byte(blocks(np.maximum(np.abs(x) - err, 0))), scale_byte(blocks(np.abs(x) + err))
    ok = (lo <= byte) & (byte <= hi)
    assert ok.all(), f"{what}: {(~ok).sum()} scale bytes off, first at {np.argwhere(~ok)[0]}"
    got = mx.decode(code, byte)
    ok = (rounded(x - err, byte) <= got) & (got <= rounded(x + err, byte))
    assert ok.all(), f"{what}: {(~ok).sum()} codes off, first at {np.argwhere(~ok)[0]}"


def arrays(t):
    """(codes, one an entry, scale bytes) of an MxTensor."""
    c = t.codes.cpu().numpy()
    code = np.empty((t.rows, t.cols), np.uint8)
    code[:, 0::2], code[:, 1::2] = c & 15, c >> 4
    return code, t.scales.cpu().numpy()


def norm_bound(y, h, post, norm_y, gate, scale, pre, eps):
    """(x, err) of the block norm.  In fp32 a mean of squares is off by at most 54 roundings
    (32 in a lane, 6 and 16 across lanes and waves) and its root and products by 10 more:
    64 * 2^-24 = 2^-18 of each factor.  So h' is off by 2^-17 of |h| + |t|, t what is added;
    the root of mean(h'^2) by that much of the root of the mean of their squares
    (Cauchy-Schwarz), and its own 2^-18."""
    wh, x = mx.block_norm(y, h, post, norm_y, gate, scale, pre, eps)
    eh = 2.0 ** -17 * (np.abs(h) + np.abs(wh - h))
    ms = (wh * wh).mean(-1, keepdims=True) + eps
    rel = np.sqrt((eh * eh).mean(-1, keepdims=True) / ms) + 2.0 ** -17
    return x, eh / np.sqrt(ms) * (1.0 if pre is None else np.abs(pre)) + np.abs(x) * rel


def gated(g, u):
    """(silu(g) * u, err).  exp(-g) carries its argument's rounding, |g| log2(e) in units of
    2^-24, and that of log2(e): together less than 2 |g| 2^-24 of its value; the
    exponential, the sum, the quotient and the product add less than 8 * 2^-24.  Where
    exp(-g) passes fp32's range the result is 0, where it is subnormal it is off by less
    than a unit of 2^-149 times u."""
    with np.errstate(over="ignore"):
        p = g / (1 + np.exp(-g)) * u
    err = np.abs(p) * (2 * np.abs(g) + 8) * 2.0 ** -24 + 2.0 ** -148 * (1 + np.abs(u))
    return p, np.where(g < -88, np.abs(p) + err, err)
