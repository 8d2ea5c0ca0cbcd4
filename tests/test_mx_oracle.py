"""The MXFP4 tests' own oracle and comparers: a mistake planted there, on the CPU, has to
show.  CPU only; nothing of the library runs."""
import fractions

import numpy as np
import pytest
import torch

import mx_common as mx
import mx_packed


@pytest.fixture
def plant(monkeypatch):
    """plant(name, wrong): mx_common's function `name` becomes wrong(the right one)."""
    return lambda name, wrong: monkeypatch.setattr(mx, name, wrong(getattr(mx, name)))


def _operands(m=5, n=40, k=160):
    rng = np.random.default_rng(7)
    return mx.random_mx(rng, m, k), mx.random_mx(rng, n, k), k


def _products(dt):
    """(what a right kernel gives, x, w, k)."""
    x, w, k = _operands()
    return torch.from_numpy(mx.product(mx.decode(*x), mx.decode(*w))[0]).to(dt), x, w, k


def _check(got, x, w, k):
    mx.assert_product(got, *mx.product(mx.decode(*x), mx.decode(*w)), k)


def _one_block(change):
    def wrong(decode):
        def f(code, byte):
            v = decode(code, byte)
            v[-1, -32:] = change(v[-1, -32:])
            return v
        return f
    return wrong


MISTAKES = {
    "a block's scale is one binade off": ("decode", _one_block(lambda v: 2 * v)),
    "the last block is missing": ("decode", _one_block(lambda v: 0 * v)),
    "two neighbours are exchanged": ("decode", _one_block(lambda v: v.reshape(-1, 2)[:, ::-1].ravel())),
    "one sign is wrong": ("decode", _one_block(lambda v: np.where(np.arange(32) == np.abs(v).argmax(), -v, v))),
    "the block is NaN": ("decode", _one_block(lambda v: v * np.nan)),
    "two rows are exchanged": ("product", lambda f: lambda x, w: tuple(v[[1, 0, *range(2, len(v))]] for v in f(x, w))),
    "the weight's rows are one off": ("product", lambda f: lambda x, w: f(x, np.roll(w, 1, 0))),
}


@pytest.mark.parametrize("dt", mx.DT.values())
@pytest.mark.parametrize("what", MISTAKES)
def test_a_wrong_product_is_noticed(what, dt, plant):
    args = _products(dt)
    _check(*args)
    plant(*MISTAKES[what])
    with pytest.raises(AssertionError):
        _check(*args)


def test_encode_and_decode_follow_the_definition():
    """In exact arithmetic: the block's power of two, the nearest grid value, halves to the
    even code, six at most."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((6, 64)) * np.exp2(rng.integers(-130, 120, (6, 1)).astype(np.float64))
    x[0, :9] = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9, -0.25]) * 2.0 ** 10
    x[0, 9:32], x[5, 32:] = 0, 0
    code, byte = mx.encode(x)
    values = mx.decode(code, byte)
    grid = [fractions.Fraction(v) for v in mx.GRID]
    for r in range(6):
        for b in range(2):
            block = [fractions.Fraction(float(v)) for v in x[r, 32 * b:32 * b + 32]]
            top, e = max(map(abs, block)), 0
            while top and top < fractions.Fraction(2) ** e:
                e -= 1
            while top >= fractions.Fraction(2) ** (e + 1):
                e += 1
            want = max(e - 2 + 127, 0) if top else 0
            assert byte[r, b] == want
            unit = fractions.Fraction(2) ** (want - 127)
            for j, v in enumerate(block):
                a = min(abs(v) / unit, 6)
                best = min(range(8), key=lambda i: (abs(a - grid[i]), i % 2))
                assert code[r, 32 * b + j] & 7 == best
                assert fractions.Fraction(float(values[r, 32 * b + j])) == (-1 if v < 0 else 1) * grid[best] * unit


def _packed():
    x = np.random.default_rng(5).standard_normal((4, 96))
    return (*mx.encode(x), x, np.abs(x) * 2.0 ** -16)


def test_a_wrong_encoding_is_noticed():
    code, byte, x, err = _packed()
    mx_packed.assert_packed(code, byte, x, err)
    for change in (lambda c, b: (c ^ 1, b), lambda c, b: (c ^ 8, b), lambda c, b: (c, b + 1), lambda c, b: (c, b - 1),
                   lambda c, b: (np.roll(c, 1, 1), b), lambda c, b: (np.roll(c, 1, 0), b), lambda c, b: (c, np.roll(b, 1, 1)[:, ::-1] + 2),
                   lambda c, b: (0 * c, b)):
        with pytest.raises(AssertionError):
            mx_packed.assert_packed(*change(code, byte), x, err)


def _norm():
    """(arguments, codes, scale bytes) of a right packed norm."""
    rng = np.random.default_rng(9)
    y, h, post, pre = rng.standard_normal((4, 64)), rng.standard_normal((4, 64)), *rng.standard_normal((2, 64))
    args = (y, h, post, True, None, 0.75, pre, 1e-5)
    return args, *mx.encode(mx.block_norm(*args)[1])


def test_a_wrong_norm_is_noticed(plant):
    args, code, byte = _norm()
    mx_packed.assert_packed(code, byte, *mx_packed.norm_bound(*args))
    plant("rms", lambda f: lambda v, w, eps: f(v, w, eps) * np.sqrt(63 / 64))  # the mean's divisor is one off
    with pytest.raises(AssertionError):
        mx_packed.assert_packed(code, byte, *mx_packed.norm_bound(*args))


def test_a_norm_rounded_before_it_is_packed_is_noticed():
    rng = np.random.default_rng(9)
    h = rng.standard_normal((400, 512))
    args = (None, h, None, False, None, 1.0, None, 1e-5)
    x, err = mx_packed.norm_bound(*args)
    mx_packed.assert_packed(*mx.encode(x), x, err)
    with pytest.raises(AssertionError):  # 8 bits of fraction
        mx_packed.assert_packed(*mx.encode(torch.from_numpy(x).bfloat16().double().numpy()), x, err)
