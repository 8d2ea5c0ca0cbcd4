"""How products at the ends of their range are cut: every tile of the result is there once,
as long as a result of that many could exist.  CPU only."""
import pytest

from test_i8_paths import plan  # noqa: F401  (a fixture)

INT32_MAX = 2 ** 31 - 1
SIZES = [(2 ** 30, 2 ** 30, 131056, 0), (2 ** 30, 2 ** 18, 131056, 4096), (2 ** 30, 1, 131056, 0), (2 ** 30, 2 ** 18, 16, 0),
         (2 ** 30, 129, 16, 0), (2 ** 20 + 1, 2 ** 20 - 1, 4096, 0), (2 ** 22, 2 ** 22, 16, 0), (3 * 2 ** 20, 77, 20000, 5),
         (2 ** 24, 2 ** 15, 131056, 0), (1, 2 ** 30, 131056, 0), (1, 1, 131056, 0)]


@pytest.mark.parametrize("m,n,k,experts", SIZES)
def test_every_tile_once(plan, m, n, k, experts):  # noqa: F811
    kind, wide, high, full, rest, split, halves = plan(m, n, k, experts)
    assert kind == "tile" and (wide, high) in {(256, 256), (256, 128), (128, 128)}
    # an expert's last tile is a part: at most one more for each of them
    tiles = (-(-m // high) + min(experts, m)) * -(-n // wide)
    assert full + rest == min(tiles, INT32_MAX)
    assert (split == 1 and rest == 0) or (2 <= split <= 8 and 0 < rest * split <= 256 * (2 if wide == 128 else 1))
    assert halves == 0 or (high == 256 and rest == 0 and 0 < halves <= min(full, 128))
    if experts:
        assert rest == halves == 0


@pytest.mark.parametrize("m,n,k,experts,want", [
    (1, 2 ** 30, 16, 0, ("stream", 4, 1, 1, 16)), (2 ** 30, 16, 16, 4096, ("stream", 1, 1, 4, 64)),
    (2 ** 30, 1, 131056, 0, ("tile", 128, 128)), (2 ** 30, 2 ** 18, 131056, 4096, ("tile", 256, 256))])
def test_forms(plan, m, n, k, experts, want):  # noqa: F811
    assert plan(m, n, k, experts)[:len(want)] == want
