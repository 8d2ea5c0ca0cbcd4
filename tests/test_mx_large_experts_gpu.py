"""MXFP4 products on the kernels' forms that no smaller size reaches: experts in tiles of
256 rows, split tiles of 256 rows, and the stream kernel's other forms for experts.
test_mx_paths.py asserts which form each size runs on (bound:
``mx_common.assert_product``)."""
import pytest

import mx_common as mx
import test_mx_shapes_gpu as shapes

pytestmark = pytest.mark.gpu

# experts whose rows fill tiles of 256, others of one row or none; widths that end inside a
# tile and a store, K that ends inside a window, more tiles than compute units
GROUPS = [(2083, 544, [900, 0, 1, 2100, 513]), (1000, 1056, [257, 2600, 0, 1500, 1, 255, 256, 3100]),
          (4100, 512, [700, 0, 1301]), (4099, 1504, [3000, 256, 1, 2000])]
SMALL = [(400, 992, [(7 * i) % 41 for i in range(40)]), (100, 6176, [(3 * i) % 9 for i in range(30)])]
TILES_128 = [(700, 1056, [1, 900, 257, 0, 1500])]
SPLIT = [(4721, 3361, 2080), (4209, 3870, 2112)]


@pytest.mark.parametrize("gather,holes", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("n,k,sizes", GROUPS)
def test_tiles_of_256_rows(n, k, sizes, gather, holes):
    shapes.grouped(n, k, sizes, gather, holes, mx.DT.values())


@pytest.mark.parametrize("gather,holes", [(False, False), (True, True)])
@pytest.mark.parametrize("n,k,sizes", SMALL + TILES_128)
def test_other_forms(n, k, sizes, gather, holes):
    shapes.grouped(n, k, sizes, gather, holes, mx.DT.values())


@pytest.mark.parametrize("m,n,k", SPLIT)
def test_split_tiles_of_256_rows(m, n, k):
    shapes.check(m, n, k, mx.DT.values())
