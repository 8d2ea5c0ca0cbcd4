"""MXFP4 products of few rows with a short K, many row tiles a workgroup: chunks of
whole short rows, more of them under way (bound: ``mx_common.assert_product``)."""
import pytest
import torch

import test_mx_shapes_gpu as shapes

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n,k", [(1, 50001, 544), (16, 40000, 1056), (3, 70000, 32), (20, 40003, 1024), (32, 33000, 2048),
                                   (50, 40000, 992), (64, 36000, 2048), (9, 33333, 2016)])
def test_many_short_rows(m, n, k):
    shapes.check(m, n, k, [torch.bfloat16])


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("n,k,sizes", [(700, 1056, [(5 * i) % 17 for i in range(120)]), (1503, 2048, [(3 * i) % 40 for i in range(40)]),
                                       (90, 512, [(7 * i) % 90 for i in range(300)]), (16, 96, [1] * 900)])
def test_experts_of_short_rows(n, k, sizes, gather):
    shapes.grouped(n, k, sizes, gather)
