"""Packed results of the block norm and the gated encoder against their formulas in 64
bits: gates, many rows a workgroup and every width of a row's lanes; gates of silu far
from zero.  The bounds are those of mx_packed."""
import numpy as np
import pytest
import torch

import mx_common as mx
import mx_packed
import nvfp4_razer_w4a16_amd as rz

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")]
DT = mx.DT


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("rows,cols,gates", [(9, 64, 9), (130, 512, 10), (7, 96, 1), (1030, 544, 2), (1000, 1024, 1000), (258, 32, 3),
                                             (6, 1056, 2), (5, 2048, 0), (12, 4128, 3), (300, 4096, 4), (3, 8192, 3),
                                             (4, 8224, 2), (2, 16416, 1), (3, 32768, 3)])
def test_block_norm(rows, cols, gates, dt):
    rng = np.random.default_rng(rows + cols)
    t = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(DT[dt])  # noqa: E731
    y, h, post, pre = t(rows, cols) * 4, t(rows, cols), t(cols), t(cols)
    gate = t(gates, cols) if gates else None
    h[:, ::37] *= 30  # outlier channels
    for norm_y in (True, False):
        x, err = mx_packed.norm_bound(*(None if v is None else v.double().numpy() for v in (y, h, post)), norm_y,
                                      None if gate is None else gate.double().numpy(), 0.75, pre.double().numpy(), 1e-5)
        _, q = rz.razer_block_norm(y.cuda(), h.cuda(), post_weight=post.cuda(), post_norm=norm_y,
                                   gate=None if gate is None else gate.cuda(), residual_scale=0.75, pre_weight=pre.cuda(),
                                   packed=True)
        mx_packed.assert_packed(*mx_packed.arrays(q), x, err, (rows, cols, gates, dt, norm_y))


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("rows,cols", [(5, 64), (300, 1024), (2, 4096)])
def test_norm_without_y(rows, cols, dt):
    h = torch.from_numpy(np.random.default_rng(rows).standard_normal((rows, cols))).to(DT[dt])
    x, err = mx_packed.norm_bound(None, h.double().numpy(), None, False, None, 1.0, None, 1e-5)
    _, q = rz.razer_block_norm(None, h.cuda(), packed=True)
    mx_packed.assert_packed(*mx_packed.arrays(q), x, err, (rows, cols, dt))


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("centre", [-95, -80, -40, -5, 0, 5, 40, 90])
def test_gated_encode(centre, dt):
    """Blocks whose gates lie around one value each: where silu is tiny, the block scale is too."""
    rng = np.random.default_rng(centre + 100)
    rows, cols = 70, 544
    g = rng.standard_normal((rows, cols)) * 4 + centre
    gu = torch.from_numpy(np.concatenate([g, rng.standard_normal((rows, cols)) * 3], 1)).to(DT[dt])
    p, err = mx_packed.gated(gu[:, :cols].double().numpy(), gu[:, cols:].double().numpy())
    mx_packed.assert_packed(*mx_packed.arrays(rz.razer_mx_quantize_gated(gu.cuda())), p, err, (centre, dt))
