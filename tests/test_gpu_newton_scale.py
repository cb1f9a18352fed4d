"""The smallest scale of the Newton-Schulz update: a power of two only moves the
exponents of the last step's factors, so the result is the unscaled one times it."""

import pytest
import torch

import implicit_gemm_conv_dp_amd as skg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tile", skg.NS_TILES)
@pytest.mark.parametrize("rows,cols", [(150, 210), (210, 150)])
def test_smallest_scale(tile, rows, cols):
    g = torch.randn(rows, cols, generator=torch.Generator().manual_seed(1)).cuda()
    one, small, none = (torch.full((rows, cols), float("nan"), device="cuda") for _ in range(3))
    for out, scale in ((one, 1.0), (small, 2.0 ** -100), (none, 0.0)):
        skg.newton_schulz(g, out, rows=rows, cols=cols, dtype="f32", scale=scale, tile=tile)
    assert torch.equal(small, one * 2.0 ** -100) and one.abs().max() > 0.01
    assert not none.any()
