"""Scales of the product with a scale for each 128 of K at the ends of what the header
allows: their products are fp32's smallest normal number and near its largest."""

import numpy as np
import pytest
import torch

from oracle import codecs

from test_gpu_block import DIRECT, RING, T, f64, multiply, poison

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tile", DIRECT + RING + ["auto"])
@pytest.mark.parametrize("scale_mode", ["block128", "row128"])
@pytest.mark.parametrize("dtype_c", ["f32", "bf16"])
@pytest.mark.parametrize("pa,pb", [(-60, -66), (-126, 0), (20, -126), (60, 59), (127, -8), (-126, 127)])
def test_products_of_scales(tile, scale_mode, dtype_c, pa, pb):
    """Sums of ones, at most 2^8, times powers of two: no rounding anywhere.  One row and one
    column of zeros, whose scales' product may leave the range below."""
    M, N, K = 40, 136, 256
    rng = np.random.default_rng(1)
    a, b = ((rng.random((n, K)) < 0.5) * rng.choice([-1.0, 1.0], (n, 1)) for n in (M, N))
    a[3], b[5] = 0, 0
    sa, sb = np.full((2, M), 2.0 ** pa), np.full((2, N if scale_mode == "row128" else 2), 2.0 ** pb)
    sa[:, 3] = 2.0 ** -126
    C = poison(M, N, dtype=T[dtype_c])
    d = [torch.from_numpy(t).cuda() for t in (codecs.encode("e4m3", a).astype(np.uint8), sa.astype(np.float32),
                                              codecs.encode("e4m3", b).astype(np.uint8), sb.astype(np.float32))]
    multiply(*d, C, M=M, N=N, K=K, dtype_ab="e4m3", dtype_c=dtype_c, scale_mode=scale_mode, tile=tile)
    assert np.array_equal(f64(C), a @ b.T * 2.0 ** (pa + pb))
