"""The norm without an eps: rows whose mean of squares is zero, subnormal in
fp32, or just normal.

The elements are powers of two, so their squares and the sum are exact and the
mean too (2^k columns).  1 / sqrt of a power of two to an even power is exact
in fp32, to an odd one within the reciprocal root's 2^-23 and the scaling is
by a power of two: DELTA of the other tests leaves room."""

import math

import numpy as np
import pytest
import torch

import implicit_gemm_conv_dp_amd as skg
from oracle import codecs, lowp

from test_gpu_norm import DELTA, HALF, T, f64, out

pytestmark = pytest.mark.gpu

# of the mean of squares; fp32 is subnormal below -126 and ends at -149
POWERS = [-149, -148, -147, -140, -139, -128, -127, -126, -125, -120, -101, -100, -99, -60, 0, 100]


def row(power, cols):
    """cols values whose squares have a mean of 2^power."""
    if power % 2:   # one in two columns holds 2^((power + 1) / 2)
        x = torch.zeros(cols, dtype=torch.float64)
        x[::2] = 2.0 ** ((power + 1) // 2)
        return x
    return torch.full((cols,), 2.0 ** (power // 2), dtype=torch.float64)


@pytest.mark.parametrize("cols", [64, 256, 1024, 4096])
def test_reciprocal_root_of_small_means(cols):
    # Squares of 2^-75 and less are below fp32's range: those rows have one
    # larger element instead.
    rows = []
    for p in POWERS:
        x = row(p, cols)
        if p < -146:
            x = torch.zeros(cols, dtype=torch.float64)
            k = int(math.log2(cols))
            if (p + k) % 2:
                x[:2] = 2.0 ** ((p + k - 1) // 2)
            else:
                x[0] = 2.0 ** ((p + k) // 2)
        rows.append(x)
    x = torch.stack(rows).float().cuda()
    n = len(POWERS)
    y, rstd = out((n, cols), torch.float32), out((n,), torch.float32)
    skg.rmsnorm(x, y, rows=n, cols=cols, dtype="f32", rstd=rstd, eps=0.0)
    torch.cuda.synchronize()
    ref, rr = lowp.rmsnorm(f64(x), np.ones(cols), 0.0)
    assert np.all(np.abs(f64(rstd) - rr) <= DELTA * rr), (f64(rstd) / rr)
    assert np.all(np.abs(f64(y) - ref) <= (DELTA + HALF["f32"]) * np.abs(ref))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_empty_rows(dtype):
    """1 / sqrt(0) is infinite, and 0 times it is no number."""
    rows, cols = 5, 320
    x = torch.ones(rows, cols).to(T[dtype]).cuda()
    x[1] = 0
    x[3] = -0.0
    y, rstd = out((rows, cols), T[dtype]), out((rows,), torch.float32)
    skg.rmsnorm(x, y, rows=rows, cols=cols, dtype=dtype, rstd=rstd, eps=0.0)
    q, sc = out((rows, cols), torch.uint8), out((rows,), torch.float32)
    skg.rmsnorm(x, q, rows=rows, cols=cols, dtype=dtype, y_scale=sc, dtype_y="e4m3", eps=0.0)
    torch.cuda.synchronize()
    empty, rest = [1, 3], [0, 2, 4]
    assert (rstd[empty] == float("inf")).all() and (rstd[rest] == 1).all()
    assert torch.isnan(y[empty].float()).all() and (y[rest] == 1).all()
    codes = codecs.decode("e4m3", q.cpu().numpy())
    assert torch.isnan(sc[empty]).all() and np.isnan(codes[empty]).all()
    assert (codes[rest] == 448).all()
