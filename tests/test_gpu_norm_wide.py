"""Gradients of wide rows where a workgroup of 8 or 16 waves takes several rows
in turn (more than 256 of them), its two sets of reduction slots alternating."""

import numpy as np
import pytest
import torch

import implicit_gemm_conv_dp_amd as skg
from oracle import lowp

from test_gpu_norm import EPS, HALF, T, f64, out, rows_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(257, 4104), (600, 4099), (520, 8200), (777, 8191), (300, 16385), (520, 12000),
                                       (300, 32768)])
def test_wide_gradients(rows, cols, dtype):
    h, dy, dres = (rows_of(s, rows, cols, dtype) for s in (60, 61, 62))
    w = rows_of(63, 1, cols, "f32").reshape(-1)
    rstd = torch.rsqrt(h.double().square().mean(1) + EPS).float()
    kw = dict(rows=rows, cols=cols, dtype=dtype, weight=w, dtype_w="f32", dres=dres)
    dx, dw = out((rows, cols), T[dtype]), out((cols,), torch.float32)
    skg.rmsnorm_bwd(dy, h, rstd, dx, dw=dw, **kw)
    for _ in range(3):
        dx2, dw2 = out((rows, cols), T[dtype]), out((cols,), torch.float32)
        skg.rmsnorm_bwd(dy, h, rstd, dx2, dw=dw2, **kw)
        torch.cuda.synchronize()
        assert torch.equal(dx2, dx) and torch.equal(dw2, dw)
    H, DY, W, S, R = (f64(t) for t in (h, dy, w, rstd, dres))
    rx, rw = lowp.rmsnorm_bwd(DY, H, S, W)
    rx = rx + R
    u = 2.0 ** -24
    n, g = H * S[:, None], DY * W
    # as in the gradient's tests at other widths
    tol = S[:, None] * (8 * u * np.abs(g) + np.abs(n) * 80 * u * np.mean(np.abs(g * n), 1, keepdims=True))
    tiny = float(torch.finfo(T[dtype]).smallest_normal) * HALF[dtype] * 2
    tol = tol + 8 * u * np.abs(R) + HALF[dtype] * np.abs(rx) * (1 + 2.0 ** -10) + tiny
    assert np.all(np.abs(f64(dx) - rx) <= tol)
    assert np.all(np.abs(f64(dw) - rw) <= (rows + 4) * u * np.sum(np.abs(DY * n), 0) + 2.0 ** -126)
