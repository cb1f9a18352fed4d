"""The weight's gradient has the same bits wherever dx is written, at sizes
that take one launch and sizes that take two."""

import pytest
import torch

import implicit_gemm_conv_dp_amd as skg

from test_gpu_norm import EPS, T, out, rows_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 5), (33, 8), (509, 1111), (1024, 1024), (64, 16384), (65, 16384), (1025, 300)])
def test_weight_gradient_in_place(rows, cols, dtype):
    h, dy, dres = (rows_of(s, rows, cols, dtype) for s in (50, 51, 52))
    rstd = torch.rsqrt(h.double().square().mean(1) + EPS).float()
    kw = dict(rows=rows, cols=cols, dtype=dtype, dres=dres)
    dx, dw = out((rows, cols), T[dtype]), out((cols,), torch.float32)
    skg.rmsnorm_bwd(dy, h, rstd, dx, dw=dw, **kw)
    over_dy, over_h, dw2, dw3 = dy.clone(), h.clone(), torch.empty_like(dw), torch.empty_like(dw)
    skg.rmsnorm_bwd(over_dy, h, rstd, over_dy, dw=dw2, **kw)
    skg.rmsnorm_bwd(dy, over_h, rstd, over_h, dw=dw3, **kw)
    torch.cuda.synchronize()
    for t in (over_dy, over_h):
        assert torch.equal(t, dx)
    for t in (dw2, dw3):
        assert torch.equal(t, dw)
