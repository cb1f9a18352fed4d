"""The 4-bit product's stream-K modes captured into a graph, every fix-up:
integer-exact operands, so that the atomic one has the same bits too, replayed
with other work between, C and the workspace spoilt before each replay."""

import numpy as np
import pytest
import torch

import implicit_gemm_conv_dp_amd as skg
from oracle import lowp

from test_gpu_fp4 import LAUNCHES, TILES, dev, f64, operand, poison

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pad", [0, 8])
@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("mode,red,ctas", [x for x in LAUNCHES if x[0] != "dp"])
def test_graph_of_stream_k(tile, mode, red, ctas, pad):
    tm = int(tile.split("x")[0])
    M, N, K = tm + 40, tm + 72, 9 * 256
    (aq, as_), (bq, bs) = operand(31, M, K, True), operand(32, N, K, True)
    a, sa, b, sb = dev(lowp.pack(aq)), dev(as_), dev(lowp.pack(bq)), dev(bs)
    B = lowp.mx_values(bs, bq, "e2m1")
    C = poison((M, N + pad), torch.float32)
    kw = dict(M=M, N=N, K=K, ldc=N + pad, dtype_ab="e2m1", dtype_c="f32", scale_mode="mx", tile=tile, mode=mode,
              reduction=red, ctas=ctas)
    plan = skg.plan_gemm(**kw)
    assert plan["sk_ctas"] > 0
    ws = skg.workspace_for(plan, "cuda")
    skg.gemm(a, b, C, sa, sb, workspace=ws, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        skg.gemm(a, b, C, sa, sb, workspace=ws, **kw)
    for i in range(4):
        q, s = operand(40 + i, M, K, True)
        R = lowp.mx_values(s, q, "e2m1") @ B.T
        a.copy_(dev(lowp.pack(q)))
        sa.copy_(dev(s))
        for again in range(2):
            C.view(torch.uint8).fill_(0xFF)
            ws.fill_(0xFF)
            if again:
                skg.gemm(a, b, C, sa, sb, workspace=ws, **kw)
            else:
                g.replay()
            torch.cuda.synchronize()
            got = f64(C)
            assert np.array_equal(got[:, :N], R), (i, again, np.nanmax(np.abs(got[:, :N] - R)))
            assert np.isnan(got[:, N:]).all()
