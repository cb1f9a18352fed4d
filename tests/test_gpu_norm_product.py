"""The norm's 8- and 4-bit outputs as the operand of the product that follows:
e4m3 codes with row scales as A and scale_a, MX blocks of e4m3 and e2m1 with
their scales.

Rows of +-1 without an eps have the factor 1, so y is +-gain; with gains that the
codes hold, and a largest one of which 1/448 is a power of two where a row has
one scale, codes and scales are exact and so is every sum: the product has to
be that of the values, to the bit."""

import pytest
import torch

import implicit_gemm_conv_dp_amd as skg

from test_gpu_norm import T, out

pytestmark = pytest.mark.gpu

SHAPES = [(1, 72, 128), (37, 264, 640), (200, 136, 2048), (300, 520, 4096)]
GAINS = {"e4m3": [1, 2, 3, 4, 5, 6, 7], "e2m1": [1, 2, 3, 4, 6]}


def signs(seed, rows, cols):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, 2, (rows, cols), generator=g).mul(2).sub(1)


def layer(M, N, K, fmt):
    """(x, residual, gain, weight) as float64 on the CPU: x + residual is +-1,
    the weight holds small whole numbers with a 7 in every row."""
    h = signs(71, M, K).double()
    r = signs(72, M, K).double() * 2
    g = torch.Generator().manual_seed(73)
    pick = torch.tensor(GAINS[fmt], dtype=torch.float64)
    gain = pick[torch.randint(0, len(pick), (K,), generator=g)]
    gain[K // 3] = pick[-1]
    w = pick[torch.randint(0, len(pick), (N, K), generator=g)] * signs(74, N, K)
    w[:, 5] = pick[-1]
    return h - r, r, gain, w


def dev(t):
    return t.to(torch.bfloat16).cuda()


@pytest.mark.parametrize("dtype_c", ["bf16", "f32"])
@pytest.mark.parametrize("tile", ["128x128x128", "256x256x128"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_row_scales(M, N, K, tile, dtype_c):
    x, r, gain, w = layer(M, N, K, "e4m3")
    q, sa = out((M, K), torch.uint8), out((M,), torch.float32)
    skg.rmsnorm(dev(x), q, rows=M, cols=K, dtype="bf16", weight=dev(gain), residual=dev(r), y_scale=sa,
                dtype_y="e4m3", eps=0.0)
    # the weight's codes by hand, 64 to its 1
    wq, sb = (w * 64).to(torch.float8_e4m3fn).cuda(), torch.full((N,), 1 / 64, device="cuda")
    R = ((x + r) * gain) @ w.t().contiguous()
    for mode, red, ctas in (("dp", "linear", 1), ("dp_sk", "tree", 5)):
        C = out((M, N), T[dtype_c])
        skg.gemm(q, wq, C, sa, sb, M=M, N=N, K=K, dtype_ab="e4m3", dtype_c=dtype_c, tile=tile, mode=mode,
                 reduction=red, ctas=ctas)
        torch.cuda.synchronize()
        assert torch.equal(C.cpu(), R.to(T[dtype_c])), mode


@pytest.mark.parametrize("dtype_c", ["bf16", "f32"])
@pytest.mark.parametrize("fmt,tile", [("e4m3", "128x128x128"), ("e4m3", "256x256x128"), ("e2m1", "auto"),
                                      ("e2m1", "256x256x256")])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_mx_blocks(M, N, K, fmt, tile, dtype_c):
    x, r, gain, w = layer(M, N, K, fmt)
    width = K if fmt == "e4m3" else K // 2
    q, sa = out((M, width), torch.uint8), out((M, K // 32), torch.uint8)
    skg.rmsnorm(dev(x), q, rows=M, cols=K, dtype="bf16", weight=dev(gain), residual=dev(r), y_scale=sa,
                dtype_y=fmt, scale_mode="mx", eps=0.0)
    wq, sb = out((N, width), torch.uint8), out((N, K // 32), torch.uint8)
    skg.mx_quant(dev(w), wq, sb, rows=N, cols=K, dtype="bf16", dtype_q=fmt)
    C = out((M, N), T[dtype_c])
    skg.gemm(q, wq, C, sa, sb, M=M, N=N, K=K, dtype_ab=fmt, dtype_c=dtype_c, tile=tile, mode="dp",
             reduction="linear", ctas=1, scale_mode="mx")
    torch.cuda.synchronize()
    R = ((x + r) * gain) @ w.t().contiguous()
    assert torch.equal(C.cpu(), R.to(T[dtype_c]))
