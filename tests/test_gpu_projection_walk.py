"""Products and updates of more tiles than there are CUs, on which a workgroup takes
tile after tile: the next tile's first stages travel behind the last one's copy-out,
through the ring's entries where that one left them.  Odd tile counts and, for the
products, reductions of a number of stages that no ring's depth divides."""

import functools

import numpy as np
import pytest
import torch

import implicit_gemm_conv_dp_amd as skg
from oracle import projection as pj

from test_gpu_block import DIRECT, RING, T, f64, multiply, operand, poison
from test_gpu_newton import EPS, HALF, MUON

pytestmark = pytest.mark.gpu


@functools.lru_cache(maxsize=2)
def whole_numbers(M, N, K, fmt, block):
    a, sa, A = operand(1, M, K, fmt, "1x128", True)
    b, sb, B = operand(2, N, K, fmt, block, True)
    return a, sa, b, sb, A @ B.T


def check_product(M, N, K, fmt, scale_mode, tile, dtype_c):
    """Sums of small whole numbers times powers of two, exact in fp32; no product is cut by
    the 8-bit instructions; then one rounding."""
    a, sa, b, sb, want = whole_numbers(M, N, K, fmt, "128x128" if scale_mode == "block128" else "1x128")
    ldc = pj.up(N, 8) + 8
    C = poison(M, ldc, dtype=T[dtype_c])
    multiply(a, sa, b, sb, C, M=M, N=N, K=K, ldc=ldc, dtype_ab=fmt, dtype_c=dtype_c, scale_mode=scale_mode, tile=tile)
    got = f64(C)
    assert np.array_equal(got[:, :N], f64(torch.from_numpy(want).to(T[dtype_c]))) and np.isnan(got[:, N:]).all()


@pytest.mark.parametrize("tile,M,N,K", [("128x128x128", 2201, 2190, 640), ("256x128x128", 4201, 2190, 640),
                                        ("256x256x128", 4201, 4190, 640), ("128x128x128", 2201, 2190, 256)])
@pytest.mark.parametrize("scale_mode", ["block128", "row128"])
@pytest.mark.parametrize("dtype_c", ["f32", "f16", "bf16"])
def test_product(tile, M, N, K, scale_mode, dtype_c):
    check_product(M, N, K, "e4m3" if scale_mode == "block128" else "e5m2", scale_mode, tile, dtype_c)


@pytest.mark.parametrize("tile", DIRECT + RING + ["auto"])
@pytest.mark.parametrize("scale_mode", ["block128", "row128"])
@pytest.mark.parametrize("dtype_c", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(17, 40, 384), (257, 520, 256)])
def test_product_of_one_round_to_16_bits(tile, scale_mode, dtype_c, M, N, K):
    check_product(M, N, K, "e4m3", scale_mode, tile, dtype_c)


def steps(g, coefficients, rounded):
    """oracle.projection.newton_schulz in float64 on the GPU."""
    def keep(v, power):
        return (v * 2.0 ** power).half().double() * 2.0 ** -power if rounded else v

    tall = g.shape[0] > g.shape[1]
    x = g.double().t().contiguous() if tall else g.double()
    x = keep(x / (x.square().sum().sqrt() + EPS), 13)
    for i, (a, b, c) in enumerate(coefficients):
        s = keep(x @ x.t(), 12)
        p = b * s + c * (s @ s)
        d = torch.diag(torch.diag(p))
        p = keep(p - d, 11) + d
        x = a * x + p @ x
        if i + 1 < len(coefficients):
            x = keep(x, 13)
    return x.t() if tall else x


# Symmetric products of more than 256 tiles have 23 rows of them (an update's wider
# product has more): 128 x 128 and 192 x 192 here; 256 x 256, 256 x 192 and 320 x 256
# walk in the wider one.
@pytest.mark.parametrize("tile,rows,cols,dtype_out", [
    ("128x128", 2900, 2950, "f32"), ("128x128", 2950, 2900, "bf16"), ("192x192", 4300, 4250, "bf16"),
    ("256x192", 4250, 4300, "f32"), ("256x256", 4300, 4250, "f16"), ("320x256", 5200, 5250, "bf16"),
    ("256x256", 5700, 5650, "f32"), ("auto", 2900, 2900, "bf16")])
def test_update(tile, rows, cols, dtype_out):
    """As on small matrices (the distance from the unrounded steps is at most half as much
    again as the rounded steps' own); and nowhere, in squares of 128, more than twice
    that: an entry's error is a sum of thousands of roundings, so those of a square
    hardly differ in size."""
    gen = torch.Generator(device="cuda").manual_seed(rows)
    r = rows // 8
    g = torch.randn(rows, r, generator=gen, device="cuda") @ torch.randn(r, cols, generator=gen, device="cuda") / r ** 0.5
    g = 1e-3 * (g + 0.5 * torch.randn(rows, cols, generator=gen, device="cuda"))
    cs = (MUON,) * 2
    out = torch.full((rows, cols + 8), float("nan"), dtype=T[dtype_out], device="cuda")
    skg.newton_schulz(g, out, rows=rows, cols=cols, dtype="f32", dtype_out=dtype_out, steps=2, ldo=cols + 8, tile=tile)
    torch.cuda.synchronize()
    assert torch.isnan(out[:, cols:]).all()
    want = steps(g, cs, False)
    near = steps(g, cs, True)
    got = out[:, :cols].double()
    n = want.norm()
    own = (near - want).norm()
    bound = 1.5 * own + (2.0 ** -14 + HALF[dtype_out]) * n
    off = got - want
    assert off.norm() <= bound, (off.norm() / n, own / n)
    R, C = -(-rows // 128) * 128, -(-cols // 128) * 128
    pad = torch.zeros(R, C, dtype=torch.float64, device="cuda")
    pad[:rows, :cols] = off
    squares = pad.reshape(R // 128, 128, C // 128, 128).square().sum((1, 3)).sqrt()
    assert squares.max() <= 2 * bound * 128 / (rows * cols) ** 0.5
    del pad, off, got, want, near, out, g
    torch.cuda.empty_cache()


def test_repeated_updates_give_the_same_bits():
    gen = torch.Generator(device="cuda").manual_seed(3)
    g = torch.randn(2900, 3100, generator=gen, device="cuda")
    first = None
    for _ in range(3):
        out = torch.full((2900, 3100), float("nan"), device="cuda")
        skg.newton_schulz(g, out, rows=2900, cols=3100, dtype="f32", steps=2, tile="128x128")
        first = out if first is None else first
        assert torch.equal(out, first)
