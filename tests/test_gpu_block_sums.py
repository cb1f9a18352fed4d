"""Sums of the product with a scale for each 128 of K where a channel of each block
is far larger than the others, alone or cancelled by another, against float64.

f16 and f32 outputs hold sums of exact products: with each of the K additions and
the blocks' scalings off by at most one unit of 2^-23 of the sum of magnitudes,
(K + 16) 2^-23 of that sum bounds them, and the output's rounding adds half a step.

bf16 outputs come from instructions that cut the products of eight consecutive K
towards zero to multiples of 2^(E - 13), E the largest sum of two codes' exponents
(a subnormal code's, and a zero's here, as the smallest normal one's): each of the
group's products but the one of E loses less than one such multiple (that one, of
two factors of at most 4 bits, is a multiple of 2^(E - 6)), so 7 2^(E - 13) a group,
times the block's scales, comes on top."""

import numpy as np
import pytest
import torch

import implicit_gemm_conv_dp_amd as skg
from oracle import codecs, projection as pj

from test_gpu_block import DIRECT, HALF, RING, T, TINY, f64, multiply, poison

pytestmark = pytest.mark.gpu

LOWEST = {"e4m3": -6, "e5m2": -14}   # exponent of the smallest normal code


def operands(fmt, block, M, N, K, factor, cancel, positive, seed=0):
    """Quantised operands whose channel 3 of each block is ``factor`` larger, and
    channel 5 (of the same eight) its negative counterpart where ``cancel``."""
    rng = np.random.default_rng(seed)
    x, w = rng.standard_normal((M, K)), rng.standard_normal((N, K))
    if positive:
        x, w = np.abs(x), np.abs(w)
    x[:, 3::128] *= factor
    w[:, 3::128] *= factor
    if cancel:
        x[:, 5::128], w[:, 5::128] = x[:, 3::128], -w[:, 3::128]
    out = []
    for v, b in ((x / factor, "1x128"), (w / factor, block)):   # (an f16 output's range)
        s, q = pj.block_quantize(v, fmt, b)
        s = s.astype(np.float32)
        out.append((torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), pj.block_values(s, q, fmt, b), q))
    return out


def cut(fmt, a, b, sa, sb, scale_mode):
    """Largest sum of what the groups of eight lose."""
    M, K = a.shape
    N = b.shape[0]
    ea, eb = (np.floor(np.log2(np.maximum(np.abs(codecs.decode(fmt, q)), 2.0 ** LOWEST[fmt]))) for q in (a, b))
    if scale_mode == "block128":
        sb = np.repeat(sb, 128, axis=1)[:, :N]
    out = np.zeros((M, N))
    for k in range(0, K, 8):
        E = (ea[:, None, k:k + 8] + eb[None, :, k:k + 8]).max(2)
        out += 7 * 2.0 ** (E - 13) * sa[k // 128][:, None] * sb[k // 128]
    return out


@pytest.mark.parametrize("tile", DIRECT + RING + ["auto"])
@pytest.mark.parametrize("scale_mode", ["block128", "row128"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("factor,cancel,positive", [(2.0 ** 6, False, False), (2.0 ** 10, False, True),
                                                    (2.0 ** 6, True, False), (2.0 ** 10, True, True)])
def test_larger_channels(tile, scale_mode, fmt, factor, cancel, positive):
    M, N, K = 70, 136, 384
    block = "128x128" if scale_mode == "block128" else "1x128"
    (a, sa, A, qa), (b, sb, B, qb) = operands(fmt, block, M, N, K, factor, cancel, positive)
    want, size = A @ B.T, np.abs(A) @ np.abs(B).T
    sums = (K + 16) * 2.0 ** -23 * size
    lost = cut(fmt, qa, qb, f64(sa), f64(sb), scale_mode)
    for dtype_c in ("f32", "f16", "bf16"):
        C = poison(M, N, dtype=T[dtype_c])
        multiply(a, sa, b, sb, C, M=M, N=N, K=K, dtype_ab=fmt, dtype_c=dtype_c, scale_mode=scale_mode, tile=tile)
        tol = sums + (lost if dtype_c == "bf16" else 0)
        tol = tol + HALF[dtype_c] * (np.abs(want) + tol) + TINY[dtype_c]
        off = np.abs(f64(C) - want)
        assert np.all(off <= tol), (dtype_c, (off / tol).max())


@pytest.mark.parametrize("tile", DIRECT + RING)
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_subnormal_codes(tile, fmt):
    """Products of subnormal codes alone: whole multiples of the smallest one, whose sums
    of 128 are exact in fp32, and nothing of them is cut."""
    M, N, K = 40, 56, 128
    rng = np.random.default_rng(1)
    n = 8 if fmt == "e4m3" else 4
    a, b = (rng.integers(0, n, (rows, K)) | rng.integers(0, 2, (rows, K)) << 7 for rows in (M, N))
    one = torch.ones(1, M, device="cuda"), torch.ones(1, N, device="cuda")
    want = codecs.decode(fmt, a) @ codecs.decode(fmt, b).T
    for dtype_c in ("f32", "bf16"):
        C = poison(M, N, dtype=T[dtype_c])
        multiply(torch.from_numpy(a.astype(np.uint8)).cuda(), one[0], torch.from_numpy(b.astype(np.uint8)).cuda(), one[1], C,
                 M=M, N=N, K=K, dtype_ab=fmt, dtype_c=dtype_c, scale_mode="row128", tile=tile)
        assert np.array_equal(f64(C), f64(torch.from_numpy(want).to(T[dtype_c]))), dtype_c
