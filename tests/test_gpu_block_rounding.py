"""Block quantisation of fp32 elements next to the borders between two codes: the
nearest code, of the real quotient, has to come out.

An element is a border times its block's largest magnitude over MAX, rounded to fp32,
or one of that number's neighbours, so its quotient is within some 2^-23 of the
border.  x MAX has at most 27 bits and a border times the block's largest magnitude
at most 29, so a quotient that is not on a border is 2^-30 of itself away from it, and
one in float64 (2^-53) stays on its side: the oracle's codes are exact."""

import numpy as np
import pytest
import torch

import implicit_gemm_conv_dp_amd as skg
from oracle import codecs, projection as pj

from test_gpu_block import poison

pytestmark = pytest.mark.gpu


def near_borders(seed, rows, cols, fmt, block, power, zeros=0.0):
    rng = np.random.default_rng(seed)
    v = codecs.decode(fmt, np.arange(128))
    v = np.sort(v[np.isfinite(v)])
    borders = (v[1:] + v[:-1]) / 2
    h = 128 if block == "128x128" else 1
    top = rng.uniform(1, 2, (-(-rows // h), cols // 128)).astype(np.float32).astype(np.float64) * 2.0 ** power
    wide = np.repeat(np.repeat(top, h, axis=0), 128, axis=1)[:rows]
    x = (rng.choice(borders, (rows, cols)) * wide / pj.LARGEST[fmt]).astype(np.float32)
    x = (x.view(np.int32) + rng.integers(-1, 2, x.shape, dtype=np.int32)).view(np.float32)
    x = np.minimum(x, wide.astype(np.float32)) * rng.choice([-1, 1], x.shape).astype(np.float32)
    x[::h, ::128] = wide[::h, ::128]
    x[rng.random(x.shape) < zeros] = 0.0
    x[rng.random(x.shape) < zeros] = -0.0
    return x


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("block", ["1x128", "128x128"])
@pytest.mark.parametrize("along", ["rows", "columns", "both"])
@pytest.mark.parametrize("power", [0, -100, 126])
def test_elements_next_to_a_border(fmt, block, along, power):
    # "both" reads one matrix twice over: blocks along its rows have the tops that are
    # planned, those along its columns some border's
    rows, cols = 261, 256
    x = near_borders(abs(power) + len(along), rows, cols, fmt, block, power)
    if along == "columns":
        x = np.ascontiguousarray(x.T)
    n, k = x.shape
    tall = block == "128x128"
    kq, kqt = pj.up(k, 128), pj.up(n, 128)
    q, qt = poison(n, kq), poison(k, kqt)
    s = poison(kq // 128, -(-n // 128) if tall else n, dtype=torch.float32)
    st = poison(kqt // 128, -(-k // 128) if tall else k, dtype=torch.float32)
    r, c = along != "columns", along != "rows"
    skg.block_quant(torch.from_numpy(x).cuda(), q if r else None, s if r else None, qt if c else None, st if c else None,
                    rows=n, cols=k, dtype="f32", dtype_q=fmt, block=block)
    torch.cuda.synchronize()
    for wanted, m, got, scales in ((r, x, q, s), (c, x.T, qt, st)):
        if wanted:
            ws, wq = pj.block_quantize(m.astype(np.float64), fmt, block)
            assert np.array_equal(scales.cpu().numpy(), ws)
            assert np.array_equal(got.cpu().numpy(), wq), (got.cpu().numpy() != wq).sum()


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("block", ["1x128", "128x128"])
def test_zeros_next_to_such_elements(fmt, block):
    """Zeros of both signs and quotients far below the smallest code keep their signs."""
    x = near_borders(7, 130, 256, fmt, block, 0, zeros=0.2)
    x[5, 1:] *= np.float32(2.0 ** -60)
    q, qt = poison(130, 256), poison(256, 256)
    tall = block == "128x128"
    s, st = poison(2, 2 if tall else 130, dtype=torch.float32), poison(2, 2 if tall else 256, dtype=torch.float32)
    skg.block_quant(torch.from_numpy(x).cuda(), q, s, qt, st, rows=130, cols=256, dtype="f32", dtype_q=fmt, block=block)
    torch.cuda.synchronize()
    for m, got in ((x, q), (x.T, qt)):
        assert np.array_equal(got.cpu().numpy()[:, :m.shape[1]], pj.block_quantize(m.astype(np.float64), fmt, block)[1][:, :m.shape[1]])
