"""Pins of the low-precision oracle: the e2m1 code table and its roundings,
MX scales against the exponent by definition, the norm against its closed
forms and its gradient against differences."""

import numpy as np
import pytest

from oracle import lowp


def test_e2m1_round_trip_and_ties():
    codes = np.arange(16)
    assert np.array_equal(lowp.encode_e2m1(lowp.decode_e2m1(codes)), codes)
    mids = (lowp.E2M1[:-1] + lowp.E2M1[1:]) / 2
    for i, m in enumerate(mids):
        assert lowp.encode_e2m1(m) == (i if i % 2 == 0 else i + 1)
        assert lowp.encode_e2m1(np.nextafter(m, 0)) == i
        assert lowp.encode_e2m1(np.nextafter(m, 9)) == i + 1
        assert lowp.encode_e2m1(-m) == (i if i % 2 == 0 else i + 1) + 8
    assert lowp.encode_e2m1(100.0) == 7 and lowp.encode_e2m1(-7.0) == 15


def test_pack():
    c = np.arange(16, dtype=np.uint8).reshape(1, 16)
    assert lowp.pack(c)[0, 0] == 0x10 and np.array_equal(lowp.unpack(lowp.pack(c)), c)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_mx_scales_by_definition(fmt):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((5, 96)) * np.exp2(rng.integers(-40, 40, (5, 1)))
    s, q = lowp.mx_quantize(x, fmt)
    top = np.abs(x.reshape(5, 3, 32)).max(-1)
    assert np.array_equal(s.astype(int) - 127, np.floor(np.log2(top)).astype(int) - lowp.EMAX[fmt])
    big = {"e2m1": 6.0, "e4m3": 448.0}[fmt]
    assert np.abs(lowp.decode(fmt, q)).max() <= big
    x[0, 3], x[1, 40], x[2, 64:] = np.nan, np.inf, 0
    s, q = lowp.mx_quantize(x, fmt)
    assert s[0, 0] == 255 and s[1, 1] == 255 and s[2, 2] == 0
    assert not q[0, :32].any() and not q[2, 64:].any()


def test_norm_and_gradient():
    rng = np.random.default_rng(4)
    h, w, dy = rng.standard_normal((3, 7)), rng.standard_normal(7), rng.standard_normal((3, 7))
    y, r = lowp.rmsnorm(h, w, 0.0)
    assert np.allclose(np.mean((y / w) ** 2, axis=1), 1)
    eps = 1e-3
    y, r = lowp.rmsnorm(h, w, eps)
    dx, dw = lowp.rmsnorm_bwd(dy, h, r, w)
    d = 1e-6
    for i in range(3):
        for j in range(7):
            p, m = h.copy(), h.copy()
            p[i, j] += d
            m[i, j] -= d
            num = np.sum((lowp.rmsnorm(p, w, eps)[0] - lowp.rmsnorm(m, w, eps)[0]) * dy) / (2 * d)
            # central differences: d^2 of curvature and rounding / d
            assert abs(num - dx[i, j]) < 1e-7
    for j in range(7):
        p, m = w.copy(), w.copy()
        p[j] += d
        m[j] -= d
        num = np.sum((lowp.rmsnorm(h, p, eps)[0] - lowp.rmsnorm(h, m, eps)[0]) * dy) / (2 * d)
        assert abs(num - dw[j]) < 1e-7
