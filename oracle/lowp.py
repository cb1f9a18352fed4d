"""Low-precision layer operators in float64 (oracle side).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

* MX blocks of e2m1 or e4m3 elements: OCP Microscaling formats with one E8M0
  scale per 32 elements; the scale's exponent is that of the block's largest
  magnitude less the element format's largest exponent.
* e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 by codes 0..7, sign in bit 3; two codes a
  byte, the even element in the low four bits.
* Root-mean-square norm and its gradient, written from the definition.
"""

import numpy as np

from . import codecs

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
EMAX = {"e2m1": 2, "e4m3": 8}


def decode_e2m1(codes):
    c = np.asarray(codes).astype(np.int64)
    return np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]


def encode_e2m1(x):
    """Nearest code, ties to the even code, saturating at 6."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 6.0)
    hi = np.clip(np.searchsorted(E2M1, a, side="left"), 0, 7)
    lo = np.maximum(hi - 1, 0)
    up, down = E2M1[hi] - a, a - E2M1[lo]
    code = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    return (code | np.where(np.signbit(x), 8, 0)).astype(np.uint8)


def pack(codes):
    c = np.asarray(codes, dtype=np.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def unpack(packed):
    p = np.asarray(packed, dtype=np.uint8)
    out = np.empty(p.shape[:-1] + (2 * p.shape[-1],), dtype=np.uint8)
    out[..., 0::2] = p & 15
    out[..., 1::2] = p >> 4
    return out


def encode(fmt, x):
    return encode_e2m1(x) if fmt == "e2m1" else codecs.encode("e4m3", x)


def decode(fmt, codes):
    return decode_e2m1(codes) if fmt == "e2m1" else codecs.decode("e4m3", codes)


def scale_value(codes):
    c = np.asarray(codes).astype(np.int64)
    return np.where(c == 255, np.nan, np.ldexp(1.0, np.minimum(c, 254) - 127))


def mx_scales(x, fmt):
    """E8M0 codes of the blocks of 32 along the last axis."""
    b = np.asarray(x, dtype=np.float64).reshape(x.shape[:-1] + (-1, 32))
    top = np.max(np.abs(b), axis=-1)
    bad = ~np.isfinite(top)
    e = np.frexp(np.where(bad | (top == 0), 1.0, top))[1] - 1
    code = np.where(top == 0, 0, np.maximum(e - EMAX[fmt] + 127, 0))
    return np.where(bad, 255, code).astype(np.uint8)


def mx_quantize(x, fmt):
    """(scale codes, element codes) of float64 ``x`` along its last axis, whose
    length is a multiple of 32."""
    x = np.asarray(x, dtype=np.float64)
    s = mx_scales(x, fmt)
    d = np.repeat(scale_value(s), 32, axis=-1)
    with np.errstate(invalid="ignore"):
        q = encode(fmt, np.where(np.isnan(d), 0.0, x / d))
    return s, np.where(np.isnan(d), 0, q).astype(np.uint8)


def mx_values(s, q, fmt):
    return decode(fmt, q) * np.repeat(scale_value(s), 32, axis=-1)


def rmsnorm(h, w, eps):
    """(y, rstd) of float64 rows."""
    rstd = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
    return h * rstd[:, None] * w, rstd


def rmsnorm_bwd(dy, h, rstd, w):
    """(dx, dw) of float64 rows, without what the residual stream adds."""
    g = dy * w
    dot = np.mean(g * h, axis=1, keepdims=True)
    r = rstd[:, None]
    return r * (g - h * r * r * dot), np.sum(dy * h * r, axis=0)
