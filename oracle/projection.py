"""Operators of an 8-bit attention projection in float64 (oracle side).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

* Blocks of 128: codes of e4m3 or e5m2 with one fp32 scale for 1 x 128 or
  128 x 128 elements, and the product of such operands.
* Norms of heads with the rotation of pairs, and their gradient.
* Newton-Schulz steps, and the same with the factors rounded to fp16.
"""

import numpy as np

from . import codecs

LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
FLOOR = 2.0 ** -126


def up(n, m):
    return -(-n // m) * m


def block_tops(x, block):
    """Largest magnitudes of the blocks of ``x`` padded to whole blocks, and the
    padded matrix."""
    rows, cols = x.shape
    h = 128 if block == "128x128" else 1
    p = np.zeros((up(rows, h), up(cols, 128)))
    p[:rows, :cols] = x
    b = np.abs(p).reshape(p.shape[0] // h, h, p.shape[1] // 128, 128)
    return b.max(axis=(1, 3)), p, h


def block_quantize(x, fmt, block="1x128", slack=0.0):
    """(scales as K/128 lines of blocks, codes of the rows padded to whole
    blocks) of finite float64 ``x``; ``slack`` moves every quotient by that much
    of itself before it is rounded."""
    rows = x.shape[0]
    top, p, h = block_tops(np.asarray(x, dtype=np.float64), block)
    top = np.maximum(top, LARGEST[fmt] * FLOOR)
    wide = np.repeat(np.repeat(top, h, axis=0), 128, axis=1)
    q = codecs.encode(fmt, np.clip(p * LARGEST[fmt] / wide * (1 + slack), -LARGEST[fmt], LARGEST[fmt]))
    return np.ascontiguousarray((top / LARGEST[fmt]).astype(np.float32).T), q[:rows].astype(np.uint8)


def block_values(scales, codes, fmt, block="1x128"):
    d = np.asarray(scales, dtype=np.float64).T
    if block == "128x128":
        d = np.repeat(d, 128, axis=0)[:codes.shape[0]]
    return codecs.decode(fmt, codes) * np.repeat(d, 128, axis=1)


def rotate(v, cos, sin, style, back=False):
    """(tokens, heads, dim) with pairs turned by the tokens' angles."""
    half = cos.shape[1]
    c, s = cos[:, None, :], (-sin if back else sin)[:, None, :]
    out = np.array(v, dtype=np.float64)
    i, j = (slice(0, half), slice(half, 2 * half)) if style == "half" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    a, b = out[..., i].copy(), out[..., j].copy()
    out[..., i] = a * c - b * s
    out[..., j] = b * c + a * s
    return out


def turned_size(v, cos, sin, style):
    """Sum of the magnitudes that an element of ``rotate`` is made of."""
    half = cos.shape[1]
    c, s = np.abs(cos)[:, None, :], np.abs(sin)[:, None, :]
    out = np.abs(np.array(v, dtype=np.float64))
    i, j = (slice(0, half), slice(half, 2 * half)) if style == "half" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    a, b = out[..., i].copy(), out[..., j].copy()
    out[..., i] = a * c + b * s
    out[..., j] = b * c + a * s
    return out


def head_norm(x, w, eps):
    """(n, rstd) of heads (tokens, heads, dim)."""
    r = 1 / np.sqrt(np.mean(x * x, axis=2, keepdims=True) + eps)
    return x * r * w, r


def head_norm_bwd(dy, x, w, eps, cos, sin, style):
    """(dx, dw, the sizes of the terms of both)."""
    g = rotate(dy, cos, sin, style, back=True)
    size = turned_size(dy, cos, sin, style)
    r = 1 / np.sqrt(np.mean(x * x, axis=2, keepdims=True) + eps)
    gw = g * w
    dot = np.mean(gw * x, axis=2, keepdims=True)
    dx = r * (gw - x * r * r * dot)
    dsize = r * (size * np.abs(w) + np.abs(x) * r * r * np.mean(size * np.abs(w * x), axis=2, keepdims=True))
    return dx, np.sum(g * x * r, axis=(0, 1)), dsize, np.sum(size * np.abs(x) * r, axis=(0, 1))


def newton_schulz(g, coefficients, eps, scale=1.0, rounded=False):
    """``coefficients``: rows of (a, b, c).  ``rounded``: X, S and the polynomial
    kept as fp16 times 2^13, 2^12 and 2^11, the polynomial's diagonal apart and
    unrounded, as the GPU keeps them."""
    def keep(v, power):
        if not rounded:
            return v
        return (v * 2.0 ** power).astype(np.float16).astype(np.float64) * 2.0 ** -power

    x = np.asarray(g, dtype=np.float64)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    x = keep(x / (np.sqrt(np.sum(x * x)) + eps), 13)
    for i, (a, b, c) in enumerate(coefficients):
        s = keep(x @ x.T, 12)
        p = b * s + c * (s @ s)
        d = np.diag(np.diag(p))
        p = keep(p - d, 11) + d
        x = a * x + p @ x
        if i + 1 < len(coefficients):
            x = keep(x, 13)
    return scale * (x.T if tall else x)
