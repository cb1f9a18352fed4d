"""Pins of the oracle of an 8-bit attention projection (no GPU)."""

import numpy as np
import pytest
import torch

from oracle import codecs, projection as pj


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("block", ["1x128", "128x128"])
def test_blocks_by_loops(fmt, block):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((131, 200)).astype(np.float32).astype(np.float64)
    s, q = pj.block_quantize(x, fmt, block)
    h = 128 if block == "128x128" else 1
    assert s.shape == (2, -(-131 // h)) and q.shape == (131, 256)
    for r in (0, 5, 127, 128, 130):
        for k in (0, 1):
            part = x[r // h * h:r // h * h + h, 128 * k:128 * k + 128]
            top = np.abs(part).max()
            assert s[k, r // h] == np.float32(top / pj.LARGEST[fmt])
            want = torch.tensor(x[r, 128 * k:128 * k + 128] * pj.LARGEST[fmt] / top).to(
                torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2).double().numpy()
            got = codecs.decode(fmt, q[r, 128 * k:128 * k + 128][:want.size])
            assert np.array_equal(got, want)
    assert not q[:, 200:].any()
    v = pj.block_values(s, q, fmt, block)[:, :200]
    step = 2.0 ** (-4 if fmt == "e4m3" else -3)
    assert np.all(np.abs(v - x) <= step * 1.01 * np.abs(x) + 0.01 * np.abs(x).max())


def test_empty_blocks_take_the_smallest_scale():
    s, q = pj.block_quantize(np.zeros((2, 128)), "e4m3")
    assert np.all(s == np.float32(2.0 ** -126)) and not q.any()


@pytest.mark.parametrize("style", ["half", "pairs"])
@pytest.mark.parametrize("dim,half", [(8, 4), (10, 3), (6, 0)])
def test_heads_against_autograd(style, dim, half):
    rng = np.random.default_rng(2)
    x, dy = rng.standard_normal((2, 5, 3, dim))
    w = rng.standard_normal(dim)
    ang = rng.standard_normal((5, half))
    cos, sin = np.cos(ang), np.sin(ang)
    tx, tw = (torch.tensor(v, requires_grad=True) for v in (x, w))
    n = tx * torch.rsqrt(tx.square().mean(2, keepdim=True) + 0.1) * tw
    z = torch.polar(torch.ones(5, 1, half, dtype=torch.float64), torch.tensor(ang)[:, None])
    if style == "half":
        t = torch.complex(n[..., :half], n[..., half:2 * half]) * z
        y = torch.cat((t.real, t.imag, n[..., 2 * half:]), 2)
    else:
        t = torch.view_as_complex(n[..., :2 * half].reshape(5, 3, half, 2).contiguous()) * z
        y = torch.cat((torch.view_as_real(t).flatten(2), n[..., 2 * half:]), 2)
    y.backward(torch.tensor(dy))
    got = pj.rotate(pj.head_norm(x, w, 0.1)[0], cos, sin, style)
    np.testing.assert_allclose(got, y.detach().numpy(), rtol=1e-12, atol=1e-12)
    dx, dw, _, _ = pj.head_norm_bwd(dy, x, w, 0.1, cos, sin, style)
    np.testing.assert_allclose(dx, tx.grad.numpy(), rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(dw, tw.grad.numpy(), rtol=1e-10, atol=1e-12)


def test_newton_schulz_acts_on_singular_values():
    rng = np.random.default_rng(3)
    for shape in ((7, 12), (12, 7), (5, 5)):
        g = rng.standard_normal(shape)
        u, s, vt = np.linalg.svd(g, full_matrices=False)
        t = s / (np.sqrt(np.sum(s * s)) + 1e-7)
        cs = [(3.4445, -4.7750, 2.0315), (2.0, -1.5, 0.5)]
        for a, b, c in cs:
            t = a * t + b * t ** 3 + c * t ** 5
        np.testing.assert_allclose(pj.newton_schulz(g, cs, 1e-7, 0.5), 0.5 * (u * t) @ vt, rtol=1e-9, atol=1e-12)


def test_rounded_newton_schulz_is_near():
    rng = np.random.default_rng(4)
    g = rng.standard_normal((40, 90))
    cs = [(3.4445, -4.7750, 2.0315)] * 5
    e, r = pj.newton_schulz(g, cs, 1e-7), pj.newton_schulz(g, cs, 1e-7, rounded=True)
    d = np.linalg.norm(e - r) / np.linalg.norm(e)
    assert 0 < d < 2.0 ** -8
