"""Scales of the Newton-Schulz update whose factors leave fp32's normal numbers are refused
(no GPU)."""

import pytest

import implicit_gemm_conv_dp_amd as skg

from test_lowp_host import P, refused


@pytest.mark.parametrize("scale", [1e-36, -1e-40, 2.0 ** -100 * 0.99, float("inf"), float("nan")])
def test_scales(scale):
    kw = dict(g=P, out=P, rows=48, cols=70, dtype="f32", scale=scale)
    refused(lambda: skg.skg_run_newton_schulz(skg.newton_schulz_args(**kw), 0x10000, 1 << 24, 0), "scale")
    refused(lambda: skg.skg_newton_schulz_workspace_bytes(skg.newton_schulz_args(**kw)), "scale")


@pytest.mark.parametrize("scale", [0.0, 2.0 ** -100, -2.0 ** -100, 1e30])
def test_scales_that_are_taken(scale):
    assert skg.skg_newton_schulz_workspace_bytes(skg.newton_schulz_args(rows=48, cols=70, dtype="f32", scale=scale))
