"""Plans whose launch would have 2^32 threads or more along its axis, which the
runtime does not take, are refused (no GPU)."""

import pytest

import implicit_gemm_conv_dp_amd as skg

from test_lowp_host import plan, refused

MOST = (1 << 24) - 1   # workgroups of 256 threads


@pytest.mark.parametrize("kw", [
    dict(tile="16x16x512", N=8),
    dict(tile="32x64x512", N=8),
    dict(tile="128x128x32", N=8, dtype_ab="bf16", scale_mode="rowcol", K=32),
])
def test_too_many_workgroups(kw):
    kw = dict(dict(ldc=8, K=128, mode="dp"), **kw)
    tm = int(kw["tile"].split("x")[0])
    assert plan(M=MOST * tm, **kw)()["grid"] == MOST
    refused(plan(M=MOST * tm + 1, **kw), "workgroups")


def test_a_ring_tile_walks_any_grid():
    assert plan(M=(1 << 31) - 256, N=129, ldc=136, K=128, tile="128x128x256")()["grid"] > MOST


def test_auto_takes_a_tile_that_can_be_launched():
    p = plan(M=(1 << 31) - 256, N=8, K=128, ldc=8, tile="auto", mode="auto")()
    assert p["tiles"] <= MOST or p["tk"] == 256
