"""The 4-bit product's choice of a tile (no GPU) passes over tiles whose rows
lie too far apart for them: a tile's rows have to lie within the 2 GiB that one
offset spans."""

import pytest

import implicit_gemm_conv_dp_amd as skg

from test_lowp_host import plan, refused


# Rows 16 MiB apart, and a reduction as long.
@pytest.mark.parametrize("kw", [dict(lda=1 << 25), dict(ldb=1 << 25), dict(K=1 << 25)])
def test_auto_takes_a_tile_that_spans_its_rows(kw):
    kw = dict(dict(M=4096, N=4096, K=8192), **kw)
    refused(plan(tile="256x256x256", mode="auto", **kw), "row pitch")
    p = plan(tile="auto", mode="auto", **kw)()
    span = max(p["tm"] * max(kw.get("lda", 0), kw["K"]), p["tn"] * max(kw.get("ldb", 0), kw["K"])) // 2
    assert span <= (1 << 31) - 1


def test_rows_that_no_tile_spans():
    assert min(min(skg.skg_tile_info(t).tm, skg.skg_tile_info(t).tn) for t in range(9, 19)) == 16
    refused(plan(M=64, N=64, K=1 << 29, ldc=64, tile="auto", mode="auto"), "row pitch")
