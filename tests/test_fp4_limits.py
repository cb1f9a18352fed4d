"""The largest 4-bit products (no GPU): sizes whose last tile would pass 32
bits are refused."""

import pytest

from test_lowp_host import plan, refused

MOST = (1 << 31) - 256   # the last tile of 256 ends within 31 bits


@pytest.mark.parametrize("tile", ["256x256x256", "128x128x256", "64x64x512", "auto"])
def test_last_tile_stays_within_32_bits(tile):
    kw = dict(K=128, tile=tile, mode="dp")
    refused(plan(M=MOST + 1, N=8, ldc=8, **kw), "too large")
    refused(plan(M=8, N=MOST + 1, ldc=MOST + 256, **kw), "too large")
    if tile != "64x64x512":   # (too many workgroups for one launch)
        plan(M=MOST, N=8, ldc=8, **kw)()
        plan(M=8, N=MOST, ldc=MOST, **kw)()
