"""The workspace of the norm's gradient (no GPU): what a caller asks before it
knows where dx goes is a matter of the sizes alone and enough for every dx."""

import pytest

import implicit_gemm_conv_dp_amd as skg

from test_lowp_host import P, Ptr

DY, H, APART = Ptr(0x100000000), Ptr(0x200000000), Ptr(0x300000000)
SIZES = [(1, 1), (1, 16384), (509, 1111), (1024, 1024), (1024, 1025), (1025, 64), (65, 16384), (4096, 4096)]


def args(rows, cols, dtype, dx, dy=DY, h=H, dw=P):
    return skg.rmsnorm_bwd_args(dy, h, P, dx, rows=rows, cols=cols, dtype=dtype, dw=dw)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_size_does_not_depend_on_the_pointers(rows, cols, dtype):
    n = skg.skg_rmsnorm_bwd_workspace_bytes(args(rows, cols, dtype, APART))
    for dx in (None, DY, H, Ptr(DY.p + 64)):
        assert skg.skg_rmsnorm_bwd_workspace_bytes(args(rows, cols, dtype, dx)) == n
    assert skg.skg_rmsnorm_bwd_workspace_bytes(args(rows, cols, dtype, None, None, None)) == n
    assert skg.skg_rmsnorm_bwd_workspace_bytes(args(rows, cols, dtype, DY, dw=None)) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_size_is_enough_for_a_dx_over_dy_or_h(rows, cols, dtype):
    n = skg.skg_rmsnorm_bwd_workspace_bytes(args(rows, cols, dtype, APART))
    for dx in (DY, H):
        a = args(rows, cols, dtype, dx)
        need, launched = skg.skg_plan_run_rmsnorm_bwd(a, 0, 0, 0)
        assert 0 < need <= n and not launched
        for short in (0, need - 1):
            with pytest.raises(skg.SkgError) as ei:
                skg.skg_run_rmsnorm_bwd(a, 0x10000, short, 0)
            assert ei.value.status == -2 and "workspace" in ei.value.msg


def test_plan_and_run_in_one_refuses_as_the_run_does():
    a = args(4, 64, "bf16", DY)
    a.dy = 0
    with pytest.raises(skg.SkgError) as ei:
        skg.skg_plan_run_rmsnorm_bwd(a, 0, 0, 0)
    assert ei.value.status == -2 and "null" in ei.value.msg
