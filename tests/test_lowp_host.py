"""Refusals and plans of the low-precision layer operators (no GPU): every
argument check returns -2 with its reason before anything touches a device,
and empty calls succeed without one."""

import pytest

import implicit_gemm_conv_dp_amd as skg


class Ptr:
    """Stands for a device tensor at an address; never dereferenced."""

    def __init__(self, p=0x10000):
        self.p = p

    def data_ptr(self):
        return self.p


P = Ptr()


def refused(call, word):
    with pytest.raises(skg.SkgError) as ei:
        call()
    assert ei.value.status == -2 and word in ei.value.msg, ei.value.msg


def norm(**kw):
    base = dict(x=P, y=P, rows=4, cols=64, dtype="bf16")
    base.update(kw)
    return lambda: skg.skg_run_rmsnorm(skg.rmsnorm_args(**base), 0)


@pytest.mark.parametrize("kw,word", [
    (dict(dtype="e4m3"), "f16, bf16 or f32"),
    (dict(dtype_w="f16"), "weight"),
    (dict(dtype_y="f16"), "output"),
    (dict(dtype_y="e5m2"), "output"),
    (dict(dtype_y="e4m3", scale_mode="tensor", y_scale=P), "scales"),
    (dict(dtype_y="e2m1", y_scale=P), "MX"),
    (dict(dtype_y="e2m1", scale_mode="mx", cols=48, y_scale=P), "multiple of 32"),
    (dict(dtype_y="e2m1", scale_mode="mx", ldy=65, y_scale=P), "even"),
    (dict(dtype_y="e4m3"), "scales"),
    (dict(rows=-1), "rows"),
    (dict(rows=1 << 31), "rows"),
    (dict(cols=0), "cols"),
    (dict(cols=32769), "SKG_NORM_MAX_COLS"),
    (dict(ldx=63), "leading"),
    (dict(ldy=63), "leading"),
    (dict(residual=P, ldr=63), "leading"),
    (dict(h=P, ldh=63), "leading"),
    (dict(eps=-1.0), "eps"),
    (dict(eps=float("nan")), "eps"),
    (dict(x=None), "null"),
    (dict(y=None), "null"),
    (dict(x=Ptr(0x10001)), "aligned"),
    (dict(rstd=Ptr(0x10002)), "aligned"),
    (dict(weight=Ptr(0x10002), dtype_w="f32"), "aligned"),
])
def test_norm_refusals(kw, word):
    refused(norm(**kw), word)


def bwd(ws=(0x10000, 1 << 20), **kw):
    base = dict(dy=P, h=P, rstd=P, dx=P, rows=4, cols=64, dtype="bf16", dw=P)
    base.update(kw)
    return lambda: skg.skg_run_rmsnorm_bwd(skg.rmsnorm_bwd_args(**base), ws[0], ws[1], 0)


@pytest.mark.parametrize("kw,word", [
    (dict(dtype="e4m3"), "f16, bf16 or f32"),
    (dict(dtype_w="f16"), "weight"),
    (dict(rows=-1), "rows"),
    (dict(cols=0), "cols"),
    (dict(cols=40000), "SKG_NORM_MAX_COLS"),
    (dict(lddy=63), "leading"),
    (dict(ldh=63), "leading"),
    (dict(lddx=63), "leading"),
    (dict(dres=P, lddres=63), "leading"),
    (dict(dy=None), "null"),
    (dict(h=None), "null"),
    (dict(rstd=None), "null"),
    (dict(dx=None, dw=None), "neither"),
    (dict(dy=Ptr(0x10001)), "aligned"),
    (dict(dw=Ptr(0x10002)), "aligned"),
    (dict(ws=(0x10000, 16)), "workspace"),
    (dict(ws=(0, 1 << 20)), "workspace"),
    (dict(ws=(0x10001, 1 << 20)), "workspace"),
])
def test_norm_bwd_refusals(kw, word):
    refused(bwd(**kw), word)


def mx(quant=True, **kw):
    base = dict(x=P, q=P, scales=P, rows=4, cols=64, dtype="bf16", dtype_q="e2m1")
    base.update(kw)
    run = skg.skg_run_mx_quant if quant else skg.skg_run_mx_dequant
    return lambda: run(skg.mx_args(**base), 0)


@pytest.mark.parametrize("quant", [True, False])
@pytest.mark.parametrize("kw,word", [
    (dict(dtype="e4m3"), "f16, bf16 or f32"),
    (dict(dtype_q="e5m2"), "e4m3 or e2m1"),
    (dict(rows=-1), "negative"),
    (dict(cols=-32), "negative"),
    (dict(kq=32), "kq"),
    (dict(kq=80), "kq"),
    (dict(ldx=63), "leading"),
    (dict(ldq=32), "leading"),
    (dict(ldq=65), "even"),
    (dict(rows=1 << 31), "large"),
    (dict(x=None), "null"),
    (dict(q=None), "null"),
    (dict(scales=None), "null"),
    (dict(x=Ptr(0x10001)), "aligned"),
])
def test_mx_refusals(quant, kw, word):
    refused(mx(quant, **kw), word)


def test_mx_dequant_does_not_transpose():
    refused(mx(False, transpose=True, kq=32), "transpose")


def test_empty_calls_need_no_device():
    norm(rows=0)()
    mx(rows=0)()
    mx(cols=0, kq=0)()
    mx(False, rows=0)()
    assert skg.skg_rmsnorm_bwd_workspace_bytes(
        skg.rmsnorm_bwd_args(P, P, P, P, rows=0, cols=64, dtype="f32", dw=P)) == 0


def plan(**kw):
    base = dict(M=256, N=256, K=512, dtype_ab="e2m1", dtype_c="bf16", tile="256x256x256",
                mode="dp", reduction="linear", ctas=8, scale_mode="mx")
    base.update(kw)
    return lambda: skg.plan_gemm(**base)


@pytest.mark.parametrize("kw,word", [
    (dict(scale_mode="rowcol"), "MX"),
    (dict(scale_mode="tensor"), "MX"),
    (dict(tile="256x256x128"), "fp4"),
    (dict(tile="256x256x64"), "fp4"),
    (dict(K=576), "multiple of 128"),
    (dict(lda=500), "leading"),
    (dict(lda=528), "16 bytes"),
    (dict(ldc=257), "16 bytes"),
    (dict(M=0), "positive"),
    (dict(dtype_c="e2m1"), "C dtype"),
    (dict(reduction="atomic"), "fp32"),
])
def test_fp4_gemm_refusals(kw, word):
    refused(plan(**kw), word)


def test_fp4_tiles_refuse_other_inputs():
    for dt in ("bf16", "e4m3"):
        refused(plan(dtype_ab=dt, scale_mode="rowcol"), "instance")
        refused(plan(dtype_ab=dt, scale_mode="rowcol", tile="auto"), "unknown tile")


def test_fp4_plan():
    p = plan(M=300, N=520, K=640)()
    assert (p["tm"], p["tn"], p["tk"], p["tiles_m"], p["tiles_n"], p["iters_per_tile"]) == \
        (256, 256, 256, 2, 3, 3)


@pytest.mark.parametrize("kw,word", [
    (dict(tile="16x16x512", mode="dp_sk", reduction="tree"), "mode dp or auto"),
    (dict(tile="64x64x512", mode="splitk", reduction="linear"), "mode dp or auto"),
    (dict(tile="32x32x512", mode="persistent"), "mode dp or auto"),
    (dict(tile="16x16x512", scale_mode="rowcol"), "MX"),
])
def test_direct_tile_refusals(kw, word):
    refused(plan(**kw), word)


def test_direct_plan():
    p = plan(M=20, N=70, K=1152, ldc=72, tile="16x32x512", mode="auto")()
    assert (p["tm"], p["tn"], p["tk"], p["tiles_m"], p["tiles_n"], p["iters_per_tile"]) == (16, 32, 512, 2, 3, 3)
    assert p["workspace_bytes"] == 0 and p["sk_ctas"] == 0 and p["grid"] == 6
    assert p["mode"] == skg.MODES["dp"] and p["requested_mode"] == skg.MODES["auto"]


def test_auto_tile():
    """Small tiles for few rows, large ones for many, never a workspace; a
    stream-K mode takes a tile that has it."""
    for (M, N, K), most in (((1, 4096, 4096), 16), ((48, 4863, 4096), 48), ((200, 300, 512), 32)):
        p = plan(M=M, N=N, K=K, ldc=-(-N // 8) * 8, tile="auto", mode="auto")()
        assert p["tm"] <= most and p["tn"] <= 64 and p["workspace_bytes"] == 0
    p = plan(M=8192, N=8192, K=8192, tile="auto", mode="auto")()
    assert (p["tm"], p["tn"]) == (256, 256) and p["mode"] == skg.MODES["dp"]
    p = plan(M=48, N=4864, K=4096, tile="auto", mode="dp_sk", reduction="tree", ctas=64)()
    assert p["tm"] >= 128 and p["sk_ctas"] == 64


def test_plan_and_run_in_one_refuses_as_the_two_do():
    a = skg.gemm_args(None, P, P, M=8, N=8, K=128, dtype_ab="e2m1", dtype_c="bf16", scale_a=P, scale_b=P,
                      scale_mode="mx", tile="auto", mode="auto", reduction="auto", ctas=1)
    refused(lambda: skg.skg_plan_run_gemm(a, 0, 0, 0), "null A, B or C")
    a.A, a.K = P.data_ptr(), 100
    refused(lambda: skg.skg_plan_run_gemm(a, 0, 0, 0), "multiple of 128")
