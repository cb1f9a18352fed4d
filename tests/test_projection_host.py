"""Refusals and plans of the operators of an 8-bit attention projection (no
GPU): every argument check returns -2 with its reason before anything touches
a device, and empty calls succeed without one."""

import ctypes
import struct

import pytest
import torch

import implicit_gemm_conv_dp_amd as skg

from test_lowp_host import P, Ptr, refused


# --- block quantisation --------------------------------------------------------
def quant(**kw):
    base = dict(x=P, q=P, scales=P, qt=P, scales_t=P, rows=4, cols=64, dtype="bf16", dtype_q="e4m3")
    base.update(kw)
    return lambda: skg.skg_run_block_quant(skg.block_quant_args(**base), 0)


@pytest.mark.parametrize("kw,word", [
    (dict(dtype="e4m3"), "f16, bf16 or f32"),
    (dict(dtype_q="e2m1"), "e4m3 or e5m2"),
    (dict(block=7), "block"),
    (dict(rows=-1), "negative"),
    (dict(cols=-1), "negative"),
    (dict(rows=1 << 31), "large"),
    (dict(cols=1 << 31), "large"),
    (dict(kq=1 << 31), "large"),
    (dict(kq=64), "128"),
    (dict(kq=200), "128"),
    (dict(kqt=0), "128"),
    (dict(kqt=130), "128"),
    (dict(cols=300, kq=256), "128"),
    (dict(ldx=63), "leading"),
    (dict(ldq=127), "leading"),
    (dict(ldqt=127), "leading"),
    (dict(q=None, qt=None), "neither"),
    (dict(scales=None), "scales"),
    (dict(scales_t=None), "scales"),
    (dict(x=None), "null"),
    (dict(x=Ptr(0x10001)), "aligned"),
    (dict(scales=Ptr(0x10002)), "aligned"),
    (dict(scales_t=Ptr(0x10002)), "aligned"),
])
def test_quant_refusals(kw, word):
    refused(quant(**kw), word)


def test_empty_quant():
    quant(rows=0, qt=None, scales_t=None, x=None)()
    quant(cols=0, q=None, scales=None, x=None)()
    quant(rows=0, cols=0, x=None)()


def test_unknown_names():
    for kw in (dict(block="64x64"), dict(dtype_q="int8"), dict(dtype="f64")):
        with pytest.raises(ValueError):
            quant(**kw)()


# --- the product ---------------------------------------------------------------
def product(run=False, **kw):
    base = dict(M=256, N=256, K=512, dtype_ab="e4m3", dtype_c="bf16", tile="auto", mode="auto",
                reduction="auto", ctas=8, scale_mode="block128")
    base.update(kw)
    if not run:
        return lambda: skg.plan_gemm(**base)
    ptrs = {n: base.pop(n, P) for n in ("A", "B", "C", "scale_a", "scale_b")}
    return lambda: skg.skg_run_gemm(skg.gemm_args(**ptrs, **base), 0, 0, 0)


@pytest.mark.parametrize("scale_mode", ["block128", "row128"])
@pytest.mark.parametrize("kw,word", [
    (dict(dtype_ab="bf16"), "fp8"),
    (dict(dtype_ab="e2m1"), "fp8"),
    (dict(dtype_ab="f32"), "dtype"),
    (dict(dtype_c="e4m3"), "C dtype"),
    (dict(K=576), "multiple of 128"),
    (dict(K=0), "positive"),
    (dict(M=0), "positive"),
    (dict(N=-1), "positive"),
    (dict(mode="dp_sk"), "dp or auto"),
    (dict(mode="persistent"), "dp or auto"),
    (dict(mode="splitk"), "dp or auto"),
    (dict(tile="128x128x64"), "no GEMM instance"),
    (dict(tile="256x256x256"), "no GEMM instance"),
    (dict(lda=400), "leading"),
    (dict(ldb=520), "16 bytes"),
    (dict(ldc=264, N=260, dtype_c="bf16", lda=500), "leading"),
    (dict(N=258), "ldc"),
    (dict(M=1 << 31), "large"),
    (dict(N=1 << 31, ldc=1 << 31), "large"),
    (dict(M=1 << 30, K=1 << 10), "scale array"),
    (dict(lda=1 << 30), "pitch"),
    (dict(ctas=0), "ctas"),
])
def test_product_refusals(scale_mode, kw, word):
    refused(product(scale_mode=scale_mode, **kw), word)


@pytest.mark.parametrize("kw,word", [
    (dict(scale_a=None), "both scale"),
    (dict(scale_b=None), "both scale"),
    (dict(A=None), "null"),
    (dict(C=Ptr(0x10008)), "aligned"),
    (dict(scale_b=Ptr(0x10004)), "aligned"),
])
def test_product_pointer_refusals(kw, word):
    refused(product(True, **kw), word)


@pytest.mark.parametrize("tile", ["16x16x128", "16x32x128", "32x32x128", "32x64x128", "64x64x128", "256x128x128"])
def test_tiles_of_this_mode_alone(tile):
    refused(product(tile=tile, scale_mode="rowcol", mode="dp"), "scale for each 128")
    refused(product(tile=tile, scale_mode="mx", mode="dp"), "")
    p = product(tile=tile)()
    assert p["mode"] == skg.MODES["dp"] and p["workspace_bytes"] == 0 and p["sk_ctas"] == 0


@pytest.mark.parametrize("tile", ["256x256x128", "128x128x128"])
def test_shared_tiles(tile):
    p = product(tile=tile, mode="auto")()
    assert p["mode"] == skg.MODES["dp"] and p["n_waves"] == 8 and p["requested_mode"] == skg.MODES["auto"]
    # the engine's own kernels on these tiles are as they were
    q = product(tile=tile, scale_mode="rowcol", mode="dp_sk", reduction="tree", ctas=3)()
    assert q["n_waves"] == 4 and q["sk_ctas"] == 3


def test_auto_takes_a_tile_for_any_sizes():
    for M in (1, 17, 100, 1000, 5000, 70000):
        for N in (8, 4864, 100000):
            for K in (128, 4096):
                p = product(M=M, N=N, K=K)()
                assert p["tk"] == 128 and p["workspace_bytes"] == 0


# --- heads -----------------------------------------------------------------------
def heads(**kw):
    base = dict(q=P, k=P, yq=P, yk=P, seq=4, heads_q=4, heads_k=2, head_dim=64, dtype="bf16", cos=P,
                sin=P, table_rows=16)
    base.update(kw)
    return lambda: skg.skg_run_qknorm_rope(skg.qknorm_rope_args(**base), 0)


def heads_bwd(ws=(0x10000, 1 << 22), **kw):
    base = dict(q=P, k=P, yq=P, yk=P, dyq=P, dyk=P, dwq=P, dwk=P, seq=4, heads_q=4, heads_k=2,
                head_dim=64, dtype="bf16", cos=P, sin=P, table_rows=16)
    base.update(kw)
    return lambda: skg.skg_run_qknorm_rope_bwd(skg.qknorm_rope_args(**base), ws[0], ws[1], 0)


class Positions(Ptr):
    def __init__(self, size, p=0x10000):
        super().__init__(p)
        self.size = size

    def element_size(self):
        return self.size


@pytest.mark.parametrize("call", [heads, heads_bwd])
@pytest.mark.parametrize("kw,word", [
    (dict(dtype="e4m3"), "f16, bf16 or f32"),
    (dict(dtype_w="f16"), "weight"),
    (dict(batch=-1), "negative"),
    (dict(seq=-1), "negative"),
    (dict(heads_q=-1), "negative"),
    (dict(head_dim=0), "head_dim"),
    (dict(head_dim=513), "head_dim"),
    (dict(rope_dim=63), "rope_dim"),
    (dict(rope_dim=66), "rope_dim"),
    (dict(rope_dim=-2), "rope_dim"),
    (dict(style=2), "style"),
    (dict(eps=-1.0), "eps"),
    (dict(eps=float("nan")), "eps"),
    (dict(positions=Positions(2)), "32 or 64"),
    (dict(table_rows=0), "table_rows"),
    (dict(table_rows=1 << 31), "table_rows"),
    (dict(seq=1 << 31), "32-bit"),
    (dict(seq=1 << 20, batch=1 << 20), "32-bit"),
    (dict(seq=1 << 30, heads_q=4), "32-bit"),
    (dict(q=None), "null"),
    (dict(k=None), "null"),
    (dict(cos=None), "tables"),
    (dict(sin=None), "tables"),
    (dict(q=Ptr(0x10001)), "aligned"),
    (dict(k=Ptr(0x10001)), "aligned"),
    (dict(yk=Ptr(0x10001)), "aligned"),
    (dict(cos=Ptr(0x10002)), "aligned"),
    (dict(weight_q=Ptr(0x10002), dtype_w="f32"), "aligned"),
    (dict(positions=Positions(8, 0x10004)), "aligned"),
])
def test_heads_refusals(call, kw, word):
    refused(call(**kw), word)


@pytest.mark.parametrize("kw,word", [(dict(yq=None), "null"), (dict(yk=None), "null")])
def test_heads_forward_refusals(kw, word):
    refused(heads(**kw), word)


@pytest.mark.parametrize("kw,word", [
    (dict(dyq=None), "null"),
    (dict(dyk=None), "null"),
    (dict(dyq=Ptr(0x10001)), "aligned"),
    (dict(dwk=Ptr(0x10002)), "aligned"),
    (dict(ws=(0x10000, 16)), "workspace"),
    (dict(ws=(0, 1 << 22)), "workspace"),
    (dict(ws=(0x10004, 1 << 22)), "workspace"),
])
def test_heads_backward_refusals(kw, word):
    refused(heads_bwd(**kw), word)


def test_empty_heads():
    heads(seq=0, q=None, k=None, yq=None, yk=None, cos=None, sin=None)()
    heads(batch=0, q=None)()
    heads(heads_q=0, heads_k=0, q=None, k=None)()
    heads_bwd(seq=0, dwq=None, dwk=None, q=None, dyq=None)()
    heads_bwd(yq=None, yk=None, dwq=None, dwk=None)()   # nothing is asked for


def test_heads_workspace_goes_by_what_is_asked():
    def need(**kw):
        base = dict(seq=1000, heads_q=8, heads_k=2, head_dim=128, dtype="bf16")
        base.update(kw)
        return skg.skg_qknorm_rope_bwd_workspace_bytes(skg.qknorm_rope_args(**base))
    assert need() == 0
    assert need(dwq=P) > 0 and need(dwk=P) > 0 and need(dwq=P, dwk=P) == need(dwq=P) + need(dwk=P)
    assert need(dwq=P, seq=0) == 0
    assert need(dwq=P, dwk=P, seq=1 << 20) <= 1026 * 128 * 4


# --- the update ------------------------------------------------------------------
def update(ws=(0x10000, 1 << 40), **kw):
    base = dict(g=P, out=P, rows=64, cols=96, dtype="f32", dtype_out="bf16")
    base.update(kw)
    return lambda: skg.skg_run_newton_schulz(skg.newton_schulz_args(**base), ws[0], ws[1], 0)


@pytest.mark.parametrize("kw,word", [
    (dict(dtype="e4m3"), "f16, bf16 or f32"),
    (dict(dtype_out="e4m3"), "f16, bf16 or f32"),
    (dict(rows=-1), "negative"),
    (dict(cols=-1, ldg=0, ldo=0), "negative"),
    (dict(rows=1 << 23), "large"),
    (dict(cols=1 << 23), "large"),
    (dict(steps=0), "steps"),
    (dict(steps=65), "steps"),
    (dict(ldg=95), "leading"),
    (dict(ldo=95), "leading"),
    (dict(tile=7), "tile"),
    (dict(rows=1 << 20, cols=(1 << 13) + 1, ldg=1 << 14, ldo=1 << 14), "2^33"),
    (dict(tile=-2), "tile"),
    (dict(eps=-1.0), "eps"),
    (dict(eps=float("nan")), "eps"),
    (dict(scale=float("inf")), "scale"),
    (dict(coefficients=(float("nan"), 1.0, 1.0)), "coefficients"),
    (dict(g=None), "null"),
    (dict(out=None), "null"),
    (dict(g=Ptr(0x10002)), "aligned"),
    (dict(out=Ptr(0x10001)), "aligned"),
    (dict(ws=(0x10000, 64)), "workspace"),
    (dict(ws=(0, 1 << 40)), "workspace"),
    (dict(ws=(0x10080, 1 << 40)), "workspace"),
])
def test_update_refusals(kw, word):
    refused(update(**kw), word)


@pytest.mark.parametrize("coefficients", [(1.0, 2.0), (), [(1.0, 2.0, 3.0)] * 4, [(1.0, 2.0)] * 5])
def test_update_coefficients(coefficients):
    with pytest.raises((ValueError, IndexError)):
        skg.newton_schulz_args(P, P, rows=4, cols=4, dtype="f32", coefficients=coefficients)


def test_empty_update():
    update(rows=0, g=None, out=None, ws=(0, 0))()
    update(cols=0, g=None, out=None, ws=(0, 0))()
    assert skg.skg_newton_schulz_workspace_bytes(skg.newton_schulz_args(rows=0, cols=8, dtype="f32")) == 0
    assert skg.skg_newton_schulz_workspace_bytes(skg.newton_schulz_args(rows=8, cols=8, dtype="f32")) > 0


def test_heads_arguments_fill_their_structure():
    assert skg._HEADS.size == ctypes.sizeof(skg._lib.skg_heads_args_t)
    t = [torch.empty(4) for _ in range(14)]
    st = [(10 * i + 1, 10 * i + 2, 10 * i + 3) for i in range(6)]
    pos = torch.zeros(2, dtype=torch.int64)
    a = skg.qknorm_rope_args(*t[:6], batch=2, seq=3, heads_q=4, heads_k=5, head_dim=6, rope_dim=2, dtype="bf16",
                             weight_q=t[6], weight_k=t[7], dtype_w="f32", cos=t[8], sin=t[9], table_rows=11,
                             positions=pos, pos0=12, style="pairs", eps=0.25, q_strides=st[0], k_strides=st[1],
                             yq_strides=st[2], yk_strides=st[3], dyq_strides=st[4], dyk_strides=st[5], dwq=t[10],
                             dwk=t[11])
    got = {n: getattr(a, n) for n, _ in a._fields_}
    for n, v in dict(batch=2, seq=3, heads_q=4, heads_k=5, head_dim=6, rope_dim=2, dtype=skg.DTYPES["bf16"],
                     dtype_w=skg.DTYPES["f32"], style=skg.ROPE_STYLES["pairs"], pos_bits=64, table_rows=11, pos0=12,
                     eps=0.25, positions=pos.data_ptr()).items():
        assert got[n] == v, n
    for n, v in zip(("q", "k", "yq", "yk", "dyq", "dyk", "weight_q", "weight_k", "cos", "sin", "dwq", "dwk"), t):
        assert got[n] == v.data_ptr(), n
    for n, v in zip(("q", "k", "yq", "yk", "dyq", "dyk"), st):
        s = got[n + "_strides"]
        assert (s.batch, s.token, s.head) == v, n
    for bad in (dict(seq=2.5), dict(heads_q="4"), dict(q_strides=(1, 2)),
                dict(q_strides=(1, 2), k_strides=(1, 2, 3, 4)), dict(yq_strides=())):
        kw = dict(seq=3, heads_q=4, heads_k=5, head_dim=6, dtype="f32")
        with pytest.raises((TypeError, ValueError, struct.error)):
            skg.qknorm_rope_args(t[0], t[1], t[2], t[3], **dict(kw, **bad))
