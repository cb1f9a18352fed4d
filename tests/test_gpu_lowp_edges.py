"""Widths and row counts at which the norm, its gradient and MX quantisation
change how they spread rows over threads: rows narrower than a chunk, rows
that share a wave (ordinary ones beside empty ones and NaN), every change of
the group size with ragged ends, and lines of no elements."""

import numpy as np
import pytest
import torch

import implicit_gemm_conv_dp_amd as skg
from oracle import codecs, lowp
from test_gpu_norm import BWD_SHAPES, DELTA, EPS, HALF, SHAPES, T, check_codes, check_values, f64, out, rows_of

pytestmark = pytest.mark.gpu

WIDTHS = [2, 5, 8, 9, 63, 64, 65, 120, 127, 128, 129, 255, 256, 257, 511, 1023, 1024, 1025, 2047, 2049, 4095, 4097,
          8191, 8193, 16383, 16385]
assert not {c for _, c in SHAPES + BWD_SHAPES} & set(WIDTHS) - {64}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", WIDTHS)
def test_norm_widths(cols, dtype):
    rows = 70 if cols <= 512 else 5
    x, r = rows_of(1, rows, cols, dtype, cols + 1), rows_of(2, rows, cols, dtype)
    w = rows_of(3, 1, cols, dtype).reshape(-1)
    h, y, rstd = out((rows, cols), T[dtype]), out((rows, cols + 3), T[dtype]), out((rows,), torch.float32)
    kw = dict(rows=rows, cols=cols, dtype=dtype, weight=w, residual=r, eps=EPS, ldx=cols + 1)
    skg.rmsnorm(x, y, h=h, rstd=rstd, ldy=cols + 3, **kw)
    q, sc = out((rows, cols), torch.uint8), out((rows,), torch.float32)
    skg.rmsnorm(x, q, y_scale=sc, dtype_y="e4m3", **kw)
    torch.cuda.synchronize()
    want = (x[:, :cols].cpu().float() + r.cpu().float()).to(T[dtype])
    assert torch.equal(h.cpu(), want)
    ref, rr = lowp.rmsnorm(f64(want), f64(w), EPS)
    check_values(f64(y[:, :cols]), ref, dtype, "%d %s" % (cols, dtype))
    assert np.all(np.abs(f64(rstd) - rr) <= DELTA * rr)
    assert torch.isnan(y[:, cols:].float()).all()
    s = f64(sc)
    assert np.all(np.abs(s - np.maximum(np.abs(ref).max(1) / 448, 2.0 ** -126)) <= DELTA * s)
    check_codes("e4m3", codecs.decode("e4m3", q.cpu().numpy()), s[:, None], ref, "%d %s" % (cols, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", WIDTHS)
def test_gradient_widths(cols, dtype):
    rows = 2600 if cols <= 512 else 7
    h, dy, dres = (rows_of(s, rows, cols, dtype) for s in (4, 5, 6))
    w = rows_of(7, 1, cols, "f32").reshape(-1)
    rstd = torch.rsqrt(h.double().square().mean(1) + EPS).float()
    dx, dw = out((rows, cols + 1), T[dtype]), out((cols,), torch.float32)
    skg.rmsnorm_bwd(dy, h, rstd, dx, rows=rows, cols=cols, dtype=dtype, weight=w, dtype_w="f32", dres=dres, dw=dw,
                    lddx=cols + 1)
    torch.cuda.synchronize()
    H, DY, W, S, R = (f64(t) for t in (h, dy, w, rstd, dres))
    rx, rw = lowp.rmsnorm_bwd(DY, H, S, W)
    rx = rx + R
    u = 2.0 ** -24
    n, g = H * S[:, None], DY * W
    # as in the gradient's tests at other widths
    tol = S[:, None] * (8 * u * np.abs(g) + np.abs(n) * 80 * u * np.mean(np.abs(g * n), 1, keepdims=True))
    tiny = float(torch.finfo(T[dtype]).smallest_normal) * HALF[dtype] * 2
    tol = tol + 8 * u * np.abs(R) + HALF[dtype] * np.abs(rx) * (1 + 2.0 ** -10) + tiny
    assert np.all(np.abs(f64(dx[:, :cols]) - rx) <= tol)
    assert torch.isnan(dx[:, cols:].float()).all()
    assert np.all(np.abs(f64(dw) - rw) <= (rows + 4) * u * np.sum(np.abs(DY * n), 0) + 2.0 ** -126)


@pytest.mark.parametrize("cols", [32, 64, 128, 256])
def test_rows_that_share_a_wave(cols):
    """Ordinary rows give the same bits whatever their neighbours hold."""
    rows = 64
    x = rows_of(8, rows, cols, "bf16")
    clean_q, clean_s = out((rows, cols), torch.uint8), out((rows,), torch.float32)
    kw = dict(rows=rows, cols=cols, dtype="bf16", dtype_y="e4m3", eps=EPS)
    skg.rmsnorm(x, clean_q, y_scale=clean_s, **kw)
    odd = x.clone()
    odd[0, 3], odd[9, 1], odd[20] = float("nan"), float("inf"), 0
    odd[33], odd[47] = 3e38, 2.0 ** -130
    touched = [0, 9, 20, 33, 47]
    q, s = out((rows, cols), torch.uint8), out((rows,), torch.float32)
    skg.rmsnorm(odd, q, y_scale=s, **kw)
    torch.cuda.synchronize()
    rest = [i for i in range(rows) if i not in touched]
    assert torch.equal(q[rest], clean_q[rest]) and torch.equal(s[rest], clean_s[rest])
    s, v = s.cpu(), codecs.decode("e4m3", q.cpu().numpy())
    assert torch.isnan(s[[0, 9]]).all() and np.isnan(v[[0, 9]]).all()
    assert (s[[20, 33]] == 2.0 ** -126).all() and (v[[20, 33]] == 0).all()
    assert np.isfinite(v[47]).all()


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("transpose", [False, True])
def test_quant_widths(transpose, dtype, fmt):
    from test_gpu_fp4 import quant, same_codes, values
    for rows, cols in [(1, 2), (3, 7), (7, 8), (40, 9), (130, 33), (127, 129), (257, 127), (1, 257), (5, 4101)]:
        x = values(rows * 3 + cols, rows, cols, dtype)
        axis = rows if transpose else cols
        kq = -(-axis // 32) * 32
        q, s = quant(x.cuda(), fmt, rows, cols, dtype, kq, transpose)
        v = f64(x).T if transpose else f64(x)
        v = np.concatenate([v, np.zeros((v.shape[0], kq - axis))], 1)
        same_codes(q, s, v, fmt, "%dx%d %s %s" % (rows, cols, dtype, fmt))


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_lines_of_no_elements(fmt):
    """Lines without elements become padding: zero codes, the smallest scale."""
    for rows, cols, tr in ((3, 0, False), (0, 5, True)):
        lines, kq = (cols if tr else rows), 64
        q = out((lines, kq if fmt == "e4m3" else kq // 2), torch.uint8)
        s = out((lines, kq // 32), torch.uint8)
        skg.mx_quant(None, q, s, rows=rows, cols=cols, dtype="bf16", dtype_q=fmt, kq=kq, transpose=tr)
        torch.cuda.synchronize()
        assert (q == 0).all() and (s == 0).all()


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_many_chunks_with_ragged_lines(fmt):
    """More than 2^20 chunks (four a thread), lines that end inside one."""
    rows, cols = 1031, 8197
    kq = -(-cols // 32) * 32
    x = torch.randn(rows, cols, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16).cuda()
    q = out((rows, kq if fmt == "e4m3" else kq // 2), torch.uint8)
    s = out((rows, kq // 32), torch.uint8)
    back = out((rows, cols + 1), torch.bfloat16)
    kw = dict(rows=rows, cols=cols, dtype="bf16", dtype_q=fmt, kq=kq)
    skg.mx_quant(x, q, s, **kw)
    skg.mx_dequant(q, s, back, ldx=cols + 1, **kw)
    torch.cuda.synchronize()
    v = np.concatenate([f64(x), np.zeros((rows, kq - cols))], 1)
    rs, rq = lowp.mx_quantize(v, fmt)
    raw = q.cpu().numpy()
    assert np.array_equal(s.cpu().numpy(), rs)
    got = lowp.decode(fmt, raw if fmt == "e4m3" else lowp.unpack(raw))
    assert np.array_equal(got, lowp.decode(fmt, rq))
    want = torch.from_numpy(lowp.mx_values(rs, rq, fmt)[:, :cols]).float().to(torch.bfloat16)
    assert torch.equal(back[:, :cols].cpu(), want) and torch.isnan(back[:, cols:].float()).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 5), (31, 274), (33, 8), (509, 1111), (1024, 1024), (1025, 300), (257, 4079),
                                       (64, 16384), (65, 16384), (700, 33)])
def test_gradients_of_few_rows(rows, cols, dtype):
    """Both sides of the size up to which one launch makes both gradients: the
    values, and the same bits whichever are asked for and wherever dx goes."""
    h, dy, dres = (rows_of(s, rows, cols, dtype) for s in (10, 11, 12))
    rstd = torch.rsqrt(h.double().square().mean(1) + EPS).float()
    kw = dict(rows=rows, cols=cols, dtype=dtype)
    dx, dw, alone = out((rows, cols), T[dtype]), out((cols,), torch.float32), out((cols,), torch.float32)
    skg.rmsnorm_bwd(dy, h, rstd, dx, dres=dres, dw=dw, **kw)
    skg.rmsnorm_bwd(dy, h, rstd, None, dw=alone, **kw)
    only = out((rows, cols), T[dtype])
    skg.rmsnorm_bwd(dy, h, rstd, only, dres=dres, **kw)
    over_res, over_dy, dw2, dw3 = dres.clone(), dy.clone(), torch.empty_like(dw), torch.empty_like(dw)
    skg.rmsnorm_bwd(dy, h, rstd, over_res, dres=over_res, dw=dw2, **kw)
    skg.rmsnorm_bwd(over_dy, h, rstd, over_dy, dres=dres, dw=dw3, **kw)
    torch.cuda.synchronize()
    for t in (only, over_res, over_dy):
        assert torch.equal(t, dx)
    assert torch.equal(alone, dw) and torch.equal(dw2, dw)
    H, DY, S, R = (f64(t) for t in (h, dy, rstd, dres))
    rx, rw = lowp.rmsnorm_bwd(DY, H, S, np.ones(cols))
    rx = rx + R
    u = 2.0 ** -24
    n = H * S[:, None]
    # as in the gradient's tests at other sizes
    tol = S[:, None] * (8 * u * np.abs(DY) + np.abs(n) * 80 * u * np.mean(np.abs(DY * n), 1, keepdims=True))
    tiny = float(torch.finfo(T[dtype]).smallest_normal) * HALF[dtype] * 2
    tol = tol + 8 * u * np.abs(R) + HALF[dtype] * np.abs(rx) * (1 + 2.0 ** -10) + tiny
    assert np.all(np.abs(f64(dx) - rx) <= tol)
    for t in (dw, dw3):
        assert np.all(np.abs(f64(t) - rw) <= (rows + 4) * u * np.sum(np.abs(DY * n), 0) + 2.0 ** -126)
