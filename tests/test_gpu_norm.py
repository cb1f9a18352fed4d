"""GPU parity of the root-mean-square norm with the residual's addition, its
quantised outputs and its gradient, against float64.

With u = 2^-24 and rows of up to 32768 elements summed in runs of at most 32
and then by a tree, the sum of squares is within 64 u, the row's factor within
40 u and y within 48 u, for which DELTA = 2^-18 leaves room; a rounding to the
row's type adds half a step.  A quantised output has to lie between the codes
of y (1 - DELTA) and y (1 + DELTA) at the scale the kernel wrote (rounding is
monotone), and its scale within DELTA of the definition's (MX: the code of a
largest magnitude within DELTA)."""

import numpy as np
import pytest
import torch

import implicit_gemm_conv_dp_amd as skg
from oracle import codecs, lowp

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
DELTA = 2.0 ** -18
EPS = 1e-5


def rows_of(seed, rows, cols, dtype, ld=None):
    """Rows with large channels, an empty row and a tiny one, in a buffer of
    pitch ld whose padding is NaN."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(torch.randn(cols, generator=g))
    if rows > 2:
        x[1] = 0
        x[2] *= 2.0 ** -12
    buf = torch.full((rows, ld or cols), float("nan"))
    buf[:, :cols] = x
    return buf.to(T[dtype]).cuda()


def f64(t):
    return t.cpu().to(torch.float64).numpy()


def out(shape, dtype):
    n = torch.empty(shape, dtype=dtype, device="cuda")
    n.view(torch.uint8).fill_(0xFF)
    return n


SHAPES = [(1, 1), (3, 7), (5, 32), (4, 512), (9, 513), (3, 1000), (2, 2048), (3, 2080), (2, 4096),
          (3, 5120), (1, 8192), (2, 8200), (2, 16384), (1, 32768), (1030, 64)]


def check_values(y, ref, dtype, label):
    # one rounding, a subnormal's absolute half step included
    tiny = float(torch.finfo(T[dtype]).smallest_normal) * HALF[dtype] * 2
    bad = np.abs(y - ref) > (DELTA + HALF[dtype]) * np.abs(ref) + tiny
    assert not bad.any(), "%s: %d off, first %s" % (label, bad.sum(), np.argwhere(bad)[:3])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(rows, cols, dtype):
    for residual, w32, pad in ((True, False, 0), (True, True, 3), (False, True, 8)):
        ld = cols + pad
        x = rows_of(1, rows, cols, dtype, ld)
        r = rows_of(2, rows, cols, dtype, cols + 1) if residual else None
        w = rows_of(3, 1, cols, "f32" if w32 else dtype).reshape(-1)
        h, y = out((rows, ld), T[dtype]), out((rows, ld), T[dtype])
        rstd = out((rows,), torch.float32)
        skg.rmsnorm(x, y, rows=rows, cols=cols, dtype=dtype, weight=w,
                    dtype_w="f32" if w32 else dtype, residual=r, h=h, rstd=rstd, eps=EPS, ldx=ld,
                    ldr=cols + 1, ldh=ld, ldy=ld)
        torch.cuda.synchronize()
        want = x[:, :cols].cpu().float()
        if residual:
            want = want + r[:, :cols].cpu().float()
        want = want.to(T[dtype])
        assert torch.equal(h[:, :cols].cpu(), want)
        ref, rr = lowp.rmsnorm(f64(want), f64(w), EPS)
        label = "%dx%d %s pad %d" % (rows, cols, dtype, pad)
        check_values(f64(y[:, :cols]), ref, dtype, label)
        assert np.all(np.abs(f64(rstd) - rr) <= DELTA * rr), label
        if pad:  # what lies between the rows is not written
            assert torch.isnan(h[:, cols:].float()).all() and torch.isnan(y[:, cols:].float()).all()


def check_codes(fmt, codes, d, y, label):
    """codes (float64 values) within the codes of y (1 -+ DELTA) at scale d."""
    a = lowp.decode(fmt, lowp.encode(fmt, y * (1 - DELTA) / d))
    b = lowp.decode(fmt, lowp.encode(fmt, y * (1 + DELTA) / d))
    bad = (codes < np.minimum(a, b)) | (codes > np.maximum(a, b))
    assert not bad.any(), "%s: %d codes off, first %s" % (label, bad.sum(), np.argwhere(bad)[:3])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_row_scaled(rows, cols, dtype):
    x, r = rows_of(4, rows, cols, dtype), rows_of(5, rows, cols, dtype)
    w = rows_of(6, 1, cols, "f32").reshape(-1)
    h, q = out((rows, cols), T[dtype]), out((rows, cols + 5), torch.uint8)
    sc = out((rows,), torch.float32)
    skg.rmsnorm(x, q, rows=rows, cols=cols, dtype=dtype, weight=w, dtype_w="f32", residual=r, h=h,
                y_scale=sc, dtype_y="e4m3", eps=EPS, ldy=cols + 5)
    torch.cuda.synchronize()
    y, _ = lowp.rmsnorm(f64(h), f64(w), EPS)
    d = np.maximum(np.abs(y).max(1) / 448, 2.0 ** -126)
    s = f64(sc)
    assert np.all(np.abs(s - d) <= DELTA * d)
    codes = codecs.decode("e4m3", q.cpu().numpy()[:, :cols])
    check_codes("e4m3", codes, s[:, None], y, "%dx%d %s" % (rows, cols, dtype))
    assert (q[:, cols:] == 0xFF).all()


def test_row_scaled_borders_are_exact():
    # Products of a power of two with small integers: half of the quotients
    # by the row's largest (448) lie exactly between two codes, and go to
    # the even one whatever the row's factor is.
    v = torch.arange(1, 449, dtype=torch.float32).repeat(2)[:512 + 320]
    x = (v * 2.0 ** -9).to(torch.bfloat16).float()
    x[0] = 448 * 2.0 ** -9
    x = x.to(torch.bfloat16).cuda().reshape(1, -1)
    cols = x.shape[1]
    q, sc = out((1, cols), torch.uint8), out((1,), torch.float32)
    skg.rmsnorm(x, q, rows=1, cols=cols, dtype="bf16", y_scale=sc, dtype_y="e4m3", eps=EPS)
    torch.cuda.synchronize()
    want = codecs.encode("e4m3", f64(x)[0] * 2.0 ** 9)
    assert np.array_equal(q.cpu().numpy()[0], want)


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 32), (7, 96), (3, 512), (5, 2080), (37, 5120), (2, 16416)])
def test_mx_outputs(rows, cols, dtype, fmt):
    x, r = rows_of(7, rows, cols, dtype), rows_of(8, rows, cols, dtype)
    w = rows_of(9, 1, cols, dtype).reshape(-1)
    ldy = cols + 32
    h, q = out((rows, cols), T[dtype]), out((rows, ldy if fmt == "e4m3" else ldy // 2), torch.uint8)
    sc = out((rows, cols // 32), torch.uint8)
    skg.rmsnorm(x, q, rows=rows, cols=cols, dtype=dtype, weight=w, residual=r, h=h, y_scale=sc,
                dtype_y=fmt, scale_mode="mx", eps=EPS, ldy=ldy)
    torch.cuda.synchronize()
    y, _ = lowp.rmsnorm(f64(h), f64(w), EPS)
    s = sc.cpu().numpy()
    lo, hi = lowp.mx_scales(y * (1 - DELTA), fmt), lowp.mx_scales(y * (1 + DELTA), fmt)
    assert np.all((s >= lo) & (s <= hi))
    n = cols if fmt == "e4m3" else cols // 2
    raw = q.cpu().numpy()
    assert (raw[:, n:] == 0xFF).all()
    codes = lowp.decode(fmt, raw[:, :n] if fmt == "e4m3" else lowp.unpack(raw[:, :n]))
    check_codes(fmt, codes, np.repeat(lowp.scale_value(s), 32, axis=1), y, "%dx%d" % (rows, cols))


def test_not_finite_rows():
    cols = 1024
    x = rows_of(10, 6, cols, "bf16")
    x[0, 5] = float("nan")
    x[3, 900] = float("inf")
    x[4] = 3e38          # the sum of squares leaves fp32: s = 0
    x[5] = 2.0 ** -130   # y far below the smallest scale's codes
    clean = x.clone()
    clean[:, :] = torch.where(torch.isfinite(x), x, 0)
    for fmt, mode in (("bf16", "rowcol"), ("e4m3", "rowcol"), ("e4m3", "mx"), ("e2m1", "mx")):
        q = out((6, cols // 2 if fmt == "e2m1" else cols), T["bf16"] if fmt == "bf16" else torch.uint8)
        sc = out((6,), torch.float32) if mode == "rowcol" else out((6, cols // 32), torch.uint8)
        skg.rmsnorm(x, q, rows=6, cols=cols, dtype="bf16", y_scale=sc, dtype_y=fmt, scale_mode=mode,
                    eps=EPS)
        torch.cuda.synchronize()
        if fmt == "bf16":
            # inf * 0 is NaN; the row's finite elements times s = 0 are 0
            y = q.float().cpu()
            assert torch.isnan(y[0]).all() and torch.isnan(y[3, 900]) and (y[3, :900] == 0).all()
            assert (y[4] == 0).all() and (y[1] == 0).all()
        elif mode == "rowcol":
            codes = codecs.decode("e4m3", q.cpu().numpy())
            s = sc.cpu()
            assert torch.isnan(s[0]) and torch.isnan(s[3])
            assert np.isnan(codes[0]).all() and np.isnan(codes[3]).all()
            assert s[1] == 2.0 ** -126 and s[4] == 2.0 ** -126
            assert (codes[1] == 0).all() and (codes[4] == 0).all()
            assert np.isfinite(codes[2]).all() and np.isfinite(codes[5]).all()
        else:
            s = sc.cpu()
            assert (s[0] == 255).all() and s[3, 900 // 32] == 255 and (s[4] == 0).all()
            assert (s[1] == 0).all() and (q[0] == 0).all() and (q[1] == 0).all()


def test_in_place_and_other_stream():
    rows, cols = 33, 3000
    x, r = rows_of(11, rows, cols, "f16"), rows_of(12, rows, cols, "f16")
    h, y, y2 = out((rows, cols), T["f16"]), out((rows, cols), T["f16"]), out((rows, cols), T["f16"])
    skg.rmsnorm(x, y, rows=rows, cols=cols, dtype="f16", residual=r, h=h, eps=EPS)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    skg.rmsnorm(x, y2, rows=rows, cols=cols, dtype="f16", residual=r, h=r, eps=EPS, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(h, r) and torch.equal(y, y2)


BWD_SHAPES = [(1, 1), (3, 7), (130, 64), (2500, 96), (5, 513), (33, 1111), (3, 2048), (40, 4096),
              (5, 8200), (2, 16384), (3, 32768), (700, 2304)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", BWD_SHAPES)
def test_backward(rows, cols, dtype):
    for res, w32, pad in ((True, True, 0), (False, False, 3)):
        ld = cols + pad
        h, dy = rows_of(13, rows, cols, dtype, ld), rows_of(14, rows, cols, dtype, ld)
        w = rows_of(15, 1, cols, "f32" if w32 else dtype).reshape(-1)
        dres = rows_of(16, rows, cols, dtype, ld) if res else None
        rstd = torch.rsqrt(h[:, :cols].double().square().mean(1) + EPS).float()
        dx, dw = out((rows, ld), T[dtype]), out((cols,), torch.float32)
        skg.rmsnorm_bwd(dy, h, rstd, dx, rows=rows, cols=cols, dtype=dtype, weight=w,
                        dtype_w="f32" if w32 else dtype, dres=dres, dw=dw, lddy=ld, ldh=ld,
                        lddres=ld, lddx=ld)
        torch.cuda.synchronize()
        H, DY, W, S = f64(h[:, :cols]), f64(dy[:, :cols]), f64(w), f64(rstd)
        rx, rw = lowp.rmsnorm_bwd(DY, H, S, W)
        R = f64(dres[:, :cols]) if res else 0.0
        rx = rx + R
        u = 2.0 ** -24
        n, g = H * S[:, None], DY * W
        # The mean of g n is within 64 u of its absolute mean; each term of dx
        # takes at most 8 roundings of fp32, then one to the row's type.
        tol = S[:, None] * (8 * u * np.abs(g) + np.abs(n) * 80 * u * np.mean(np.abs(g * n), 1, keepdims=True))
        tiny = float(torch.finfo(T[dtype]).smallest_normal) * HALF[dtype] * 2
        tol = tol + 8 * u * np.abs(R) + HALF[dtype] * np.abs(rx) * (1 + 2.0 ** -10) + tiny
        got = f64(dx[:, :cols])
        label = "%dx%d %s" % (rows, cols, dtype)
        assert np.all(np.abs(got - rx) <= tol), label
        # dw: at most `rows` additions of fp32 and a rounding of each term
        toln = (rows + 4) * u * np.sum(np.abs(DY * n), 0) + 2.0 ** -126
        assert np.all(np.abs(f64(dw) - rw) <= toln), label
        if pad:
            assert torch.isnan(dx[:, cols:].float()).all()


def test_backward_parts_and_repeats():
    rows, cols = 777, 2304
    h, dy = rows_of(17, rows, cols, "bf16"), rows_of(18, rows, cols, "bf16")
    rstd = torch.rsqrt(h.double().square().mean(1) + EPS).float()
    kw = dict(rows=rows, cols=cols, dtype="bf16")
    dx, dw = out((rows, cols), T["bf16"]), out((cols,), torch.float32)
    skg.rmsnorm_bwd(dy, h, rstd, dx, dw=dw, **kw)
    dx2, dw2 = out((rows, cols), T["bf16"]), out((cols,), torch.float32)
    skg.rmsnorm_bwd(dy, h, rstd, dx2, **kw)
    skg.rmsnorm_bwd(dy, h, rstd, None, dw=dw2, **kw)
    torch.cuda.synchronize()
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    # in place over dy, and no rows at all
    d3 = dy.clone()
    skg.rmsnorm_bwd(d3, h, rstd, d3, dw=dw2, **kw)
    torch.cuda.synchronize()
    assert torch.equal(d3, dx) and torch.equal(dw, dw2)
    skg.rmsnorm_bwd(dy, h, rstd, dx, dw=dw2, rows=0, cols=cols, dtype="bf16")
    torch.cuda.synchronize()
    assert (dw2 == 0).all()


def test_graph_capture():
    rows, cols = 64, 4096
    x, r = rows_of(19, rows, cols, "bf16"), rows_of(20, rows, cols, "bf16")
    dy = rows_of(21, rows, cols, "bf16")
    h, q = out((rows, cols), T["bf16"]), out((rows, cols), torch.uint8)
    sc, rstd, dw = out((rows,), torch.float32), out((rows,), torch.float32), out((cols,), torch.float32)
    dx, ws = out((rows, cols), T["bf16"]), out((64 << 20,), torch.uint8)

    def step():
        skg.rmsnorm(x, q, rows=rows, cols=cols, dtype="bf16", residual=r, h=h, rstd=rstd, y_scale=sc,
                    dtype_y="e4m3", eps=EPS)
        skg.rmsnorm_bwd(dy, h, rstd, dx, rows=rows, cols=cols, dtype="bf16", dw=dw, workspace=ws)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        x.copy_(rows_of(30 + i, rows, cols, "bf16"))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (h, q, sc, dx, dw)]
        for t in (h, q, sc, dx, dw):
            t.view(torch.uint8).fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, (h, q, sc, dx, dw)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
