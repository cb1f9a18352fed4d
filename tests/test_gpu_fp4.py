"""GPU parity of MX quantisation, reading back and the fp4 product, against
float64: quantisation is exact (dividing by a power of two is, and each element
is rounded once), so codes and scales are compared bit by bit; the product is
bit-exact on operands whose sums are exact in fp32 and within K roundings of
fp32 otherwise."""

import numpy as np
import pytest
import torch

import implicit_gemm_conv_dp_amd as skg
from oracle import codecs, lowp

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}


def f64(t):
    return t.cpu().to(torch.float64).numpy()


def poison(shape, dtype=torch.uint8):
    t = torch.empty(shape, dtype=dtype, device="cuda")
    t.view(torch.uint8).fill_(0xFF)
    return t


def quant(x, fmt, rows, cols, dtype, kq=None, transpose=False, ldx=None, pad=0):
    lines = cols if transpose else rows
    kq = kq or -(-(rows if transpose else cols) // 32) * 32
    ldq = kq + pad
    q = poison((lines, ldq if fmt == "e4m3" else ldq // 2))
    s = poison((lines, kq // 32))
    skg.mx_quant(x, q, s, rows=rows, cols=cols, dtype=dtype, dtype_q=fmt, kq=kq, ldx=ldx, ldq=ldq,
                 transpose=transpose)
    torch.cuda.synchronize()
    q = q.cpu().numpy()
    n = kq if fmt == "e4m3" else kq // 2
    assert (q[:, n:] == 0xFF).all()
    return (q[:, :n] if fmt == "e4m3" else lowp.unpack(q[:, :n])), s.cpu().numpy()


def same_codes(q, s, x, fmt, label):
    rs, rq = lowp.mx_quantize(x, fmt)
    assert np.array_equal(s, rs), "%s: scales differ" % label
    # the sign of a zero is not part of the value
    assert np.array_equal(lowp.decode(fmt, q), lowp.decode(fmt, rq)), "%s: codes differ" % label


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_every_bf16_value(fmt):
    """Each finite bf16 pattern at each place that a block's largest element
    gives it: 31 consecutive patterns per block beside a largest element of
    1 to 12 times 2^k of theirs."""
    bits = np.arange(0, 0x7F80, dtype=np.int64)
    rows = []
    for mul in (0, 1, 2, 4, 9, 30, 300, 1500):
        v = codecs.decode("bf16", bits)
        v = np.concatenate([v, np.zeros(-len(v) % 31)]).reshape(-1, 31)
        big = np.minimum(v.max(1, keepdims=True) * (mul * 0.37 if mul else 0), 3e38)
        rows.append(np.concatenate([v * np.where(np.arange(31) % 2, -1, 1), big], 1))
    x = torch.from_numpy(np.concatenate(rows)).to(torch.bfloat16)
    n = x.shape[0]
    q, s = quant(x.cuda(), fmt, n, 32, "bf16")
    same_codes(q, s, f64(x), fmt, "bf16 sweep")


def values(seed, rows, cols, dtype):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-9, 9, (rows, cols // 32 + 1), generator=g)
                                                          .float().repeat_interleave(32, 1)[:, :cols])
    x[:, ::7] = torch.round(x[:, ::7] * 4) / 4    # values on the codes' borders
    if rows > 1:
        x[1, :33] = 0
    return x.to(T[dtype])


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_shapes(dtype, fmt, transpose):
    for rows, cols, more, pad, ld in [(1, 32, 0, 0, 0), (1, 1, 0, 0, 0), (3, 70, 32, 32, 5), (64, 64, 0, 0, 8),
                                      (129, 130, 96, 64, 3), (300, 4096, 0, 0, 0), (32, 2049, 0, 32, 1)]:
        x = values(rows + cols, rows, cols, dtype)
        buf = torch.full((rows, cols + ld), float("nan"), dtype=T[dtype])
        buf[:, :cols] = x
        axis = rows if transpose else cols
        kq = -(-axis // 32) * 32 + more
        q, s = quant(buf.cuda(), fmt, rows, cols, dtype, kq, transpose, cols + ld, pad)
        v = f64(x).T if transpose else f64(x)
        v = np.concatenate([v, np.zeros((v.shape[0], kq - axis))], 1)
        same_codes(q, s, v, fmt, "%dx%d %s %s" % (rows, cols, dtype, fmt))


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_not_finite_and_extreme(fmt, transpose):
    x = values(5, 64, 128, "f32")
    x[0, 3], x[40, 70], x[50, 127] = float("nan"), float("inf"), float("-inf")
    x[2] = 2.0 ** -149
    x[3, :32] = 2.0 ** -126 * 1.75
    x[4, 5] = 3.4e38
    q, s = quant(x.cuda(), fmt, 64, 128, "f32", transpose=transpose)
    same_codes(q, s, f64(x).T if transpose else f64(x), fmt, fmt)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_reading_back(fmt, dtype):
    rng = np.random.default_rng(6)
    for rows, cols, more, pad in [(16, 32, 0, 0), (5, 70, 32, 64), (33, 4096, 0, 0)]:
        kq = -(-cols // 32) * 32 + more
        s = rng.integers(100, 140, (rows, kq // 32)).astype(np.uint8)
        s[0, 0], s[1, 0] = 255, 0
        q = rng.integers(0, 16 if fmt == "e2m1" else 256, (rows, kq)).astype(np.uint8)
        q[2, :16] = np.arange(16)
        raw = lowp.pack(q) if fmt == "e2m1" else q
        dq = torch.from_numpy(np.ascontiguousarray(raw)).cuda()
        y = poison((rows, cols + pad), T[dtype])
        skg.mx_dequant(dq, torch.from_numpy(s).cuda(), y, rows=rows, cols=cols, kq=kq, ldx=cols + pad,
                       dtype_q=fmt, dtype=dtype)
        torch.cuda.synchronize()
        want = torch.from_numpy(lowp.mx_values(s, q, fmt)[:, :cols]).float().to(T[dtype])
        assert np.array_equal(f64(y[:, :cols]), f64(want), equal_nan=True)
        assert torch.isnan(y[:, cols:].float()).all()


# --- the product ---------------------------------------------------------------
def operand(seed, rows, K, exact):
    rng = np.random.default_rng(seed)
    q = rng.integers(0, 16, (rows, K)).astype(np.uint8)
    if exact:  # magnitudes 0, 0.5, 1, 1.5, 2
        q = (q & 8) | np.minimum(q & 7, 4)
        s = rng.integers(126, 129, (rows, K // 32))
    else:
        s = rng.integers(119, 136, (rows, K // 32))
    return q, s.astype(np.uint8)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def product(aq, as_, bq, bs, M, N, K, dtype_c, ldc=None, lda=None, ldb=None, **kw):
    ldc = ldc or -(-N // 8) * 8
    C = poison((M, ldc), T[dtype_c])
    plan = skg.gemm(aq, bq, C, as_, bs, M=M, N=N, K=K, lda=lda, ldb=ldb, ldc=ldc, dtype_ab="e2m1",
                    dtype_c=dtype_c, scale_mode="mx", **kw)
    torch.cuda.synchronize()
    C = f64(C)
    assert np.isnan(C[:, N:]).all(), "padding written"
    return C[:, :N], plan


TILES = ["128x128x256", "256x256x256"]
LAUNCHES = [("dp", "linear", 1), ("dp_sk", "linear", 5), ("dp_sk", "tree", 7), ("dp_sk", "atomic", 5),
            ("dp_sk", "workspace", 13), ("persistent", "tree", 5), ("persistent", "linear", 3),
            ("persistent", "workspace", 7), ("splitk", "scatter", 3), ("splitk", "workspace", 2)]


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("K", [128, 256, 1152, 2304])
def test_exact_products(tile, K):
    """Sums of multiples of 2^-4 below 2^15: exact in fp32 in any order, so a
    wrong scale, block, row or tail changes the result.  K = 128 and 1152
    end half way through a tile's 256."""
    tm = int(tile.split("x")[0])
    M, N = tm + 40, tm + 77
    (aq, as_), (bq, bs) = operand(1, M, K, True), operand(2, N, K, True)
    R = lowp.mx_values(as_, aq, "e2m1") @ lowp.mx_values(bs, bq, "e2m1").T
    # the bytes after the last row's scales are NaN codes
    d = [dev(lowp.pack(aq)), dev(np.append(as_.reshape(-1), [255] * 16).astype(np.uint8)), dev(lowp.pack(bq)),
         dev(np.append(bs.reshape(-1), [255] * 16).astype(np.uint8))]
    for mode, red, ctas in LAUNCHES:
        if red == "scatter" and (K // 256) % 3:
            continue
        Y, plan = product(*d, M, N, K, "f32", mode=mode, reduction=red, ctas=ctas, tile=tile)
        assert np.array_equal(Y, R), "%s K=%d %s %s: max diff %g" % (tile, K, mode, red, np.nanmax(np.abs(Y - R)))


@pytest.mark.parametrize("tile", TILES)
def test_scale_of_a_neighbouring_row_is_not_read(tile):
    """K = 384: the second half of the tile's last iteration lies past K, and
    the next row's NaN scale must not reach it."""
    M, N, K = 70, 90, 384
    (aq, as_), (bq, bs) = operand(3, M, K, True), operand(4, N, K, True)
    as_[5], bs[7] = 255, 255
    Y, _ = product(dev(lowp.pack(aq)), dev(as_), dev(lowp.pack(bq)), dev(bs), M, N, K, "f32", mode="dp",
                   reduction="linear", ctas=1, tile=tile)
    R = lowp.mx_values(as_, aq, "e2m1") @ lowp.mx_values(bs, bq, "e2m1").T
    assert np.array_equal(np.isnan(Y), np.isnan(R))
    ok = ~np.isnan(R)
    assert ok.sum() == (M - 1) * (N - 1) and np.array_equal(Y[ok], R[ok])


@pytest.mark.parametrize("dtype_c", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 128), (1, 64, 4096), (3, 257, 1280), (16, 500, 896), (17, 130, 640),
                                   (48, 4863, 512), (65, 100, 8192), (200, 333, 384), (513, 1025, 1024)])
def test_auto(M, N, K, dtype_c):
    (aq, as_), (bq, bs) = operand(5, M, K, False), operand(6, N, K, False)
    A, B = lowp.mx_values(as_, aq, "e2m1"), lowp.mx_values(bs, bq, "e2m1")
    Y, plan = product(dev(lowp.pack(aq)), dev(as_), dev(lowp.pack(bq)), dev(bs), M, N, K, dtype_c, tile="auto",
                      mode="auto", reduction="auto", ctas=-1)
    R, S = A @ B.T, np.abs(A) @ np.abs(B).T
    # K additions of fp32, each off by at most one unit in the last place
    # of a sum no larger than S, then one rounding
    tol = K * 2.0 ** -23 * S + HALF[dtype_c] * np.abs(R) * (1 + 2.0 ** -10)
    if dtype_c == "f16":
        tol = tol + 2.0 ** -25
    big = np.abs(R) > 65504 if dtype_c == "f16" else np.zeros_like(R, bool)
    assert np.all((np.abs(Y - R) <= tol) | big), (plan, np.max(np.abs(Y - R) - tol))


@pytest.mark.parametrize("M", [1, 20, 130])
def test_padded_rows(M):
    N, K = 72, 512
    (aq, as_), (bq, bs) = operand(7, M, K, True), operand(8, N, K, True)
    lda, ldb, ldc = K + 32, K + 96, N + 8
    pa, pb = np.full((M, lda // 2), 0x77, np.uint8), np.full((N, ldb // 2), 0x77, np.uint8)
    pa[:, :K // 2], pb[:, :K // 2] = lowp.pack(aq), lowp.pack(bq)
    R = lowp.mx_values(as_, aq, "e2m1") @ lowp.mx_values(bs, bq, "e2m1").T
    for tile in TILES + ["auto"]:
        Y, _ = product(dev(pa), dev(as_), dev(pb), dev(bs), M, N, K, "f32", ldc, lda, ldb, tile=tile, mode="auto",
                       reduction="auto", ctas=-1)
        assert np.array_equal(Y, R), tile


@pytest.mark.parametrize("M,N,K", [(1, 512, 4096), (40, 300, 8192), (300, 512, 2048)])
def test_graph_capture(M, N, K):
    (aq, as_), (bq, bs) = operand(9, M, K, False), operand(10, N, K, False)
    a, sa, b, sb = dev(lowp.pack(aq)), dev(as_), dev(lowp.pack(bq)), dev(bs)
    C = poison((M, -(-N // 8) * 8), torch.float32)
    kw = dict(M=M, N=N, K=K, ldc=C.shape[1], dtype_ab="e2m1", dtype_c="f32", scale_mode="mx", tile="auto",
              mode="auto", reduction="auto", ctas=-1)
    ws = skg.workspace_for(skg.plan_gemm(**kw), "cuda")
    skg.gemm(a, b, C, sa, sb, workspace=ws, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        skg.gemm(a, b, C, sa, sb, workspace=ws, **kw)
    for i in range(4):
        q, s = operand(20 + i, M, K, True)
        a.copy_(dev(lowp.pack(q)))
        sa.copy_(dev(s))
        skg.gemm(a, b, C, sa, sb, workspace=ws, **kw)
        torch.cuda.synchronize()
        want = f64(C)
        C.view(torch.uint8).fill_(0xFF)
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        got = f64(C)
        tol = K * 2.0 ** -23 * (np.abs(lowp.mx_values(s, q, "e2m1")) @ np.abs(lowp.mx_values(bs, bq, "e2m1")).T)
        assert np.all(np.abs(got - want)[:, :N] <= 2 * tol)


def test_largest_shape_sampled():
    """8192 x 8192 x 8192 through the largest tile, on sampled entries."""
    M = N = K = 8192
    rng = np.random.default_rng(11)
    q = [rng.integers(0, 256, (8192, K // 2)).astype(np.uint8) for _ in range(2)]
    s = [rng.integers(120, 134, (8192, K // 32)).astype(np.uint8) for _ in range(2)]
    Y, plan = product(dev(q[0]), dev(s[0]), dev(q[1]), dev(s[1]), M, N, K, "f32", tile="auto", mode="auto",
                      reduction="auto", ctas=-1)
    assert not np.isnan(Y).any()
    for _ in range(300):
        m, n = rng.integers(0, 8192, 2)
        a = lowp.mx_values(s[0][m], lowp.unpack(q[0][m]), "e2m1")
        b = lowp.mx_values(s[1][n], lowp.unpack(q[1][n]), "e2m1")
        assert abs(Y[m, n] - a @ b) <= K * 2.0 ** -23 * (np.abs(a) @ np.abs(b))
