"""Every fp4 tile of the product by itself, on operands whose sums are exact in
fp32 in any order: multiples of 2^-4 below 2^15, so a wrong scale, block, row,
tail or hand-over between waves changes the result."""

import numpy as np
import pytest
import torch

import implicit_gemm_conv_dp_amd as skg
from oracle import lowp

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TILES = ["16x16x512", "16x32x512", "16x64x512", "32x32x512", "32x64x512", "48x32x512", "64x64x512",
         "128x128x256", "256x256x256", "256x128x256"]


def operand(seed, rows, K):
    rng = np.random.default_rng(seed)
    q = rng.integers(0, 16, (rows, K)).astype(np.uint8)
    q = (q & 8) | np.minimum(q & 7, 4)  # magnitudes 0, 0.5, 1, 1.5, 2
    return q, rng.integers(126, 129, (rows, K // 32)).astype(np.uint8)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def spaced(q, ld):
    """Packed codes in rows of ld elements whose padding holds codes of 6; the
    last row ends with its own."""
    buf = np.full((q.shape[0], ld // 2), 0x77, np.uint8)
    buf[:, :q.shape[1] // 2] = lowp.pack(q)
    return dev(buf.reshape(-1)[:(q.shape[0] - 1) * (ld // 2) + q.shape[1] // 2])


def product(a, sa, b, sb, M, N, K, dtype_c, tile, lda=None, ldb=None):
    ldc = -(-N // 8) * 8 + 8
    C = torch.empty(M, ldc, dtype=T[dtype_c], device="cuda")
    C.view(torch.uint8).fill_(0xFF)
    plan = skg.gemm(a, b, C, sa, sb, M=M, N=N, K=K, lda=lda, ldb=ldb, ldc=ldc, dtype_ab="e2m1",
                    dtype_c=dtype_c, scale_mode="mx", tile=tile, mode="auto", reduction="auto", ctas=-1)
    torch.cuda.synchronize()
    assert plan["workspace_bytes"] == 0 and "%dx%dx%d" % (plan["tm"], plan["tn"], plan["tk"]) == tile
    C = C.cpu().double().numpy()
    assert np.isnan(C[:, N:]).all(), "columns past N written"
    return C[:, :N]


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("K", [128, 256, 384, 1024, 1152, 2304, 5120])
def test_exact(tile, K):
    tm, tn = map(int, tile.split("x")[:2])
    for M, N in ((1, 1), (tm, tn), (tm + 3, 2 * tn + 5), (2 * tm + 1, tn - 1)):
        (aq, as_), (bq, bs) = operand(1, M, K), operand(2, N, K)
        R = lowp.mx_values(as_, aq, "e2m1") @ lowp.mx_values(bs, bq, "e2m1").T
        # the bytes after the last row's scales are NaN codes
        s = [dev(np.append(v.reshape(-1), [255] * 64).astype(np.uint8)) for v in (as_, bs)]
        Y = product(dev(lowp.pack(aq)), s[0], dev(lowp.pack(bq)), s[1], M, N, K, "f32", tile)
        assert np.array_equal(Y, R), "%s %dx%dx%d: max diff %g" % (tile, M, N, K, np.nanmax(np.abs(Y - R)))


@pytest.mark.parametrize("tile", TILES)
def test_padded_rows_and_types(tile):
    tm, tn = map(int, tile.split("x")[:2])
    M, N, K = tm + 7, tn + 9, 640
    (aq, as_), (bq, bs) = operand(3, M, K), operand(4, N, K)
    R = lowp.mx_values(as_, aq, "e2m1") @ lowp.mx_values(bs, bq, "e2m1").T
    lda, ldb = K + 32, K + 160
    a, b = spaced(aq, lda), spaced(bq, ldb)
    for dt in T:
        Y = product(a, dev(as_), b, dev(bs), M, N, K, dt, tile, lda, ldb)
        want = torch.from_numpy(R).float().to(T[dt]).double().numpy()
        assert np.array_equal(Y, want), (tile, dt)


@pytest.mark.parametrize("tile", TILES)
def test_not_a_number_stays_in_its_row(tile):
    """A NaN scale reaches its own row or column, whole, and nothing else:
    neither a neighbour whose reduction ends within an iteration (K = 384, 640)
    nor rows past the operand's end."""
    for K in (384, 640, 1152):
        M, N = 21, 40
        (aq, as_), (bq, bs) = operand(5, M, K), operand(6, N, K)
        as_[5, 0], bs[7, -1] = 255, 255
        as_[6, -1] = 255
        R = lowp.mx_values(as_, aq, "e2m1") @ lowp.mx_values(bs, bq, "e2m1").T
        Y = product(dev(lowp.pack(aq)), dev(as_), dev(lowp.pack(bq)), dev(bs), M, N, K, "f32", tile)
        assert np.array_equal(np.isnan(Y), np.isnan(R))
        ok = ~np.isnan(R)
        assert ok.sum() == (M - 2) * (N - 1) and np.array_equal(Y[ok], R[ok])


@pytest.mark.parametrize("tile,dtype_c", [("128x128x256", "bf16"), ("128x128x256", "f32"), ("256x256x256", "f16"),
                                          ("256x256x256", "f32"), ("256x128x256", "bf16"), ("64x64x512", "bf16")])
def test_more_tiles_than_workgroups(tile, dtype_c):
    """Workgroups that take a second and a third tile, with the last strips of
    tiles cut short, for reductions of one, two and five iterations."""
    tm, tn = map(int, tile.split("x")[:2])
    for K in (256, 384, 1280):
        M, N = 18 * tm + 5, 29 * tn + 3
        (aq, as_), (bq, bs) = operand(7, M, K), operand(8, N, K)
        A, B = (torch.from_numpy(lowp.mx_values(s, q, "e2m1")).float().cuda() for s, q in ((as_, aq), (bs, bq)))
        R = (A @ B.t()).to(T[dtype_c])  # exact in fp32, then one rounding
        C = torch.full((M, -(-N // 8) * 8), float("nan"), dtype=T[dtype_c], device="cuda")
        for _ in range(2):
            C.fill_(float("nan"))
            skg.gemm(dev(lowp.pack(aq)), dev(lowp.pack(bq)), C, dev(as_), dev(bs), M=M, N=N, K=K, ldc=C.shape[1],
                     dtype_ab="e2m1", dtype_c=dtype_c, scale_mode="mx", tile=tile, mode="dp", reduction="tree",
                     ctas=1)
            torch.cuda.synchronize()
            assert torch.equal(C[:, :N], R), (tile, K)
            assert torch.isnan(C[:, N:].float()).all()


@pytest.mark.parametrize("tile", TILES)
def test_repeats_give_the_same_bits(tile):
    """Sums that are not exact, five times, and replayed from a graph with
    other work between the replays."""
    M, N, K = 150, 170, 4096
    rng = np.random.default_rng(9)
    a, b = (dev(rng.integers(0, 256, (n, K // 2)).astype(np.uint8)) for n in (M, N))
    sa, sb = (dev(rng.integers(119, 136, (n, K // 32)).astype(np.uint8)) for n in (M, N))
    C = torch.empty(M, 176, device="cuda")
    kw = dict(M=M, N=N, K=K, ldc=176, dtype_ab="e2m1", dtype_c="f32", scale_mode="mx", tile=tile, mode="dp",
              reduction="linear", ctas=1)
    skg.gemm(a, b, C, sa, sb, **kw)
    want = C[:, :N].clone()
    A, B = lowp.mx_values(sa.cpu().numpy(), lowp.unpack(a.cpu().numpy()), "e2m1"), \
        lowp.mx_values(sb.cpu().numpy(), lowp.unpack(b.cpu().numpy()), "e2m1")
    assert np.all(np.abs(want.cpu().double().numpy() - A @ B.T) <= K * 2.0 ** -23 * (np.abs(A) @ np.abs(B).T))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        skg.gemm(a, b, C, sa, sb, **kw)
    for i in range(4):
        C.fill_(float("nan"))
        if i % 2:
            g.replay()
        else:
            skg.gemm(a, b, C, sa, sb, **kw)
        torch.cuda.synchronize()
        assert torch.equal(C[:, :N], want)
        (torch.ones(1000, device="cuda") * 2).sum().item()
