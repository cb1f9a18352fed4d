"""GPU parity of the Newton-Schulz update against float64.

What the GPU does is the iteration with X, S and the polynomial rounded to fp16
at three places a step; the oracle runs just that in float64 (``rounded``).  Both
differ from the unrounded iteration by roundings of the same sizes at the same
places, propagated by the same maps, so the GPU's distance from it is the
oracle's up to which way single roundings fall (fp32 sums move an element over a
border now and then): at most half as much again, and 2^-14 of the result for
the fp32 sums of up to 2000 terms that are rounded at random, each 2^-24.  The
output's own rounding comes on top, half a step an element."""

import numpy as np
import pytest
import torch

import implicit_gemm_conv_dp_amd as skg
from oracle import projection as pj

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
MUON = (3.4445, -4.7750, 2.0315)
EPS = 1e-7


def f64(t):
    return t.cpu().to(torch.float64).numpy()


def gradient(seed, rows, cols, dtype, ld=None, size=1e-3):
    g = torch.Generator().manual_seed(seed)
    r = max(1, min(rows, cols) // 8)
    x = torch.randn(rows, r, generator=g) @ torch.randn(r, cols, generator=g) / r ** 0.5
    x = size * (x + 0.5 * torch.randn(rows, cols, generator=g))
    buf = torch.full((rows, ld or cols), float("nan"))
    buf[:, :cols] = x
    return buf.to(T[dtype]).cuda()


def run(g, rows, cols, dtype, dtype_out="f32", pad=0, **kw):
    out = torch.full((rows, cols + pad), float("nan"), dtype=T[dtype_out], device="cuda")
    skg.newton_schulz(g, out, rows=rows, cols=cols, dtype=dtype, dtype_out=dtype_out, ldg=g.shape[1], ldo=cols + pad, **kw)
    torch.cuda.synchronize()
    assert torch.isnan(out[:, cols:]).all()
    return f64(out)[:, :cols]


def check(got, g, dtype_out, coefficients=(MUON,) * 5, eps=EPS, scale=1.0):
    want = pj.newton_schulz(g, coefficients, eps, scale)
    near = pj.newton_schulz(g, coefficients, eps, scale, rounded=True)
    n = np.linalg.norm(want)
    off, own = np.linalg.norm(got - want), np.linalg.norm(near - want)
    assert off <= 1.5 * own + (2.0 ** -14 + HALF[dtype_out]) * n, (off / n, own / n)


SHAPES = [(1, 1), (1, 300), (300, 1), (5, 3), (33, 70), (64, 64), (70, 33), (128, 200), (200, 129), (300, 1111), (257, 256), (64, 4096)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype,dtype_out", [("f32", "bf16"), ("bf16", "f32"), ("f16", "f16")])
def test_update(rows, cols, dtype, dtype_out):
    g = gradient(rows + cols, rows, cols, dtype, cols + 3)
    check(run(g, rows, cols, dtype, dtype_out, pad=5), f64(g)[:, :cols], dtype_out)


TILES = [t for t in skg.NS_TILES if t != "auto"]


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("rows,cols,dtype_out", [(200, 129, "bf16"), (129, 200, "f32"), (5, 3, "f16"), (700, 333, "f32"),
                                                 (333, 700, "bf16"), (513, 512, "bf16")])
def test_update_on_every_tile(tile, rows, cols, dtype_out):
    pad = 0 if rows == 513 else 3
    g = gradient(rows, rows, cols, "f32")
    check(run(g, rows, cols, "f32", dtype_out, pad=pad, tile=tile), f64(g), dtype_out)


@pytest.mark.parametrize("tile", ["auto"] + TILES)
def test_cubic_steps(tile):
    """c = 0: the polynomial is a multiple of S."""
    cs = [(1.5, -0.5, 0.0)] * 6
    g = gradient(14, 150, 210, "f32")
    check(run(g, 150, 210, "f32", steps=6, coefficients=cs, tile=tile), f64(g), "f32", cs)


def test_linear_steps():
    """b = c = 0, and no product at all contributes."""
    cs = [(1.25, 0.0, 0.0)] * 3
    g = gradient(15, 64, 40, "f32")
    check(run(g, 64, 40, "f32", steps=3, coefficients=cs), f64(g), "f32", cs)


@pytest.mark.parametrize("tile", TILES)
def test_repeated_updates_give_the_same_bits(tile):
    g = gradient(16, 400, 300, "f32")
    first = run(g, 400, 300, "f32", tile=tile)
    for _ in range(3):
        assert np.array_equal(run(g, 400, 300, "f32", tile=tile), first)


def test_aligned_output_of_large_update():
    g = gradient(7, 600, 520, "f32")
    check(run(g, 600, 520, "f32", "bf16"), f64(g), "bf16")


def test_coefficients_of_each_step_and_scale():
    cs = [(3.2, -4.1, 1.9), MUON, (2.0, -1.5, 0.5)]
    g = gradient(8, 90, 150, "f32")
    got = run(g, 90, 150, "f32", steps=3, coefficients=cs, scale=0.2, eps=1e-3)
    check(got, f64(g), "f32", cs, 1e-3, 0.2)


def test_one_step():
    g = gradient(9, 40, 30, "bf16")
    check(run(g, 40, 30, "bf16", steps=1), f64(g), "f32", (MUON,))


@pytest.mark.parametrize("size", [1e-30, 1e-12, 1e12, 1e30])
def test_sizes_of_gradients(size):
    """The norm is summed in fp64: no square leaves its range.  A gradient far
    below eps stays small."""
    g = gradient(10, 60, 80, "f32", size=size)
    eps = EPS if size > 1e-20 else 0.0
    check(run(g, 60, 80, "f32", eps=eps), f64(g), "f32", eps=eps)
    if size < 1e-20:
        assert np.abs(run(g, 60, 80, "f32")).max() < 1e-18


def test_empty_and_bad_gradients():
    z = torch.zeros(48, 70, device="cuda")
    assert not run(z, 48, 70, "f32").any()
    z[3, 4] = float("nan")
    assert np.isnan(run(z, 48, 70, "f32")).any()


def test_one_entry():
    g = torch.zeros(30, 50, device="cuda")
    g[7, 9] = 3.0
    want = np.zeros((30, 50))
    t = 1.0
    for _ in range(5):
        t = MUON[0] * t + MUON[1] * t ** 3 + MUON[2] * t ** 5
    want[7, 9] = t
    got = run(g, 30, 50, "f32", eps=0.0)
    # three roundings a step of one number, each 2^-11, five steps whose maps are
    # no steeper than |a + 3 b t^2 + 5 c t^4| <= 3 near one
    assert np.count_nonzero(got) == 1 and abs(got[7, 9] - t) <= 0.1


def test_in_place():
    g = gradient(11, 100, 140, "bf16")
    want = run(g, 100, 140, "bf16", "bf16")
    skg.newton_schulz(g, g, rows=100, cols=140, dtype="bf16")
    torch.cuda.synchronize()
    assert np.array_equal(f64(g), want)


def test_captured_update_replays():
    rows, cols = 130, 190
    g = gradient(12, rows, cols, "f32")
    out = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    kw = dict(rows=rows, cols=cols, dtype="f32", dtype_out="bf16")
    ws = torch.empty(skg.skg_newton_schulz_workspace_bytes(skg.newton_schulz_args(g, out, **kw)), dtype=torch.uint8, device="cuda")
    skg.newton_schulz(g, out, workspace=ws, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        skg.newton_schulz(g, out, workspace=ws, **kw)
    for i in range(4):
        g.copy_(gradient(20 + i, rows, cols, "f32"))
        skg.newton_schulz(g, out, **kw)
        torch.cuda.synchronize()
        want = out.clone()
        out.fill_(float("nan"))
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
