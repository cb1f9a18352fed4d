"""The operators of an 8-bit attention projection on tensors of more than 2^31 elements:
what lies at their ends, against float64."""

import numpy as np
import pytest
import torch

import implicit_gemm_conv_dp_amd as skg
from oracle import codecs, projection as pj

from test_gpu_block import check_codes
from test_gpu_newton import EPS, MUON

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def f64(t):
    return t.cpu().to(torch.float64).numpy()


@pytest.mark.parametrize("tile", ["64x64x128", "128x128x128", "256x128x128", "auto"])
def test_product(tile):
    M, N, K = 70001, 32760, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    a, b = (torch.randint(0, 64, (n, K), generator=g, device="cuda").to(torch.uint8) for n in (M, N))
    sa, sb = torch.ones(1, M, device="cuda"), torch.ones(1, -(-N // 128), device="cuda")
    c = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    assert c.numel() > 1 << 31
    skg.gemm(a, b, c, sa, sb, M=M, N=N, K=K, dtype_ab="e4m3", dtype_c="bf16", scale_mode="block128", tile=tile,
             mode="auto", reduction="auto", ctas=-1)
    torch.cuda.synchronize()
    rows = [0, 1, 65537, M - 130, M - 2, M - 1]
    A, B = codecs.decode("e4m3", a[rows].cpu().numpy()), codecs.decode("e4m3", b.cpu().numpy())
    want, size = A @ B.T, np.abs(A) @ np.abs(B).T
    # 128 products of one sign: at most 2^-12 of the largest dropped of each
    drop = 128 * 2.0 ** -12 * np.abs(A).max(1)[:, None] * np.abs(B).max(1)
    assert np.all(np.abs(f64(c[rows]) - want) <= drop + 2.0 ** -8 * (want + drop) + (K + 16) * 2.0 ** -23 * size)
    assert not torch.isnan(c[::4096].float()).any() and not torch.isnan(c[:, -1].float()).any()


@pytest.mark.parametrize("block", ["1x128", "128x128"])
def test_quantisation(block):
    rows, cols = 33001, 65544
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.bfloat16)
    assert x.numel() > 1 << 31
    kq, kqt = pj.up(cols, 128), pj.up(rows, 128)
    tall = block == "128x128"
    q = torch.empty(rows, kq, dtype=torch.uint8, device="cuda")
    qt = torch.empty(cols, kqt, dtype=torch.uint8, device="cuda")
    s = torch.empty(kq // 128, kqt // 128 if tall else rows, device="cuda")
    st = torch.empty(kqt // 128, kq // 128 if tall else cols, device="cuda")
    skg.block_quant(x, q, s, qt, st, rows=rows, cols=cols, dtype="bf16", dtype_q="e4m3", block=block)
    torch.cuda.synchronize()
    at = rows // 128 * 128  # the last block of rows, and of columns
    check_codes((s[:, at // 128 if tall else at:].cpu().numpy(), q[at:].cpu().numpy()), f64(x[at:]), "e4m3", block,
                "bf16", "rows")
    at = cols // 128 * 128
    check_codes((st[:, at // 128 if tall else at:].cpu().numpy(), qt[at:].cpu().numpy()), f64(x[:, at:]).T, "e4m3",
                block, "bf16", "columns")


def test_heads_and_their_gradient():
    T, H, G, D, pitch = 120003, 3, 1, 128, 20000
    g = torch.Generator(device="cuda").manual_seed(3)
    def buffer():
        return torch.empty(T, pitch, dtype=torch.bfloat16, device="cuda")
    x, y, dy = buffer(), buffer(), buffer()
    assert x.numel() > 1 << 31
    n = (H + G) * D
    x[:, :n].normal_(generator=g)
    dy[:, :n].normal_(generator=g)
    y[:, n] = 7
    angle = torch.rand(T, D // 2, generator=g, device="cuda", dtype=torch.float64) * 6
    cos, sin = angle.cos().float(), angle.sin().float()
    w = (torch.rand(2, D, generator=g, device="cuda") + 0.5).bfloat16()
    st = (T * pitch, pitch, D)
    kw = dict(seq=T, heads_q=H, heads_k=G, head_dim=D, dtype="bf16", weight_q=w[0], weight_k=w[1], cos=cos, sin=sin,
              table_rows=T, q_strides=st, k_strides=st, yq_strides=st, yk_strides=st)
    skg.qknorm_rope(x, x[:, H * D:], y, y[:, H * D:], **kw)
    torch.cuda.synchronize()
    ends = [0, 1, T // 2, T - 2, T - 1]
    c, s, wf = f64(cos[ends]), f64(sin[ends]), f64(w)
    weights = np.repeat(wf, [H, G], axis=0)
    X, DY = (f64(t[ends, :n]).reshape(len(ends), H + G, D) for t in (x, dy))
    normed, _ = pj.head_norm(X, weights, 1e-6)
    want, size = pj.rotate(normed, c, s, "half"), pj.turned_size(normed, c, s, "half")
    got = f64(y[ends, :n]).reshape(want.shape)
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + (D + 16) * 2.0 ** -24 * size)
    assert (y[:, n] == 7).all()
    skg.qknorm_rope_bwd(dy, dy[:, H * D:], x, x[:, H * D:], y, y[:, H * D:], dyq_strides=st, dyk_strides=st, **kw)
    torch.cuda.synchronize()
    want, _, size, _ = pj.head_norm_bwd(DY, X, weights, 1e-6, c, s, "half")
    got = f64(y[ends, :n]).reshape(want.shape)
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + (D + 16) * 2.0 ** -23 * size)
    assert (y[:, n] == 7).all()


@pytest.mark.parametrize("tall", [True, False])
def test_update(tall):
    """G M, M of the polynomials of G^T G alone: 130 columns, in float64."""
    rows, cols = 4000000, 130
    g = torch.Generator(device="cuda").manual_seed(4)
    u = torch.randn(rows, cols, generator=g, device="cuda")
    a = u if tall else u.t().contiguous()
    o = torch.empty(a.shape, dtype=torch.bfloat16, device="cuda")
    skg.newton_schulz(a, o, rows=a.shape[0], cols=a.shape[1], dtype="f32", dtype_out="bf16", eps=EPS)
    torch.cuda.synchronize()
    ws = skg.skg_newton_schulz_workspace_bytes(skg.newton_schulz_args(a, o, rows=a.shape[0], cols=a.shape[1], dtype="f32"))
    assert ws > 4 * rows * cols * 2 and rows * 192 * 2 * 2 > 1 << 31
    gram = np.zeros((cols, cols))
    for i in range(0, rows, 500000):
        part = u[i:i + 500000].double()
        gram += f64(part.t() @ part)
    norm = np.sqrt(np.trace(gram)) + EPS
    M, S = np.eye(cols) / norm, gram / norm ** 2
    for a_, b, c in (MUON,) * 5:
        Q = a_ * np.eye(cols) + b * S + c * S @ S
        M, S = M @ Q, Q @ S @ Q
    for at in (slice(0, 500), slice(rows // 2, rows // 2 + 500), slice(rows - 500, rows)):
        want = f64(u[at]) @ M
        got = f64(o[at]) if tall else f64(o[:, at]).T
        # X, S and P are kept in fp16: 3 roundings of 2^-11 a step.  On a matrix this
        # tall all singular values are alike, so a step scales them and their errors
        # alike; the output is rounded to bf16.
        assert np.linalg.norm(got - want) <= (15 * 2.0 ** -11 + 2.0 ** -8) * np.linalg.norm(want)
