"""GPU parity of the norms of heads with the rotation, and of their gradient,
against float64.

A head of up to 512 elements is summed in runs of eight and by a tree of six:
its mean square is within 16 units of 2^-24, the factor within 12, and the
normed element within 16; the turned one is within 20 of the sum of its two
products' magnitudes, for which DELTA = 2^-18 leaves room, and a rounding to the
heads' type adds half a step.  The gradient's terms likewise.  dw is a sum of
at most 64 heads a group in turn, of 32 groups and of 64 partial sums, each
addition off by 2^-24 of the sum of magnitudes: 2^-16 of it."""

import numpy as np
import pytest
import torch

import implicit_gemm_conv_dp_amd as skg
from oracle import projection as pj

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -149}
DELTA, SUM = 2.0 ** -18, 2.0 ** -16
EPS = 1e-6


def f64(t):
    return t.cpu().to(torch.float64).numpy()


class Case:
    def __init__(self, tokens, hq, hk, dim, rope, dtype, style="half", w32=True, weights=True, table=64, seed=0,
                 layout="packed", pos_type=torch.int32):
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.style, self.dim, self.tokens = dtype, style, dim, tokens
        x = torch.randn(tokens, hq + 2 * hk, dim, generator=g) * torch.exp(0.5 * torch.randn(dim, generator=g))
        if tokens > 1:
            x[1, :1] = 0                      # an empty head
            x[0] *= 2.0 ** -9
        x = x.to(T[dtype])
        heads = {"q": (0, hq), "k": (hq, hk)}
        self.x = {n: x[:, a:a + h] for n, (a, h) in heads.items()}
        self.dy = {n: (torch.randn(tokens, h, dim, generator=g) * 0.1).to(T[dtype]) for n, (_, h) in heads.items()}
        w = {n: 1 + 0.3 * torch.randn(dim, generator=g) for n in "qk"}
        self.w = {n: (w[n] if w32 else w[n].to(T[dtype])) if weights else None for n in "qk"}
        ang = torch.rand(table, max(rope // 2, 1), generator=g) * 6.28
        self.cos, self.sin = ang.cos()[:, :rope // 2].contiguous(), ang.sin()[:, :rope // 2].contiguous()
        self.pos = torch.randint(0, table, (tokens,), generator=g).to(pos_type)
        self.kw = dict(seq=tokens, heads_q=hq, heads_k=hk, head_dim=dim, rope_dim=rope, dtype=dtype,
                       dtype_w="f32" if w32 else dtype, style=style, eps=EPS, table_rows=table)
        d = {}
        if layout == "packed":                # slices of a projection's output
            buf = x.reshape(tokens, -1).cuda()
            pitch = buf.shape[1]
            d["q"], d["k"] = buf, buf[:, hq * dim:]
            self.strides = {n: (0, pitch, dim) for n in "qk"}
        else:                                 # head by head
            d = {n: self.x[n].transpose(0, 1).contiguous().cuda() for n in "qk"}
            self.strides = {n: (0, dim, tokens * dim) for n in "qk"}
        self.d = d
        self.kw.update(q_strides=self.strides["q"], k_strides=self.strides["k"])
        self.dev = dict(weight_q=None if not weights else self.w["q"].cuda(),
                        weight_k=None if not weights else self.w["k"].cuda(),
                        cos=self.cos.cuda(), sin=self.sin.cuda(), positions=self.pos.cuda())

    def tables(self):
        i = self.pos.long()
        return f64(self.cos[i]), f64(self.sin[i])

    def weight(self, n):
        return np.ones(self.dim) if self.w[n] is None else f64(self.w[n])

    def outputs(self):
        o = {}
        for n in "qk":
            o[n] = torch.empty(self.tokens, self.x[n].shape[1], self.dim, dtype=T[self.dtype], device="cuda")
            o[n].view(torch.uint8).fill_(0xFF)
        return o

    def check(self, y):
        c, s = self.tables()
        for n in "qk":
            v, _ = pj.head_norm(f64(self.x[n]), self.weight(n), EPS)
            want, size = pj.rotate(v, c, s, self.style), pj.turned_size(v, c, s, self.style)
            tol = DELTA * size + HALF[self.dtype] * (np.abs(want) + DELTA * size) + TINY[self.dtype]
            bad = ~(np.abs(f64(y[n]) - want) <= tol)
            assert not bad.any(), "%s: %d off, first %s" % (n, bad.sum(), np.argwhere(bad)[:3])

    def check_grad(self, dx, dw):
        c, s = self.tables()
        for n in "qk":
            want, wdw, size, wsize = pj.head_norm_bwd(f64(self.dy[n]), f64(self.x[n]), self.weight(n), EPS, c, s, self.style)
            if dx is not None:
                tol = DELTA * size + HALF[self.dtype] * (np.abs(want) + DELTA * size) + TINY[self.dtype]
                bad = ~(np.abs(f64(dx[n]) - want) <= tol)
                assert not bad.any(), "d%s: %d off, first %s" % (n, bad.sum(), np.argwhere(bad)[:3])
            if dw is not None:
                bad = ~(np.abs(f64(dw[n]) - wdw) <= SUM * wsize + 1e-30)
                assert not bad.any(), "dw%s: %d off, first %s" % (n, bad.sum(), np.argwhere(bad)[:3])


def forward(c, **kw):
    y = c.outputs()
    skg.qknorm_rope(c.d["q"], c.d["k"], y["q"], y["k"], **dict(c.kw, **c.dev, **kw))
    torch.cuda.synchronize()
    return y


def backward(c, want_dx=True, want_dw=True, **kw):
    dx, dw = c.outputs(), {n: torch.full((c.dim,), float("nan"), device="cuda") for n in "qk"}
    dy = {n: c.dy[n].cuda() for n in "qk"}
    skg.qknorm_rope_bwd(dy["q"], dy["k"], c.d["q"], c.d["k"], dx["q"] if want_dx else None, dx["k"] if want_dx else None,
                        dwq=dw["q"] if want_dw else None, dwk=dw["k"] if want_dw else None, **dict(c.kw, **c.dev, **kw))
    torch.cuda.synchronize()
    return dx, dw


DIMS = [(1, 0), (2, 2), (6, 4), (8, 8), (16, 12), (20, 20), (64, 64), (80, 20), (96, 48), (100, 50), (128, 128),
        (128, 32), (192, 128), (256, 256), (260, 130), (512, 512)]


@pytest.mark.parametrize("dim,rope", DIMS)
@pytest.mark.parametrize("style", ["half", "pairs"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_forward_and_backward(dim, rope, style, dtype):
    c = Case(37, 3, 2, dim, rope, dtype, style, w32=dim % 3 == 0, seed=dim + rope,
             layout="packed" if dim % 5 else "heads")
    c.check(forward(c))
    c.check_grad(*backward(c))


@pytest.mark.parametrize("tokens,hq,hk", [(1, 1, 1), (1, 32, 8), (3, 5, 0), (3, 0, 5), (700, 32, 8), (2500, 7, 7), (9, 1, 0)])
@pytest.mark.parametrize("layout", ["packed", "heads"])
def test_counts_of_tokens_and_heads(tokens, hq, hk, layout):
    c = Case(tokens, hq, hk, 128, 128, "bf16", seed=tokens, layout=layout)
    c.check(forward(c))
    c.check_grad(*backward(c))


def test_without_weights():
    c = Case(11, 4, 2, 64, 32, "f32", weights=False)
    c.check(forward(c))
    c.check_grad(*backward(c))


@pytest.mark.parametrize("pos_type", [torch.int32, torch.int64])
def test_positions_outside_the_table(pos_type):
    c = Case(8, 3, 2, 64, 32, "f32", pos_type=pos_type)
    good = c.pos.clone()
    for i, p in ((1, -1), (4, 64), (6, 2 ** 31 - 1)):
        c.pos[i] = p
    if pos_type == torch.int64:
        c.pos[7] = 1 << 32
    c.dev["positions"] = c.pos.cuda()
    bad = (c.pos != good).numpy()
    y = forward(c)
    dx, _ = backward(c)
    c.pos = good
    for n in "qk":
        assert torch.isnan(y[n][bad][..., :32]).all() and torch.isfinite(y[n][bad][..., 32:]).all()
        assert torch.isnan(dx[n][bad]).all() and torch.isfinite(dx[n][~bad]).all()
        y[n][bad] = torch.zeros((), device="cuda")
        keep = f64(y[n])
        cs, sn = c.tables()
        want = pj.rotate(pj.head_norm(f64(c.x[n]), c.weight(n), EPS)[0], cs, sn, "half")
        assert np.abs(keep - want)[~bad].max() < 1e-4


def test_positions_counted_from_an_offset():
    """Without positions: token t of each batch at pos0 + t; strided batches."""
    B, S, hq, hk, D = 3, 5, 4, 2, 64
    c = Case(B * S, hq, hk, D, D, "bf16", table=40)
    c.pos = (torch.arange(B * S) % S + 7).to(torch.int32)
    pitch = (hq + 2 * hk) * D
    wide = torch.full((B, S + 2, pitch), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :S] = c.d["q"].view(B, S, pitch)
    y = {n: torch.full((B, h, S, D), float("nan"), dtype=torch.bfloat16, device="cuda") for n, h in (("q", hq), ("k", hk))}
    st = ((S + 2) * pitch, pitch, D)
    kw = dict(c.kw, **c.dev, batch=B)
    kw.update(seq=S, positions=None, pos0=7, q_strides=st, k_strides=st, yq_strides=(hq * S * D, D, S * D),
              yk_strides=(hk * S * D, D, S * D))
    skg.qknorm_rope(wide, wide[:, :, hq * D:], y["q"], y["k"], **kw)
    torch.cuda.synchronize()
    c.check({n: y[n].transpose(1, 2).reshape(B * S, -1, D) for n in "qk"})


def test_in_place():
    c = Case(50, 6, 2, 128, 64, "bf16", seed=3)
    y = forward(c)
    buf = c.d["q"].clone()
    k = buf[:, 6 * 128:]
    kw = dict(c.kw, **c.dev)
    skg.qknorm_rope(buf, k, buf, k, yq_strides=c.strides["q"], yk_strides=c.strides["k"], **kw)
    torch.cuda.synchronize()
    got = buf.view(50, -1, 128)
    assert torch.equal(got[:, :6], y["q"]) and torch.equal(got[:, 6:8], y["k"])
    assert torch.equal(got[:, 8:], c.d["q"].view(50, -1, 128)[:, 8:])   # values: left as they were
    dx, dw = backward(c)
    dy = {n: c.dy[n].cuda() for n in "qk"}
    dwq, dwk = (torch.empty(128, device="cuda") for _ in range(2))
    skg.qknorm_rope_bwd(dy["q"], dy["k"], c.d["q"], c.d["k"], dy["q"], dy["k"], dwq=dwq, dwk=dwk, **kw)
    torch.cuda.synchronize()
    assert torch.equal(dy["q"], dx["q"]) and torch.equal(dy["k"], dx["k"])
    assert torch.equal(dwq, dw["q"]) and torch.equal(dwk, dw["k"])


def test_some_gradients_only():
    c = Case(90, 8, 2, 96, 96, "f32", seed=4)
    dx, dw = backward(c)
    _, dw2 = backward(c, want_dx=False)
    dx2, _ = backward(c, want_dw=False)
    for n in "qk":
        assert torch.equal(dw[n], dw2[n]) and torch.equal(dx[n], dx2[n])


def test_no_tokens_give_a_zero_gradient():
    c = Case(2, 4, 2, 64, 64, "bf16")
    c.kw["seq"] = 0
    _, dw = backward(c)
    assert not dw["q"].any() and not dw["k"].any()


def test_nan_and_infinity_stay_in_their_head():
    c = Case(6, 3, 2, 64, 64, "f32", layout="heads")
    c.d["q"][1, 2, 5] = float("nan")     # head 1 of token 2
    c.d["k"][0, 4, 9] = float("inf")
    y = forward(c)
    assert torch.isnan(y["q"][2, 1]).all() and torch.isnan(y["k"][4, 0]).any()
    y["q"][2, 1], y["k"][4, 0] = 0, 0
    assert torch.isfinite(y["q"]).all() and torch.isfinite(y["k"]).all()


def test_gradient_against_differences():
    """Along a direction: sum(dy y) moves by sum(dx d) + sum(dw e).  fp32 outputs are
    off by DELTA of their size at most, and the second difference's remainder is
    under h^2 times the third derivatives, 1e-4 here."""
    c = Case(5, 3, 2, 32, 16, "f32", "pairs", seed=9)
    dx, dw = backward(c)
    h = 2.0 ** -6
    g = torch.Generator().manual_seed(1)
    for n in "qk":
        d, e = torch.randn(c.x[n].shape, generator=g) * 0.1, torch.randn(32, generator=g) * 0.1
        cs, sn = c.tables()
        def f(t):
            v, _ = pj.head_norm(f64(c.x[n]) + t * f64(d), c.weight(n) + t * f64(e), EPS)
            return np.sum(f64(c.dy[n]) * pj.rotate(v, cs, sn, "pairs"))
        keep = np.ones(c.x[n].shape, bool)
        keep[0], keep[1, :1] = False, False   # tiny and empty heads bend too much
        d[~torch.from_numpy(keep)] = 0
        num = (f(h) - f(-h)) / (2 * h)
        ana = np.sum(f64(dx[n]) * f64(d)) + np.sum(f64(dw[n]) * f64(e))
        size = np.sum(np.abs(f64(dx[n]) * f64(d))) + np.sum(np.abs(f64(dw[n]) * f64(e)))
        assert abs(num - ana) <= 1e-3 * size, (n, num, ana)


def test_captured_backward_replays():
    c = Case(300, 8, 2, 128, 128, "bf16", seed=6)
    dy = {n: c.dy[n].cuda() for n in "qk"}
    dx, y = c.outputs(), c.outputs()
    dwq, dwk = (torch.empty(128, device="cuda") for _ in range(2))
    kw = dict(c.kw, **c.dev)
    args = skg.qknorm_rope_args(c.d["q"], c.d["k"], dx["q"], dx["k"], dy["q"], dy["k"], dwq=dwq, dwk=dwk, **kw)
    ws = torch.empty(skg.skg_qknorm_rope_bwd_workspace_bytes(args), dtype=torch.uint8, device="cuda")

    def step(workspace=None):
        skg.qknorm_rope(c.d["q"], c.d["k"], y["q"], y["k"], **kw)
        skg.qknorm_rope_bwd(dy["q"], dy["k"], c.d["q"], c.d["k"], dx["q"], dx["k"], workspace=workspace, dwq=dwq, dwk=dwk, **kw)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(ws)
    for i in range(4):
        c.d["q"].copy_(torch.randn(c.d["q"].shape, generator=torch.Generator().manual_seed(50 + i)).cuda())
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (y["q"], y["k"], dx["q"], dx["k"], dwq, dwk)]
        for t in (y["q"], y["k"], dx["q"], dx["k"], dwq, dwk):
            t.view(torch.uint8).fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip((y["q"], y["k"], dx["q"], dx["k"], dwq, dwk), want):
            assert torch.equal(a, b), i
