"""The operators of an 8-bit attention projection together: a step of the example, each
part against float64 from the codes that the step itself had, the whole against the
layer in fp32, and steps that are captured, replayed and run on several streams."""

import importlib.util
import os

import numpy as np
import pytest
import torch

import implicit_gemm_conv_dp_amd as skg
from oracle import projection as pj

from test_gpu_newton import check as check_update
from test_gpu_streams import freed_and_still_written

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "projection_step.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("projection_step", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def make(example, seed, tokens, K, H, G, D):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g) * scale).bfloat16().cuda()

    w = normal((H + 2 * G) * D, K, scale=K ** -0.5).float()
    cos, sin = example.tables(max(tokens, 1), D // 2, "cuda")
    layer = example.Projection(w, 1 + normal(D, scale=0.1), 1 + normal(D, scale=0.1), H, G, cos, sin)
    return layer, normal(tokens, K), normal(tokens, H, D), normal(tokens, G, D), normal(tokens, G * D)


@pytest.mark.parametrize("tokens", ["1", "77", "500"])
def test_step_against_fp32(example, tokens):
    e, _, _, _ = example.main(["--tokens", tokens, "--inputs", "512", "--heads", "4", "--kv-heads", "2", "--dim", "64"])
    # A code of e4m3 is off by at most 2^-4 of its value, so an operand by at most that
    # of its norm, and two operands' errors add in squares.  A norm's gradient takes q
    # twice over (its direction and its size); its own quantisation and the other
    # operand's come on top.
    one = 2.0 ** -4
    for name in ("q", "k", "v", "dgain_q", "dgain_k"):
        assert e[name] <= one * 2 ** 0.5, name
    for name in ("dx", "dW"):
        assert e[name] <= one * (2 * 4 + 2) ** 0.5, name


@pytest.mark.parametrize("tokens,K,H,G,D", [(77, 264, 3, 1, 64), (1, 128, 2, 2, 80), (300, 512, 4, 2, 128)])
def test_parts_of_a_step(example, tokens, K, H, G, D):
    layer, x, dyq, dyk, dv = make(example, tokens, tokens, K, H, G, D)
    yq, yk, v = layer.forward(x)
    dx, dw, dgq, dgk = layer.backward(dyq, dyk, dv)
    o = torch.empty(dw.shape, device="cuda")
    N = dw.shape[0]
    skg.newton_schulz(dw, o, rows=N, cols=K, dtype="f32", ldg=dw.stride(0))
    torch.cuda.synchronize()

    def back(codes, block="1x128"):
        q, s = codes
        return pj.block_values(s.cpu().numpy(), q.cpu().numpy(), "e4m3", block)

    def product(A, B, got, half):
        """The fp32 additions, the output's rounding, and what an 8-bit instruction
        drops: of its 128 products each by less than 2^-12 of the largest one."""
        want, size = A @ B.T, np.abs(A) @ np.abs(B).T
        blocks = A.shape[1] // 128
        a, b = (np.abs(t).reshape(t.shape[0], blocks, 128).max(2) for t in (A, B))
        drop = 128 * 2.0 ** -12 * (a @ b.T) if half == 2.0 ** -8 else 0
        tol = (A.shape[1] + 16) * 2.0 ** -23 * size + drop
        off = np.abs(f64(got) - want)
        assert np.all(off <= tol + half * (np.abs(want) + tol) + 2.0 ** -134)

    x_rows, w_k = example.quantise(x)[0], back(layer.along_k, "128x128")
    product(back(x_rows), w_k, layer.qkv, 2.0 ** -8)
    assert np.array_equal(w_k[:, :K], back(layer.along_n, "128x128")[:, :N].T)
    d_rows, d_tokens = example.quantise(layer.d)
    product(back(d_rows), back(layer.along_n, "128x128"), dx, 2.0 ** -8)
    product(back(d_tokens), back(layer.x_tokens), dw, 2.0 ** -24)
    # heads: some (D + 16) fp32 operations, and the rounding to bf16
    cos, sin = f64(layer.cos)[:tokens], f64(layer.sin)[:tokens]
    q, k, _ = layer.parts(f64(layer.qkv))
    dq, dk, dv_ = layer.parts(f64(layer.d))
    assert np.array_equal(dv_, f64(dv))
    for y, t, n, gain, dy, dt, dg in ((yq, q, H, layer.gains[0], dyq, dq, dgq), (yk, k, G, layer.gains[1], dyk, dk, dgk)):
        t, w = t.reshape(tokens, n, D), f64(gain)
        normed, _ = pj.head_norm(t, w, layer.eps)
        want, size = pj.rotate(normed, cos, sin, "half"), pj.turned_size(normed, cos, sin, "half")
        assert np.all(np.abs(f64(y) - want) <= 2.0 ** -8 * np.abs(want) + (D + 16) * 2.0 ** -24 * size)
        wdt, wdg, dsize, gsize = pj.head_norm_bwd(f64(dy), t, w, layer.eps, cos, sin, "half")
        assert np.all(np.abs(dt.reshape(tokens, n, D) - wdt) <= 2.0 ** -8 * np.abs(wdt) + (D + 16) * 2.0 ** -23 * dsize)
        assert np.all(np.abs(f64(dg) - wdg) <= (tokens * n + D + 16) * 2.0 ** -23 * gsize)
    check_update(f64(o), f64(dw), "f32")


def step(layer, x, dyq, dyk, dv):
    yq, yk, v = layer.forward(x)
    dx, dw, dgq, dgk = layer.backward(dyq, dyk, dv)
    o = layer.update(dw, 0.02)
    return [t.clone() for t in (yq, yk, v, dx, dw, dgq, dgk, o, layer.weight)]


def same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


def test_captured_steps(example):
    """Two captured steps of different sizes, replayed in turn with eager work between
    them: every replay against an eager step from the same weight."""
    made = [make(example, 5, 200, 384, 4, 2, 64), make(example, 6, 60, 640, 2, 1, 128)]
    graphs = []
    for layer, *io in made:
        w0 = layer.weight.clone()
        want = step(layer, *io)
        layer.weight.copy_(w0)
        layer.codes()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(layer, *io)
            layer.weight.copy_(w0)
            layer.codes()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer.weight.copy_(w0)
            layer.codes()
            got = step(layer, *io)
        graphs.append((g, got, want))
    junk = torch.empty(1 << 24, device="cuda")
    for _ in range(4):
        for g, got, want in graphs:
            for t in got:
                t.view(torch.uint8).fill_(0xFF)
            g.replay()
            junk.fill_(float("nan"))
            torch.cuda.synchronize()
            assert same(got, want)


def test_steps_on_two_streams(example):
    made = [make(example, 7, 150, 256, 2, 2, 128), make(example, 8, 90, 512, 4, 2, 64)]
    start = [m[0].weight.clone() for m in made]
    wants = []
    for (layer, *io), w0 in zip(made, start):
        wants.append(step(layer, *io))
        layer.weight.copy_(w0)
        layer.codes()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    gots = []
    for (layer, *io), s in zip(made, streams):
        with torch.cuda.stream(s):
            gots.append(step(layer, *io))
    torch.cuda.synchronize()
    assert all(same(g, w) for g, w in zip(gots, wants))


def test_workspaces_on_another_stream():
    """Memory that is freed on the current stream, where work still writes it, is not
    what a call on another stream takes for itself."""
    g = torch.Generator().manual_seed(9)
    rows, cols = 300, 700
    u = torch.randn(rows, cols, generator=g).cuda()
    o, o2 = (torch.empty(rows, cols, device="cuda") for _ in range(2))
    kw = dict(rows=rows, cols=cols, dtype="f32")
    skg.newton_schulz(u, o, **kw)
    T, H, G, D = 900, 8, 2, 128
    q, dq = (torch.randn(T, H, D, generator=g).cuda() for _ in range(2))
    k, dk = (torch.randn(T, G, D, generator=g).cuda() for _ in range(2))
    w = torch.randn(2, D, generator=g).cuda()
    hk = dict(seq=T, heads_q=H, heads_k=G, head_dim=D, rope_dim=0, dtype="f32", weight_q=w[0], weight_k=w[1])

    def heads(stream=None):
        outs = [torch.empty_like(t) for t in (q, k)] + [torch.empty(D, device="cuda") for _ in range(2)]
        torch.cuda.synchronize()
        return outs, lambda: skg.qknorm_rope_bwd(dq, dk, q, k, *outs[:2], dwq=outs[2], dwk=outs[3], stream=stream, **hk)

    want, call = heads()
    call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    need = skg.skg_newton_schulz_workspace_bytes(skg.newton_schulz_args(u, o, **kw))
    for _ in range(3):
        freed_and_still_written(need)
        skg.newton_schulz(u, o2, stream=side, **kw)
        side.synchronize()
        assert torch.equal(o2, o)
        torch.cuda.synchronize()
        got, call = heads(side)
        freed_and_still_written(2 << 20)
        call()
        side.synchronize()
        assert same(got, want)
        torch.cuda.synchronize()
