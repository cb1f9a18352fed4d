"""An attention layer's input projection in 8-bit blocks of 128, forward, backward and
its weight's update.

    q, k, v = x W^T              8-bit product, a scale for each 128 of the inputs
    q, k    = norm of each head, turned by the token's position
    dx      = [dq dk dv] W       8-bit product
    dW      = [dq dk dv]^T x     8-bit product over the tokens, to fp32
    W      -= rate * (dW orthogonalised by Newton-Schulz products)

Activations and gradients have a scale for 1 x 128 elements and are quantised along
their rows and along the tokens from one read; the weight has one for 128 x 128, so its
codes for y serve dx transposed.

    python examples/projection_step.py [--tokens M] [--inputs K] [--heads H] [--kv-heads G] [--dim D]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import implicit_gemm_conv_dp_amd as skg  # noqa: E402

COEFFICIENTS = skg.NEWTON_SCHULZ_COEFFICIENTS


def up(n, m):
    return -(-n // m) * m


def quantise(x, block="1x128"):
    """((codes, scales) along the rows, the same along the columns) of a bf16 matrix
    from one read."""
    rows, cols = x.shape
    kq, kqt = up(cols, 128), up(rows, 128)
    tall = block == "128x128"
    q = torch.empty(rows, kq, dtype=torch.uint8, device=x.device)
    qt = torch.empty(cols, kqt, dtype=torch.uint8, device=x.device)
    s = torch.empty(kq // 128, kqt // 128 if tall else rows, device=x.device)
    st = torch.empty(kqt // 128, kq // 128 if tall else cols, device=x.device)
    skg.block_quant(x, q, s, qt, st, rows=rows, cols=cols, dtype="bf16", dtype_q="e4m3", block=block)
    return (q, s), (qt, st)


def product(a, b, mode, dtype="bf16"):
    """a b^T of two quantised matrices."""
    (aq, sa), (bq, sb) = a, b
    M, N, K = aq.shape[0], bq.shape[0], aq.shape[1]
    out = torch.empty(M, up(N, 8), device=aq.device,
                      dtype=torch.float32 if dtype == "f32" else torch.bfloat16)
    skg.gemm(aq, bq, out, sa, sb, M=M, N=N, K=K, ldc=out.shape[1], dtype_ab="e4m3", dtype_c=dtype,
             scale_mode=mode, tile="auto", mode="auto", reduction="auto", ctas=-1)
    return out[:, :N]


class Projection:
    """weight (H + 2 G) D x K in fp32, of which a bf16 copy is quantised; gains D in
    bf16; K and (H + 2 G) D are multiples of 8."""

    def __init__(self, weight, gain_q, gain_k, heads, kv_heads, cos, sin, eps=1e-6):
        self.weight, self.eps = weight, eps
        self.gains, self.heads, self.kv = (gain_q, gain_k), heads, kv_heads
        self.dim, self.cos, self.sin = gain_q.numel(), cos, sin
        self.codes()

    def codes(self):
        self.along_k, self.along_n = quantise(self.weight.bfloat16(), "128x128")

    def shape(self, tokens):
        t = (self.heads + 2 * self.kv) * self.dim
        strides = (tokens * t, t, self.dim)
        return dict(seq=tokens, heads_q=self.heads, heads_k=self.kv, head_dim=self.dim, dtype="bf16",
                    weight_q=self.gains[0], weight_k=self.gains[1], cos=self.cos, sin=self.sin,
                    table_rows=self.cos.shape[0], eps=self.eps, q_strides=strides, k_strides=strides)

    def parts(self, qkv):
        h, g, d = self.heads, self.kv, self.dim
        return qkv[:, :h * d], qkv[:, h * d:(h + g) * d], qkv[:, (h + g) * d:]

    def forward(self, x):
        rows = x.shape[0]
        along, self.x_tokens = quantise(x)
        self.qkv = product(along, self.along_k, "block128")
        q, k, v = self.parts(self.qkv)
        yq = torch.empty(rows, self.heads, self.dim, dtype=torch.bfloat16, device=x.device)
        yk = torch.empty(rows, self.kv, self.dim, dtype=torch.bfloat16, device=x.device)
        skg.qknorm_rope(q, k, yq, yk, **self.shape(rows))
        return yq, yk, v

    def backward(self, dyq, dyk, dv):
        """Gradients of x, the weight and the gains from those of the outputs."""
        rows = dyq.shape[0]
        d = torch.empty_like(self.qkv)
        dq, dk, _ = self.parts(d)
        self.parts(d)[2].copy_(dv)
        q, k, _ = self.parts(self.qkv)
        dgq, dgk = torch.empty(2, self.dim, device=d.device)
        kw = self.shape(rows)
        skg.qknorm_rope_bwd(dyq, dyk, q, k, dq, dk, dwq=dgq, dwk=dgk, yq_strides=kw["q_strides"],
                            yk_strides=kw["k_strides"], **kw)
        self.d = d
        along, tokens = quantise(d)
        dx = product(along, self.along_n, "block128")
        dw = product(tokens, self.x_tokens, "row128", "f32")
        return dx, dw, dgq, dgk

    def update(self, dw, rate):
        o = torch.empty(dw.shape, device=dw.device)
        rows, cols = dw.shape
        skg.newton_schulz(dw, o, rows=rows, cols=cols, dtype="f32", ldg=dw.stride(0),
                          scale=max(1.0, rows / cols) ** 0.5)
        self.weight.sub_(o, alpha=rate)
        self.codes()
        return o


def tables(positions, half, device):
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * 1e4 ** (-torch.arange(half) / half)
    return angle.cos().float().to(device), angle.sin().float().to(device)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=500)
    ap.add_argument("--inputs", type=int, default=1024)
    ap.add_argument("--heads", type=int, default=8)
    ap.add_argument("--kv-heads", type=int, default=2)
    ap.add_argument("--dim", type=int, default=128)
    a = ap.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale

    M, K, H, G, D = a.tokens, a.inputs, a.heads, a.kv_heads, a.dim
    N = (H + 2 * G) * D
    w = normal(N, K, scale=K ** -0.5).bfloat16().float()
    gq, gk = (1 + normal(D, scale=0.1)).bfloat16(), (1 + normal(D, scale=0.1)).bfloat16()
    cos, sin = tables(M, D // 2, "cuda")
    x = normal(M, K).bfloat16()
    dyq, dyk, dv = (normal(M, n, D).bfloat16() for n in (H, G, G))
    layer = Projection(w.clone(), gq, gk, H, G, cos, sin)
    yq, yk, v = layer.forward(x)
    dx, dw, dgq, dgk = layer.backward(dyq, dyk, dv.reshape(M, G * D))
    o = layer.update(dw, 0.02)

    # The same layer in fp32, by automatic differentiation.
    def head(t, n, gain):
        t = t.reshape(M, n, D)
        t = t * torch.rsqrt(t.square().mean(2, keepdim=True) + layer.eps) * gain
        p, q = t[..., :D // 2], t[..., D // 2:]
        c, s = cos[:, None], sin[:, None]
        return torch.cat((p * c - q * s, q * c + p * s), 2)

    xf, wf, qf, kf = (t.float().requires_grad_() for t in (x, w, gq, gk))
    q, k, vf = layer.parts(xf @ wf.t())
    yqf, ykf = head(q, H, qf), head(k, G, kf)
    torch.autograd.backward([yqf, ykf, vf], [dyq.float(), dyk.float(), dv.float().reshape(M, G * D)])
    errors = {}
    for name, got, want in (("q", yq, yqf), ("k", yk, ykf), ("v", v, vf), ("dx", dx, xf.grad),
                            ("dW", dw, wf.grad), ("dgain_q", dgq, qf.grad), ("dgain_k", dgk, kf.grad)):
        errors[name] = ((got.float() - want).norm() / want.norm()).item()
        print("%-8s relative error against fp32 %.4f" % (name, errors[name]))
    return errors, layer, dw, o


if __name__ == "__main__":
    main()
