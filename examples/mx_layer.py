"""A pre-norm linear layer in MX 4-bit floating point, forward and backward.

    n  = norm(x + residual) * gain        quantised as it is written
    y  = n W^T                            4-bit product
    dn = dy W                             4-bit product
    dW = dy^T n                           4-bit product over the tokens
    dx, dgain = gradient of the norm      plus what the residual stream brings

The weight is quantised once along each axis that a product reduces over; the
gradient and the activations are quantised along the tokens for dW, padded to
the product's multiple of 128.

    python examples/mx_layer.py [--tokens M] [--inputs K] [--outputs N]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import implicit_gemm_conv_dp_amd as skg  # noqa: E402


def up(n, m):
    return -(-n // m) * m


def quantise(x, kq=None, transpose=False):
    """(codes, scales) of a bf16 matrix along its rows, or along its columns
    and transposed."""
    rows, cols = x.shape
    lines, axis = (cols, rows) if transpose else (rows, cols)
    kq = kq or up(axis, 128)
    q = torch.empty(lines, kq // 2, dtype=torch.uint8, device=x.device)
    s = torch.empty(lines, kq // 32, dtype=torch.uint8, device=x.device)
    skg.mx_quant(x, q, s, rows=rows, cols=cols, dtype="bf16", dtype_q="e2m1", kq=kq,
                 transpose=transpose)
    return q, s


def product(a, b, dtype="bf16"):
    """a b^T of two quantised matrices."""
    (aq, sa), (bq, sb) = a, b
    M, N, K = aq.shape[0], bq.shape[0], 2 * aq.shape[1]
    out = torch.empty(M, up(N, 8), device=aq.device,
                      dtype=torch.float32 if dtype == "f32" else torch.bfloat16)
    skg.gemm(aq, bq, out, sa, sb, M=M, N=N, K=K, ldc=out.shape[1], dtype_ab="e2m1", dtype_c=dtype,
             scale_mode="mx", tile="auto", mode="auto", reduction="auto", ctas=-1)
    return out[:, :N]


class Layer:
    """weight N x K and gain K in bf16; K and N are multiples of 128."""

    def __init__(self, weight, gain, eps=1e-5):
        self.gain, self.eps = gain, eps
        self.along_k = quantise(weight)                 # for y
        self.along_n = quantise(weight, transpose=True)  # for dn

    def forward(self, x, residual):
        rows, cols = x.shape
        self.h = torch.empty_like(x)
        self.rstd = torch.empty(rows, device=x.device)
        q = torch.empty(rows, cols // 2, dtype=torch.uint8, device=x.device)
        s = torch.empty(rows, cols // 32, dtype=torch.uint8, device=x.device)
        skg.rmsnorm(x, q, rows=rows, cols=cols, dtype="bf16", weight=self.gain, residual=residual,
                    h=self.h, rstd=self.rstd, y_scale=s, dtype_y="e2m1", scale_mode="mx",
                    eps=self.eps)
        self.n = q, s
        return product(self.n, self.along_k), self.h

    def backward(self, dy, dh):
        """Gradients of x (and of the residual alike), the weight and the gain,
        from those of y and of the residual stream."""
        rows, cols = self.h.shape
        dn = product(quantise(dy), self.along_n)
        n = torch.empty(rows, cols, dtype=torch.bfloat16, device=dy.device)
        skg.mx_dequant(*self.n, n, rows=rows, cols=cols, dtype="bf16", dtype_q="e2m1")
        dw = product(quantise(dy, transpose=True), quantise(n, transpose=True), "f32")
        dx = torch.empty_like(self.h)
        dgain = torch.empty(cols, device=dy.device)
        skg.rmsnorm_bwd(dn, self.h, self.rstd, dx, rows=rows, cols=cols, dtype="bf16",
                        weight=self.gain, dres=dh, dw=dgain)
        return dx, dw, dgain


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=500)
    ap.add_argument("--inputs", type=int, default=1024)
    ap.add_argument("--outputs", type=int, default=2048)
    a = ap.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()

    M, K, N = a.tokens, a.inputs, a.outputs
    w, gain = normal(N, K, scale=K ** -0.5), 1 + normal(K, scale=0.1)
    x, r, dy, dh = normal(M, K), normal(M, K), normal(M, N), normal(M, K)
    layer = Layer(w, gain)
    y, h = layer.forward(x, r)
    dx, dw, dgain = layer.backward(dy, dh)

    # The same layer in fp32, by automatic differentiation.
    xf, wf, gf = x.float().requires_grad_(), w.float().requires_grad_(), gain.float().requires_grad_()
    hf = xf + r.float()
    nf = hf * torch.rsqrt(hf.square().mean(1, keepdim=True) + layer.eps) * gf
    yf = nf @ wf.t()
    torch.autograd.backward([yf, hf], [dy.float(), dh.float()])
    errors = {}
    for name, got, want in (("y", y, yf), ("h", h, hf), ("dx", dx, xf.grad), ("dW", dw, wf.grad),
                            ("dgain", dgain, gf.grad)):
        errors[name] = ((got.float() - want).norm() / want.norm()).item()
        print("%-6s relative error against fp32 %.4f" % (name, errors[name]))
    return errors


if __name__ == "__main__":
    main()
