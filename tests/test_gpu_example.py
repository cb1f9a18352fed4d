"""The example of a 4-bit layer: its products against float64 products of the
same codes, and the whole against the layer in fp32 within what rounding to
e2m1 does."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import lowp

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mx_layer.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("mx_layer", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("tokens", ["1", "77", "500"])
def test_layer_against_fp32(example, tokens):
    e = example.main(["--tokens", tokens, "--inputs", "512", "--outputs", "768"])
    # An e2m1 block rounds to steps of 1/4 to 1/2 of its binade, uniformly in
    # effect: an operand of normal values is off by 0.115 of its norm or so,
    # at most 0.15; two operands' errors add in squares, and dW's activations
    # are rounded twice.
    assert e["h"] <= 2.0 ** -8
    assert e["y"] <= 0.15 * 2 ** 0.5 and e["dW"] <= 0.15 * 3 ** 0.5
    assert e["dx"] <= 0.15 * 2 ** 0.5 and e["dgain"] <= 0.15 * 3 ** 0.5


def test_products_of_the_same_codes(example):
    torch.manual_seed(1)
    M, N, K = 77, 256, 384
    w, gain = torch.randn(N, K).bfloat16().cuda(), torch.randn(K).bfloat16().cuda()
    x, r, dy = (torch.randn(M, n).bfloat16().cuda() for n in (K, K, N))
    layer = example.Layer(w, gain)
    y, _ = layer.forward(x, r)
    dx, dw, dgain = layer.backward(dy, torch.zeros_like(x))
    torch.cuda.synchronize()

    def back(q, s):
        return lowp.mx_values(s.cpu().numpy(), lowp.unpack(q.cpu().numpy()), "e2m1")

    A, B = back(*layer.n), back(*layer.along_k)
    tol = K * 2.0 ** -23 * (np.abs(A) @ np.abs(B).T)
    want = A @ B.T
    assert np.all(np.abs(y.double().cpu().numpy() - want) <= tol + 2.0 ** -8 * np.abs(want) * 1.01)
    # along the tokens: padded to a multiple of 128, and the padding is zero
    qd, sd = example.quantise(dy, transpose=True)
    D = back(qd, sd)
    assert D.shape == (N, 128) and not D[:, M:].any()
    s, q = lowp.mx_quantize(np.pad(A[:M].T, ((0, 0), (0, 128 - M))), "e2m1")
    E = lowp.mx_values(s, q, "e2m1")
    want = D @ E.T
    assert np.all(np.abs(dw.double().cpu().numpy() - want) <= 128 * 2.0 ** -23 * (np.abs(D) @ np.abs(E).T))
