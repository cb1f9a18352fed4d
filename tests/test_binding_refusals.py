"""The binding's calls give the library's refusals, with their reasons, where
no GPU is there to ask for a stream."""

import pytest
import torch

import implicit_gemm_conv_dp_amd as skg

from test_lowp_host import P, refused

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the machine has a GPU")


class Placed:
    device = "cuda:0"

    def data_ptr(self):
        return 0x10000


@no_gpu
@pytest.mark.parametrize("call,word", [
    (lambda: skg.gemm(P, P, Placed(), M=8, N=8, K=100, dtype_ab="bf16", dtype_c="bf16", tile="128x128x32",
                      mode="dp", reduction="linear", ctas=1), "16 bytes"),
    (lambda: skg.gemm(P, P, Placed(), P, P, M=8, N=8, K=100, dtype_ab="e2m1", dtype_c="bf16", scale_mode="mx",
                      tile="auto", mode="auto", reduction="auto", ctas=1), "multiple of 128"),
    (lambda: skg.rmsnorm(P, P, rows=1, cols=0, dtype="bf16"), "cols"),
    (lambda: skg.rmsnorm_bwd(P, P, P, P, rows=1, cols=0, dtype="bf16", dw=Placed()), "cols"),
    (lambda: skg.rmsnorm_bwd(P, P, P, P, rows=1, cols=0, dtype="bf16", dw=Placed(), workspace=torch.empty(4)), "cols"),
    (lambda: skg.mx_quant(P, P, P, rows=-1, cols=32, dtype="bf16", dtype_q="e2m1"), "negative"),
    (lambda: skg.mx_dequant(P, P, P, rows=-1, cols=32, dtype="bf16", dtype_q="e2m1"), "negative"),
])
def test_refusals_without_a_gpu(call, word):
    refused(call, word)
