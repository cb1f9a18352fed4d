"""Calls on a stream of the caller's, while work that still uses freed memory
waits on torch's current one: what a call allocates for itself is not that
memory."""

import pytest
import torch

import implicit_gemm_conv_dp_amd as skg

from test_gpu_norm import EPS, T, out, rows_of

pytestmark = pytest.mark.gpu


def freed_and_still_written(nbytes):
    """Work on the current stream that writes `nbytes` bytes after some
    milliseconds; the tensor is freed at once."""
    buf = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    torch.cuda._sleep(20_000_000)
    for _ in range(50):
        buf.fill_(0x7F)


def test_gradient_on_another_stream():
    rows, cols = 3001, 1032   # over the size that takes no workspace
    h, dy, dres = (rows_of(s, rows, cols, "bf16") for s in (40, 41, 42))
    rstd = torch.rsqrt(h.double().square().mean(1) + EPS).float()
    kw = dict(rows=rows, cols=cols, dtype="bf16", dres=dres)
    dx, dw = out((rows, cols), T["bf16"]), out((cols,), torch.float32)
    skg.rmsnorm_bwd(dy, h, rstd, dx, dw=dw, **kw)
    need = skg.skg_rmsnorm_bwd_workspace_bytes(skg.rmsnorm_bwd_args(dy, h, rstd, dx, dw=dw, **kw))
    assert need > 0
    dx2, dw2 = out((rows, cols), T["bf16"]), out((cols,), torch.float32)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(4):
        freed_and_still_written(need)
        skg.rmsnorm_bwd(dy, h, rstd, dx2, dw=dw2, stream=side, **kw)
        side.synchronize()
        assert torch.equal(dx2, dx) and torch.equal(dw2, dw)
        torch.cuda.synchronize()


@pytest.mark.parametrize("dtype_ab,tile,scale_mode", [("bf16", "128x128x64", "rowcol"),
                                                      ("e2m1", "128x128x256", "mx")])
def test_product_on_another_stream(dtype_ab, tile, scale_mode):
    """A stream-K plan: flags and partial tiles in a workspace."""
    M, N, K = 700, 648, 2048
    g = torch.Generator().manual_seed(43)
    if dtype_ab == "bf16":
        a, b = (torch.randn(n, K, generator=g).to(torch.bfloat16).cuda() for n in (M, N))
        scales = ()
    else:
        a, b = (torch.randint(0, 256, (n, K // 2), generator=g, dtype=torch.uint8).cuda() for n in (M, N))
        scales = tuple(torch.randint(120, 134, (n, K // 32), generator=g, dtype=torch.uint8).cuda() for n in (M, N))
    kw = dict(M=M, N=N, K=K, dtype_ab=dtype_ab, dtype_c="f32", tile=tile, scale_mode=scale_mode,
              mode="dp_sk", reduction="tree", ctas=16)
    c, c2 = out((M, N), torch.float32), out((M, N), torch.float32)
    plan = skg.gemm(a, b, c, *scales, **kw)
    assert plan["workspace_bytes"] > 0 and plan["sk_ctas"] > 0
    torch.cuda.synchronize()
    assert torch.isfinite(c).all()
    side = torch.cuda.Stream()
    for _ in range(4):
        freed_and_still_written(plan["workspace_bytes"])
        skg.gemm(a, b, c2, *scales, stream=side, **kw)
        side.synchronize()
        assert torch.equal(c2, c)
        torch.cuda.synchronize()
