"""Calls with more rows or tiles than one launch has room for (2^32 threads
along its axis): the rows around the seam, the first and the last ones."""

import pytest
import torch

import implicit_gemm_conv_dp_amd as skg

pytestmark = pytest.mark.gpu

WINDOW = 70


def windows(n, seam):
    return [(0, WINDOW), (seam - WINDOW, seam + WINDOW), (n - WINDOW, n)]


@pytest.fixture(autouse=True)
def empty_cache():
    yield
    torch.cuda.empty_cache()


def poisoned(shape, dtype):
    t = torch.empty(shape, dtype=dtype, device="cuda")
    t.view(torch.uint8).fill_(0xFF)
    return t


# 2^32 - 1 threads are 16777215 workgroups of 256, each of 32 rows of up to 64 columns.
SEAM = 16777215 * 32


@pytest.mark.parametrize("out", ["same", "row", "e4m3", "e2m1"])
def test_rows_of_the_norm(out):
    rows, cols = SEAM + 200, 32 if out in ("e4m3", "e2m1") else 1
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    # whole numbers 1 .. 97 by the row
    x.copy_((torch.arange(rows, device="cuda", dtype=torch.int32) % 97 + 1).to(torch.bfloat16).reshape(-1, 1).expand(-1, cols))
    kw = dict(rows=rows, cols=cols, dtype="bf16", eps=0.0)
    rstd = poisoned((rows,), torch.float32)
    if out == "same":
        y, h = poisoned((rows, cols), torch.bfloat16), poisoned((rows, cols), torch.bfloat16)
        skg.rmsnorm(x, y, rstd=rstd, h=h, residual=x, **kw)
        scale = None
    else:
        y = poisoned((rows, cols // 2 if out == "e2m1" else cols), torch.uint8)
        scale = poisoned((rows,), torch.float32) if out == "row" else poisoned((rows, 1), torch.uint8)
        skg.rmsnorm(x, y, rstd=rstd, y_scale=scale, dtype_y="e2m1" if out == "e2m1" else "e4m3",
                    scale_mode="rowcol" if out == "row" else "mx", **kw)
    torch.cuda.synchronize()
    for a, b in windows(rows, SEAM):
        v = x[a:b].float()
        if out == "same":
            v = 2 * v
            assert torch.equal(h[a:b].float(), v)
            assert (y[a:b] == 1).all()
        # |x| of every column: the factor is its reciprocal, y is 1
        assert torch.allclose(rstd[a:b], 1 / v[:, 0], rtol=2.0 ** -22, atol=0)
        if out == "row":
            assert torch.allclose(scale[a:b], torch.tensor(1 / 448, device="cuda"), rtol=2.0 ** -21, atol=0)
            assert (y[a:b] == 0x7E).all()
        elif out != "same":
            # the same rows alone
            y1, s1 = poisoned((b - a, y.shape[1]), torch.uint8), poisoned((b - a, 1), torch.uint8)
            skg.rmsnorm(x[a:b], y1, y_scale=s1, dtype_y=out, scale_mode="mx", **dict(kw, rows=b - a))
            torch.cuda.synchronize()
            assert torch.equal(y[a:b], y1) and torch.equal(scale[a:b], s1) and (s1 < 128).all()


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_tiles_of_the_transposed_quantiser(fmt):
    # 2^32 - 1 threads are 8388607 workgroups of 512, each of 128 columns.
    seam = 8388607 * 128
    cols = seam + 300
    x = torch.empty(1, cols, dtype=torch.bfloat16, device="cuda")
    x.copy_((torch.arange(cols, device="cuda", dtype=torch.int32) % 97 + 1).to(torch.bfloat16).reshape(1, -1))
    q = poisoned((cols, 16 if fmt == "e2m1" else 32), torch.uint8)
    s = poisoned((cols, 1), torch.uint8)
    kw = dict(dtype="bf16", dtype_q=fmt)
    skg.mx_quant(x, q, s, rows=1, cols=cols, transpose=True, **kw)
    torch.cuda.synchronize()
    for a, b in windows(cols, seam):
        # the same columns alone
        n = b - a
        q1, s1 = poisoned((n, q.shape[1]), torch.uint8), poisoned((n, 1), torch.uint8)
        skg.mx_quant(x[0, a:b].reshape(1, -1).contiguous(), q1, s1, rows=1, cols=n, transpose=True, **kw)
        torch.cuda.synchronize()
        assert torch.equal(q[a:b], q1) and torch.equal(s[a:b], s1) and (s1 < 140).all()
