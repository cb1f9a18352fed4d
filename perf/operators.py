"""What is measured of the low-precision layer operators: the root-mean-square
norm with the residual's addition and its gradient, microscaled (MX)
quantisation and reading back, and the product of MX 4-bit operands.

``run`` computes an operator in elementary torch operations, or, where ``own``
is set, through the framework's entry points.
"""

import math

import torch

own = False

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
EMAX = {"e2m1": 2, "e4m3": 8}


def listed():
    return [
        # One token of a decode step: the layer's input norm, codes and a row
        # scale for the 8-bit product that follows.
        dict(name="norm 1x4096 e4m3 row", op="norm", rows=1, cols=4096, dtype="bf16", out="e4m3",
             scales="row", residual=True, w32=False, pad=0),
        # A small serving batch on a slice of a wider buffer (row pitch over
        # the width), odd rows, MX 8-bit codes.
        dict(name="norm 37x5120 e4m3 mx", op="norm", rows=37, cols=5120, dtype="f16", out="e4m3",
             scales="mx", residual=True, w32=True, pad=24),
        # A training step's norm: the output stays in 16 bits, the rows'
        # factors are kept for the gradient.
        dict(name="norm 4864x4096 bf16", op="norm", rows=4864, cols=4096, dtype="bf16", out="same",
             scales="none", residual=True, w32=False, pad=0),
        # A long prompt: the largest norm.
        dict(name="norm 8192x8192 e4m3 row", op="norm", rows=8192, cols=8192, dtype="bf16",
             out="e4m3", scales="row", residual=True, w32=False, pad=0),
        # The norm's gradient on a short odd batch of an odd width, 32-bit.
        dict(name="norm grad 509x1111 f32", op="norm_grad", rows=509, cols=1111, dtype="f32",
             residual=True, w32=True),
        # The norm's gradient in a training step, with the gradient that the
        # residual stream brings from above.
        dict(name="norm grad 16384x4096", op="norm_grad", rows=16384, cols=4096, dtype="bf16",
             residual=True, w32=True),
        # A few tokens to 4-bit codes and back.
        dict(name="quant 61x4096 e2m1", op="quant", rows=61, cols=4096, dtype="f16", fmt="e2m1",
             transpose=False, pad=8),
        # A weight or a batch of activations to 4-bit codes and back.
        dict(name="quant 8192x8192 e2m1", op="quant", rows=8192, cols=8192, dtype="bf16",
             fmt="e2m1", transpose=False, pad=0),
        # Gradients to 8-bit codes along the other axis, as the weight's
        # gradient product reads them.
        dict(name="quant T 16384x4096 e4m3", op="quant", rows=16384, cols=4096, dtype="bf16",
             fmt="e4m3", transpose=True, pad=0),
        # One token through a 4-bit layer: its activations are quantised, then
        # multiplied.
        dict(name="product 1x8192x8192", op="product", M=1, N=8192, K=8192, dtype="bf16",
             act="bf16"),
        # A serving batch over an odd number of outputs.
        dict(name="product 48x4863x4096", op="product", M=48, N=4863, K=4096, dtype="f16",
             act="codes"),
        # A prompt or training step through a 4-bit layer: the largest product.
        dict(name="product 8192x8192x8192", op="product", M=8192, N=8192, K=8192, dtype="bf16",
             act="codes"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "quant", "product"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "product":
        M, N = _log(rng, 1, 8192), _log(rng, 64, 8192)
        K = 128 * _log(rng, 1, 64)
        return dict(op=op, M=M, N=N, K=K, dtype=dtype, act=rng.choice(["codes", "codes", "bf16"]))
    cols = _log(rng, 32, 16384)
    rows = _log(rng, 1, min(16384, (1 << 26) // cols))
    if op == "norm_grad":
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, residual=rng.random() < 0.7,
                    w32=rng.random() < 0.5)
    if op == "norm":
        out, scales = rng.choice([("same", "none"), ("e4m3", "row"), ("e4m3", "mx"), ("e2m1", "mx")])
        if scales == "mx":
            cols = -(-cols // 32) * 32
        rows = min(rows, (1 << 26) // cols)
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, out=out, scales=scales,
                    residual=rng.random() < 0.7, w32=rng.random() < 0.5,
                    pad=rng.choice([0, 0, 8, 24, 3]))
    transpose = rng.random() < 0.4
    if transpose:
        rows = -(-rows // 32) * 32
    else:
        cols = -(-cols // 32) * 32
    rows = max(32 if transpose else 1, min(rows, (1 << 26) // cols // 32 * 32))
    return dict(op=op, rows=rows, cols=cols, dtype=dtype, fmt=rng.choice(["e2m1", "e4m3"]),
                transpose=transpose, pad=rng.choice([0, 0, 8, 24, 3]))


def work(case):
    if case["op"] == "product":
        M, N, K = case["M"], case["N"], case["K"]
        a = M * K * (0.5 + 1 / 32) if case["act"] == "codes" else 2 * M * K
        return {"bytes": a + N * K * (0.5 + 1 / 32) + M * N * SIZE[case["dtype"]],
                "flops": 2.0 * M * N * K}
    n, size = case["rows"] * case["cols"], SIZE[case["dtype"]]
    wsize = 4 if case.get("w32") else size
    if case["op"] == "norm":
        out = {"same": size, "e4m3": 1.0, "e2m1": 2.0}[case["out"]] + (1 / 32 if case["scales"] == "mx" else 0)
        scale = 8 if case["scales"] == "row" else 4
        return {"bytes": n * (size * (3 if case["residual"] else 1) + out) + case["rows"] * scale
                + case["cols"] * wsize, "flops": 6.0 * n}
    if case["op"] == "norm_grad":
        return {"bytes": n * size * (4 if case["residual"] else 3) + case["rows"] * 4
                + case["cols"] * (wsize + 4), "flops": 9.0 * n}
    out = 1.0 if case["fmt"] == "e4m3" else 2.0
    return {"bytes": n * (size + out + 1 / 32), "flops": 3.0 * n}


# --- inputs ----------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _activations(g, rows, cols, dtype, pad=0):
    """Normal values with some channels larger than others and every 64th
    token empty (padding), in rows of cols + pad values."""
    x = torch.randn(rows, cols + pad, generator=g, device="cuda")
    x *= torch.exp(0.7 * torch.randn(cols + pad, generator=g, device="cuda"))
    x[37::64] = 0
    return x.to(TYPES[dtype])[:, :cols]


def _weight(g, cols, case):
    w = 1 + 0.2 * torch.randn(cols, generator=g, device="cuda")
    return w if case["w32"] else w.to(TYPES[case["dtype"]])


def _mx_operand(g, rows, K):
    """Packed e2m1 codes and E8M0 scales of normal values."""
    q = torch.empty(rows, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(rows, K // 32, dtype=torch.uint8, device="cuda")
    for r0 in range(0, rows, 2048):
        x = torch.randn(min(2048, rows - r0), K, generator=g, device="cuda")
        code, v = _mx_plain(x, "e2m1")
        mag = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
        c = torch.bucketize(v.abs(), mag).to(torch.uint8) | (torch.signbit(x).to(torch.uint8) << 3)
        q[r0:r0 + x.shape[0]] = c[:, 0::2] | (c[:, 1::2] << 4)
        s[r0:r0 + x.shape[0]] = code
    return q, s


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    s = {"case": c}
    op = c["op"]
    if op == "product":
        M, N, K = c["M"], c["N"], c["K"]
        s["w"], s["ws"] = _mx_operand(g, N, K)
        if c["act"] == "codes":
            s["a"], s["as"] = _mx_operand(g, M, K)
        else:
            s["x"] = _activations(g, M, K, "bf16")
            s["a"] = torch.empty(M, K // 2, dtype=torch.uint8, device="cuda")
            s["as"] = torch.empty(M, K // 32, dtype=torch.uint8, device="cuda")
        s["ldc"] = -(-N // 8) * 8
        s["c"] = torch.empty(M, s["ldc"], dtype=TYPES[c["dtype"]], device="cuda")
        return s
    rows, cols, dtype = c["rows"], c["cols"], TYPES[c["dtype"]]
    if op == "norm":
        s["x"] = _activations(g, rows, cols, c["dtype"], c["pad"])
        s["r"] = _activations(g, rows, cols, c["dtype"]) if c["residual"] else None
        s["w"] = _weight(g, cols, c)
        s["h"] = torch.empty(rows, cols, dtype=dtype, device="cuda") if c["residual"] else None
        s["rstd"] = torch.empty(rows, device="cuda")
        if c["out"] == "same":
            s["y"], s["scale"] = torch.empty(rows, cols, dtype=dtype, device="cuda"), None
        else:
            n = cols if c["out"] == "e4m3" else cols // 2
            s["y"] = torch.empty(rows, n, dtype=torch.uint8, device="cuda")
            s["scale"] = (torch.empty(rows, device="cuda") if c["scales"] == "row" else
                          torch.empty(rows, cols // 32, dtype=torch.uint8, device="cuda"))
            if c["out"] == "e2m1":
                s["values"] = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    elif op == "norm_grad":
        s["h"] = _activations(g, rows, cols, c["dtype"])
        s["w"] = _weight(g, cols, c)
        s["dy"] = (torch.randn(rows, cols, generator=g, device="cuda") * 0.1).to(dtype)
        s["dres"] = ((torch.randn(rows, cols, generator=g, device="cuda") * 0.1).to(dtype)
                     if c["residual"] else None)
        s["rstd"] = torch.rsqrt(s["h"].double().square().mean(1) + EPS).float()
        s["dx"] = torch.empty(rows, cols, dtype=dtype, device="cuda")
        s["dw"] = torch.empty(cols, device="cuda")
    else:
        s["x"] = _activations(g, rows, cols, c["dtype"], c["pad"])
        R, C = (cols, rows) if c["transpose"] else (rows, cols)
        s["q"] = torch.empty(R, C if c["fmt"] == "e4m3" else C // 2, dtype=torch.uint8, device="cuda")
        s["scale"] = torch.empty(R, C // 32, dtype=torch.uint8, device="cuda")
        if c["fmt"] == "e2m1":
            s["values"] = torch.empty(R, C, dtype=torch.bfloat16, device="cuda")
    return s


# --- the plain forms ---------------------------------------------------------

def _power(code):
    """2^(code - 127) of E8M0 codes below 255, in 32 bits."""
    code = code.to(torch.int32)
    return torch.where(code > 0, code << 23, 0x400000).view(torch.float32)


def _mx_plain(x, fmt):
    """E8M0 codes of the blocks of 32 of x's rows, and the elements' values
    (in units of the block's scale) in 32 bits."""
    rows, cols = x.shape
    b = x.float().reshape(rows, cols // 32, 32)
    top = b.abs().amax(2)
    code = (((top.view(torch.int32) >> 23) & 255) - EMAX[fmt]).clamp(min=0)
    v = b / _power(code).unsqueeze(2)
    if fmt == "e4m3":
        v = v.clamp(-448, 448).to(torch.float8_e4m3fn).float()
    else:
        a = v.abs()
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        v = torch.copysign((torch.round(a / step) * step).clamp(max=6), v)
    return code.to(torch.uint8), v.reshape(rows, cols)


def _mx_outputs(x, fmt):
    code, v = _mx_plain(x, fmt)
    scale = code.view(torch.float8_e8m0fnu)
    if fmt == "e4m3":
        return {"scale": scale, "codes": v.to(torch.float8_e4m3fn)}
    v = v.reshape(x.shape[0], -1, 32) * _power(code).unsqueeze(2)
    return {"scale": scale, "values": v.reshape(x.shape).to(torch.bfloat16)}


def _unpack(q, scale, dtype):
    """The values of packed e2m1 codes with their scales."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                         dtype=dtype, device=q.device)
    i = torch.stack((q & 15, q >> 4), 2).reshape(q.shape[0], -1)
    v = table[i.to(torch.int32)].reshape(q.shape[0], -1, 32)
    return (v * _power(scale).to(dtype).unsqueeze(2)).reshape(q.shape[0], -1)


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "product":
        if c["act"] == "codes":
            a = _unpack(s["a"], s["as"], torch.float32)
        else:
            code, v = _mx_plain(s["x"], "e2m1")
            a = (v.reshape(c["M"], -1, 32) * _power(code).unsqueeze(2)).reshape(c["M"], -1)
        return torch.matmul(a, _unpack(s["w"], s["ws"], torch.float32).t()).to(TYPES[c["dtype"]])
    if op == "norm":
        out = {}
        h = s["x"].float()
        if c["residual"]:
            out["h"] = (h + s["r"].float()).to(TYPES[c["dtype"]])
            h = out["h"].float()
        rstd = torch.rsqrt(h.square().mean(1) + EPS)
        out["rstd"] = rstd
        y = h * rstd.unsqueeze(1) * s["w"].float()
        if c["out"] == "same":
            out["y"] = y.to(TYPES[c["dtype"]])
        elif c["scales"] == "row":
            out["scale"] = (y.abs().amax(1) / 448).clamp(min=2.0 ** -126)
            out["codes"] = (y / out["scale"].unsqueeze(1)).to(torch.float8_e4m3fn)
        else:
            out.update(_mx_outputs(y, c["out"]))
        return out
    if op == "norm_grad":
        h, dy, rstd = s["h"].float(), s["dy"].float(), s["rstd"].unsqueeze(1)
        n = h * rstd
        g = dy * s["w"].float()
        dx = rstd * (g - n * (g * n).mean(1, keepdim=True))
        if c["residual"]:
            dx = dx + s["dres"].float()
        return {"dx": dx.to(TYPES[c["dtype"]]), "dw": (dy * n).sum(0)}
    return _mx_outputs(s["x"].t() if c["transpose"] else s["x"], c["fmt"])


# --- the framework's operators -----------------------------------------------

def _run_own(s):
    import implicit_gemm_conv_dp_amd as skg

    c = s["case"]
    op = c["op"]
    if op == "product":
        M, N, K = c["M"], c["N"], c["K"]
        if c["act"] != "codes":
            skg.mx_quant(s["x"], s["a"], s["as"], rows=M, cols=K, dtype="bf16", dtype_q="e2m1")
        skg.gemm(s["a"], s["w"], s["c"], s["as"], s["ws"], M=M, N=N, K=K, ldc=s["ldc"],
                 dtype_ab="e2m1", dtype_c=c["dtype"], scale_mode="mx", tile="auto", mode="auto",
                 reduction="auto", ctas=-1)
        return s["c"][:, :N]
    rows, cols = c["rows"], c["cols"]
    if op == "norm":
        quant = c["out"] != "same"
        skg.rmsnorm(s["x"], s["y"], rows=rows, cols=cols, dtype=c["dtype"], weight=s["w"],
                    dtype_w="f32" if c["w32"] else c["dtype"], residual=s["r"], h=s["h"],
                    rstd=s["rstd"], y_scale=s["scale"], dtype_y=c["out"] if quant else c["dtype"],
                    scale_mode="mx" if c["scales"] == "mx" else "rowcol", eps=EPS,
                    ldx=cols + c["pad"])
        out = {"rstd": s["rstd"]}
        if c["residual"]:
            out["h"] = s["h"]
        if not quant:
            out["y"] = s["y"]
            return out
        out["scale"] = s["scale"]
        if c["scales"] == "mx":
            out["scale"] = s["scale"].view(torch.float8_e8m0fnu)
        if c["out"] == "e4m3":
            out["codes"] = s["y"].view(torch.float8_e4m3fn)
        else:
            skg.mx_dequant(s["y"], s["scale"], s["values"], rows=rows, cols=cols, dtype_q="e2m1",
                           dtype="bf16")
            out["values"] = s["values"]
        return out
    if op == "norm_grad":
        skg.rmsnorm_bwd(s["dy"], s["h"], s["rstd"], s["dx"], rows=rows, cols=cols,
                        dtype=c["dtype"], weight=s["w"], dtype_w="f32" if c["w32"] else c["dtype"],
                        dres=s["dres"], dw=s["dw"])
        return {"dx": s["dx"], "dw": s["dw"]}
    skg.mx_quant(s["x"], s["q"], s["scale"], rows=rows, cols=cols, dtype=c["dtype"],
                 dtype_q=c["fmt"], ldx=cols + c["pad"], transpose=c["transpose"])
    scale = s["scale"].view(torch.float8_e8m0fnu)
    if c["fmt"] == "e4m3":
        return {"scale": scale, "codes": s["q"].view(torch.float8_e4m3fn)}
    R, C = (cols, rows) if c["transpose"] else (rows, cols)
    skg.mx_dequant(s["q"], s["scale"], s["values"], rows=R, cols=C, dtype_q="e2m1", dtype="bf16")
    return {"scale": scale, "values": s["values"]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# --- from the definitions, in 64 bits ----------------------------------------

def _power64(e):
    """2^e of whole e, made from its bits (a power function may be off by an
    ulp, which moves values next to a border)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _nearest(v, mantissa, lowest, largest):
    """Round to nearest even in a format of `mantissa` fraction bits whose
    smallest normal exponent is `lowest`; saturate at `largest`."""
    a = v.abs()
    step = _power64((torch.frexp(a)[1] - 1).clamp(min=lowest) - mantissa)
    return torch.copysign((torch.round(a / step) * step).clamp(max=largest), v)


def _mx_exact(x, fmt):
    b = x.double().reshape(x.shape[0], -1, 32)
    top = b.abs().amax(2)
    power = torch.where(top > 0, torch.frexp(top)[1] - 1 - EMAX[fmt], -127)
    d = _power64(power.clamp(min=-127))
    v = b / d.unsqueeze(2)
    v = _nearest(v, 1, 0, 6.0) if fmt == "e2m1" else _nearest(v, 3, -6, 448.0)
    if fmt == "e4m3":
        return {"scale": d, "codes": v.reshape(x.shape)}
    return {"scale": d, "values": (v * d.unsqueeze(2)).reshape(x.shape)}


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    op = c["op"]
    if op == "product":
        a = (_unpack(s["a"], s["as"], torch.float64) if c["act"] == "codes" else
             _mx_exact(s["x"], "e2m1")["values"])
        return torch.matmul(a, _unpack(s["w"], s["ws"], torch.float64).t())
    if op == "norm":
        out = {}
        h = s["x"].double()
        if c["residual"]:
            h = (h + s["r"].double()).to(TYPES[c["dtype"]]).double()
            out["h"] = h
        rstd = 1 / torch.sqrt((h * h).sum(1) / c["cols"] + EPS)
        out["rstd"] = rstd
        y = h * rstd[:, None] * s["w"].double()
        if c["out"] == "same":
            out["y"] = y
        elif c["scales"] == "row":
            d = (y.abs().amax(1) / 448).clamp(min=2.0 ** -126)
            out["scale"] = d
            out["codes"] = _nearest(y / d[:, None], 3, -6, 448.0)
        else:
            out.update(_mx_exact(y, c["out"]))
        return out
    if op == "norm_grad":
        h, dy, w, r = s["h"].double(), s["dy"].double(), s["w"].double(), s["rstd"].double()[:, None]
        dot = (dy * w * h).sum(1, keepdim=True)
        dx = r * dy * w - h * r ** 3 * dot / c["cols"]
        if c["residual"]:
            dx = dx + s["dres"].double()
        return {"dx": dx, "dw": (dy * h * r).sum(0)}
    return _mx_exact(s["x"].t() if c["transpose"] else s["x"], c["fmt"])
