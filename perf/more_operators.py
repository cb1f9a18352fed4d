"""What is measured of the operators of an 8-bit attention projection: block
quantisation and the product of 8-bit operands with a scale for each block of
128, norms of queries and keys for each head with the position's rotation and
their gradient, and the orthogonalisation of a weight's update by Newton-Schulz
products.

``run`` computes an operator in elementary torch operations, or, where ``own``
is set, through the framework's entry points.
"""

import math

import torch

own = False

EPS = 1e-6
NS_EPS = 1e-7
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
CODES = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}


def listed():
    return [
        # One token of a decode step through an 8-bit projection: its
        # activations are quantised, then multiplied.
        dict(name="product 1x8192x8192", op="product", M=1, N=8192, K=8192, fmt="e4m3",
             dtype="bf16", blocks="128x128", act="bf16"),
        # A serving batch over an odd number of outputs.
        dict(name="product 48x4863x4096", op="product", M=48, N=4863, K=4096, fmt="e4m3",
             dtype="f16", blocks="128x128", act="codes"),
        # A weight's gradient: both operands quantised along the tokens, 32-bit.
        dict(name="product 4096x4864x8192 f32", op="product", M=4096, N=4864, K=8192, fmt="e4m3",
             dtype="f32", blocks="1x128", act="codes"),
        # A long prompt or a training step: the largest product.
        dict(name="product 8192x8192x8192", op="product", M=8192, N=8192, K=8192, fmt="e4m3",
             dtype="bf16", blocks="128x128", act="codes"),
        # A short odd batch's gradient in the wider-ranged format, on a slice of
        # a wider buffer, along the rows and the tokens.
        dict(name="quant 509x1111 e5m2", op="quant", rows=509, cols=1111, dtype="f32", fmt="e5m2",
             blocks="1x128", along="both", pad=24),
        # A training step's gradient along the outputs (for the input's
        # gradient) and along the tokens (for the weight's) from one read.
        dict(name="quant 16384x4096 both", op="quant", rows=16384, cols=4096, dtype="bf16",
             fmt="e4m3", blocks="1x128", along="both", pad=0),
        # One token's queries and keys in a decode step, far into its context.
        dict(name="heads 1x(32+8)x128", op="heads", tokens=1, heads_q=32, heads_k=8, dim=128,
             rope=128, style="half", dtype="bf16", w32=False, table=131072),
        # A training step's queries and keys of packed sequences.
        dict(name="heads 16384x(32+8)x128", op="heads", tokens=16384, heads_q=32, heads_k=8,
             dim=128, rope=128, style="half", dtype="bf16", w32=False, table=32768),
        # Their gradient on a short odd batch: a partial rotation of odd heads
        # in neighbouring pairs, 32-bit.
        dict(name="heads grad 509x(12+12)x80", op="heads_grad", tokens=509, heads_q=12, heads_k=12,
             dim=80, rope=20, style="pairs", dtype="f32", w32=True, table=4096),
        # Their gradient in the training step.
        dict(name="heads grad 16384x(32+8)x128", op="heads_grad", tokens=16384, heads_q=32,
             heads_k=8, dim=128, rope=128, style="half", dtype="bf16", w32=True, table=32768),
        # The update of a small odd projection.
        dict(name="update 300x1111", op="update", rows=300, cols=1111, dtype="bf16", steps=5),
        # The update of a large projection from its 32-bit gradient.
        dict(name="update 4864x4096", op="update", rows=4864, cols=4096, dtype="f32", steps=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "product", "quant", "heads", "heads_grad", "update"])
    if op == "product":
        act = rng.choice(["codes", "codes", "bf16"])
        return dict(op=op, M=_log(rng, 1, 8192), N=_log(rng, 64, 8192), K=128 * _log(rng, 1, 64),
                    fmt=rng.choice(["e4m3", "e4m3", "e5m2"]),
                    dtype=rng.choice(["bf16", "bf16", "f16", "f32"]),
                    blocks=rng.choice(["128x128", "1x128"]), act=act)
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "quant":
        cols = _log(rng, 32, 16384)
        return dict(op=op, rows=_log(rng, 1, min(16384, (1 << 26) // cols)), cols=cols, dtype=dtype,
                    fmt=rng.choice(["e4m3", "e4m3", "e5m2"]),
                    blocks=rng.choice(["1x128", "128x128"]),
                    along=rng.choice(["rows", "columns", "both"]), pad=rng.choice([0, 0, 8, 24, 3]))
    if op == "update":
        rows = _log(rng, 64, 4864)
        return dict(op=op, rows=rows, cols=_log(rng, 64, 4096), dtype=rng.choice(["f32", "bf16"]),
                    steps=5)
    heads_k = rng.choice([1, 2, 4, 8, 12])
    dim = rng.choice([64, 80, 96, 128, 128, 256])
    heads_q = heads_k * rng.choice([1, 2, 4, 8])
    style = rng.choice(["half", "pairs"])
    rope = rng.choice([dim, dim, dim // 2, dim // 4])
    most = min(16384, (1 << 26) // ((heads_q + heads_k) * dim))
    return dict(op=op, tokens=_log(rng, 1, most), heads_q=heads_q, heads_k=heads_k, dim=dim,
                rope=rope, style=style, dtype=dtype, w32=rng.random() < 0.5,
                table=rng.choice([4096, 32768, 131072]))


def _up(n, m):
    return -(-n // m) * m


def work(case):
    op, c = case["op"], case
    if op == "product":
        M, N, K = c["M"], c["N"], c["K"]
        scales = 4 * (K // 128) * (-(-N // 128) if c["blocks"] == "128x128" else N)
        a = 2 * M * K if c["act"] == "bf16" else M * K + 4 * M * (K // 128)
        return {"bytes": a + N * K + scales + M * N * SIZE[c["dtype"]], "flops": 2.0 * M * N * K}
    if op == "quant":
        n = c["rows"] * c["cols"]
        return {"bytes": n * (SIZE[c["dtype"]] + (2 if c["along"] == "both" else 1)), "flops": 3.0 * n}
    if op == "update":
        m, n = sorted((c["rows"], c["cols"]))
        # The products of a matrix with its own transpose are symmetric.
        return {"bytes": c["rows"] * c["cols"] * (SIZE[c["dtype"]] + 2),
                "flops": float(c["steps"]) * (3 * m * m * n + m * m * m)}
    n = c["tokens"] * (c["heads_q"] + c["heads_k"]) * c["dim"]
    return {"bytes": n * SIZE[c["dtype"]] * (2 if op == "heads" else 3) + 4 * c["tokens"] * c["rope"],
            "flops": (8.0 if op == "heads" else 14.0) * n}


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


def _operand(g, rows, K, fmt, tall):
    """Codes and scales of normal values whose lines differ in size, in blocks
    of 1 x 128, or with tall of 128 x 128."""
    q = torch.empty(rows, K, dtype=torch.uint8, device="cuda")
    s = torch.empty(K // 128, -(-rows // 128) if tall else rows, device="cuda")
    for r0 in range(0, rows, 2048):
        n = min(2048, rows - r0)
        x = torch.randn(n, K, generator=g, device="cuda")
        x *= torch.exp(0.5 * torch.randn(n, 1, generator=g, device="cuda"))
        part = _quant_plain(x, fmt, tall)
        q[r0:r0 + n] = part["codes"].view(torch.uint8)
        w = part["scale"].shape[1]
        at = r0 // 128 if tall else r0
        s[:, at:at + w] = part["scale"]
    return q, s


def _tables(rows, half):
    """Cosines and sines of the angles of each position, from 64 bits."""
    rate = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / max(half, 1))
    a = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * rate
    return a.cos().float(), a.sin().float()


def _positions(g, tokens, table):
    """Positions of packed sequences of different lengths, each continuing at a
    place of its own; a single token stands far into its context."""
    starts = torch.rand(tokens, generator=g, device="cuda") < 4.0 / max(tokens, 4)
    starts[0] = True
    t = torch.arange(tokens, device="cuda")
    begin = torch.where(starts, t, 0).cummax(0)[0]
    run = t - begin
    offset = torch.randint(0, table, (tokens,), generator=g, device="cuda")[begin]
    return ((offset + run) % table).to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    s = {"case": c}
    op = c["op"]
    if op == "product":
        M, N, K = c["M"], c["N"], c["K"]
        s["w"], s["ws"] = _operand(g, N, K, c["fmt"], c["blocks"] == "128x128")
        if c["act"] == "codes":
            s["a"], s["as"] = _operand(g, M, K, c["fmt"], False)
        else:
            s["x"] = _activations(g, M, K, "bf16")
            s["a"] = torch.empty(M, K, dtype=torch.uint8, device="cuda")
            s["as"] = torch.empty(K // 128, M, device="cuda")
        s["ldc"] = _up(N, 8)
        s["c"] = torch.empty(M, s["ldc"], dtype=TYPES[c["dtype"]], device="cuda")
        return s
    if op == "quant":
        rows, cols = c["rows"], c["cols"]
        s["x"] = _activations(g, rows, cols, c["dtype"], c["pad"])
        tall = c["blocks"] == "128x128"
        if c["along"] != "columns":
            kq = _up(cols, 128)
            s["q"] = torch.empty(rows, kq, dtype=torch.uint8, device="cuda")
            s["s"] = torch.empty(kq // 128, -(-rows // 128) if tall else rows, device="cuda")
        if c["along"] != "rows":
            kq = _up(rows, 128)
            s["qt"] = torch.empty(cols, kq, dtype=torch.uint8, device="cuda")
            s["st"] = torch.empty(kq // 128, -(-cols // 128) if tall else cols, device="cuda")
        return s
    if op == "update":
        rows, cols = c["rows"], c["cols"]
        # A gradient has a few strong directions and many weak ones.
        r = max(1, min(rows, cols) // 8)
        x = torch.randn(rows, r, generator=g, device="cuda") @ torch.randn(r, cols, generator=g, device="cuda")
        x = x / math.sqrt(r) + 0.5 * torch.randn(rows, cols, generator=g, device="cuda")
        s["g"] = (1e-3 * x).to(TYPES[c["dtype"]])
        s["out"] = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
        return s
    T, Hq, Hk, D = c["tokens"], c["heads_q"], c["heads_k"], c["dim"]
    dtype = TYPES[c["dtype"]]
    # Queries, keys and values as a projection writes them, side by side.
    qkv = torch.randn(T, (Hq + 2 * Hk) * D, generator=g, device="cuda")
    qkv *= torch.exp(0.5 * torch.randn((Hq + 2 * Hk) * D, generator=g, device="cuda"))
    qkv = qkv.to(dtype)
    s["pitch"] = qkv.shape[1]
    s["q"], s["k"] = qkv[:, :Hq * D].view(T, Hq, D), qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
    wt = torch.float32 if c["w32"] else dtype
    s["wq"], s["wk"] = ((1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(wt) for _ in range(2))
    s["cos"], s["sin"] = _tables(c["table"], c["rope"] // 2)
    s["pos"] = _positions(g, T, c["table"])
    s["yq"], s["yk"] = (torch.empty(T, H, D, dtype=dtype, device="cuda") for H in (Hq, Hk))
    if op == "heads_grad":
        s["dq"], s["dk"] = ((torch.randn(T, H, D, generator=g, device="cuda") * 0.1).to(dtype) for H in (Hq, Hk))
        s["dwq"], s["dwk"] = (torch.empty(D, device="cuda") for _ in range(2))
    return s


# --- the plain forms ---------------------------------------------------------

def _padded(x):
    rows, cols = x.shape
    return torch.nn.functional.pad(x, (0, _up(cols, 128) - cols))


def _quant_plain(x, fmt, tall):
    """Codes of x's rows padded to whole blocks, and the blocks' scales, a line
    for each 128 columns.  A code is the one nearest to x MAX / top, top the
    block's largest magnitude; in 64 bits, as many of these quotients lie just
    between two codes."""
    rows = x.shape[0]
    x = _padded(x.double())
    if tall:
        b = torch.nn.functional.pad(x, (0, 0, 0, _up(rows, 128) - rows)).reshape(-1, 128, x.shape[1] // 128, 128)
        top = b.abs().amax((1, 3), keepdim=True)
    else:
        b = x.reshape(rows, 1, -1, 128)
        top = b.abs().amax(3, keepdim=True)
    top = top.clamp(min=LARGEST[fmt] * 2.0 ** -126)
    q = (b * LARGEST[fmt] / top).to(CODES[fmt]).reshape(-1, x.shape[1])[:rows]
    d = (top / LARGEST[fmt]).float()
    return {"codes": q, "scale": d.reshape(d.shape[0], d.shape[2]).t().contiguous()}


def _values(q, s, fmt, tall, dtype):
    """The values of codes with their blocks' scales."""
    rows, K = q.shape
    d = s.t().to(dtype)
    if tall:
        d = d.repeat_interleave(128, 0)[:rows]
    return (q.view(CODES[fmt]).to(dtype).reshape(rows, K // 128, 128) * d.unsqueeze(2)).reshape(rows, K)


def _rotate(n, cos, sin, style):
    """Rows of (tokens, heads, dim) turned in their first 2 x cos.shape[1] elements."""
    half = cos.shape[1]
    cos, sin = cos[:, None, :], sin[:, None, :]
    if style == "half":
        a, b, rest = n[..., :half], n[..., half:2 * half], n[..., 2 * half:]
        return torch.cat((a * cos - b * sin, b * cos + a * sin, rest), 2)
    a, b, rest = n[..., 0:2 * half:2], n[..., 1:2 * half:2], n[..., 2 * half:]
    return torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), 3).flatten(2), rest), 2)


def _heads_plain(x, w, cos, sin, style):
    x = x.float()
    n = x * torch.rsqrt(x.square().mean(2, keepdim=True) + EPS) * w.float()
    return _rotate(n, cos, sin, style)


def _heads_grad_plain(dy, x, w, cos, sin, style):
    x = x.float()
    g = _rotate(dy.float(), cos, -sin, style)
    r = torch.rsqrt(x.square().mean(2, keepdim=True) + EPS)
    n = x * r
    gw = g * w.float()
    return r * (gw - n * (gw * n).mean(2, keepdim=True)), (g * n).sum((0, 1))


def _update_plain(g, steps):
    x = g.float()
    wide = x.shape[0] <= x.shape[1]
    x = x if wide else x.t()
    x = x / (x.square().sum().sqrt() + NS_EPS)
    a, b, c = COEFFICIENTS
    for _ in range(steps):
        s = x @ x.t()
        x = a * x + (b * s + c * (s @ s)) @ x
    return x if wide else x.t()


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "product":
        tall = c["blocks"] == "128x128"
        a, sa = s["a"], s["as"]
        if c["act"] != "codes":
            part = _quant_plain(s["x"], c["fmt"], False)
            a, sa = part["codes"], part["scale"]
        a = _values(a, sa, c["fmt"], False, torch.float32)
        w = _values(s["w"], s["ws"], c["fmt"], tall, torch.float32)
        return torch.matmul(a, w.t()).to(TYPES[c["dtype"]])
    if op == "quant":
        tall, out = c["blocks"] == "128x128", {}
        if c["along"] != "columns":
            out["rows"] = _quant_plain(s["x"], c["fmt"], tall)
        if c["along"] != "rows":
            out["columns"] = _quant_plain(s["x"].t(), c["fmt"], tall)
        return out
    if op == "update":
        return _update_plain(s["g"], c["steps"]).to(torch.bfloat16)
    cos, sin = s["cos"][s["pos"]], s["sin"][s["pos"]]
    dtype = TYPES[c["dtype"]]
    if op == "heads":
        return {"q": _heads_plain(s["q"], s["wq"], cos, sin, c["style"]).to(dtype),
                "k": _heads_plain(s["k"], s["wk"], cos, sin, c["style"]).to(dtype)}
    dq, dwq = _heads_grad_plain(s["dq"], s["q"], s["wq"], cos, sin, c["style"])
    dk, dwk = _heads_grad_plain(s["dk"], s["k"], s["wk"], cos, sin, c["style"])
    return {"dq": dq.to(dtype), "dk": dk.to(dtype), "dwq": dwq, "dwk": dwk}


# --- the framework's operators -----------------------------------------------

def _run_own(s):
    import implicit_gemm_conv_dp_amd as skg

    c = s["case"]
    op = c["op"]
    if op == "product":
        M, N, K = c["M"], c["N"], c["K"]
        if c["act"] != "codes":
            skg.block_quant(s["x"], s["a"], s["as"], rows=M, cols=K, dtype="bf16", dtype_q=c["fmt"])
        skg.gemm(s["a"], s["w"], s["c"], s["as"], s["ws"], M=M, N=N, K=K, ldc=s["ldc"],
                 dtype_ab=c["fmt"], dtype_c=c["dtype"],
                 scale_mode="block128" if c["blocks"] == "128x128" else "row128", tile="auto",
                 mode="auto", reduction="auto", ctas=-1)
        return s["c"][:, :N]
    if op == "quant":
        rows, cols = c["rows"], c["cols"]
        skg.block_quant(s["x"], s.get("q"), s.get("s"), s.get("qt"), s.get("st"), rows=rows,
                        cols=cols, dtype=c["dtype"], dtype_q=c["fmt"], block=c["blocks"],
                        ldx=cols + c["pad"])
        out = {}
        if "q" in s:
            out["rows"] = {"codes": s["q"].view(CODES[c["fmt"]]), "scale": s["s"]}
        if "qt" in s:
            out["columns"] = {"codes": s["qt"].view(CODES[c["fmt"]]), "scale": s["st"]}
        return out
    if op == "update":
        skg.newton_schulz(s["g"], s["out"], rows=c["rows"], cols=c["cols"], dtype=c["dtype"],
                          dtype_out="bf16", steps=c["steps"], coefficients=COEFFICIENTS, eps=NS_EPS)
        return s["out"]
    D, pitch = c["dim"], (0, s["pitch"], c["dim"])
    kw = dict(seq=c["tokens"], heads_q=c["heads_q"], heads_k=c["heads_k"], head_dim=D,
              rope_dim=c["rope"], dtype=c["dtype"], weight_q=s["wq"], weight_k=s["wk"],
              dtype_w="f32" if c["w32"] else c["dtype"], cos=s["cos"], sin=s["sin"],
              table_rows=c["table"], positions=s["pos"], style=c["style"], eps=EPS,
              q_strides=pitch, k_strides=pitch)
    if op == "heads":
        skg.qknorm_rope(s["q"], s["k"], s["yq"], s["yk"], **kw)
        return {"q": s["yq"], "k": s["yk"]}
    skg.qknorm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["yq"], s["yk"], dwq=s["dwq"],
                        dwk=s["dwk"], **kw)
    return {"dq": s["yq"], "dk": s["yk"], "dwq": s["dwq"], "dwk": s["dwk"]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# --- from the definitions, in 64 bits ----------------------------------------

def _power64(e):
    """2^e of whole e, made from its bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _nearest(v, fmt):
    """Round to nearest even in the format's values; saturate at its largest."""
    mantissa, lowest = (3, -6) if fmt == "e4m3" else (2, -14)
    a = v.abs()
    step = _power64((torch.frexp(a)[1] - 1).clamp(min=lowest) - mantissa)
    return torch.copysign((torch.round(a / step) * step).clamp(max=LARGEST[fmt]), v)


def _quant_exact(x, fmt, tall):
    """By blocks on the padded matrix; the scale is the 32-bit number that is
    handed on."""
    rows = x.shape[0]
    h = 128 if tall else 1
    x = torch.nn.functional.pad(x.double(), (0, -x.shape[1] % 128, 0, -rows % h))
    top = torch.nn.functional.max_pool2d(x.abs()[None], (h, 128))[0]
    top = torch.where(top < LARGEST[fmt] * 2.0 ** -126, LARGEST[fmt] * 2.0 ** -126, top)
    wide = top.repeat_interleave(h, 0).repeat_interleave(128, 1)
    q = _nearest(LARGEST[fmt] * x / wide, fmt)
    return {"codes": q[:rows], "scale": (top / LARGEST[fmt]).float().double().t().contiguous()}


def _turn64(n, cos, sin, style, back=False):
    """Each pair as a complex number times that of its angle."""
    half = cos.shape[1]
    z = torch.complex(cos.double(), -sin.double() if back else sin.double())[:, None]
    out = n.clone()
    if half:
        if style == "half":
            p = torch.complex(n[..., :half].contiguous(), n[..., half:2 * half].contiguous()) * z
            out[..., :half], out[..., half:2 * half] = p.real, p.imag
        else:
            p = torch.complex(n[..., 0:2 * half:2].contiguous(), n[..., 1:2 * half:2].contiguous()) * z
            out[..., 0:2 * half:2], out[..., 1:2 * half:2] = p.real, p.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    op = c["op"]
    if op == "product":
        if c["act"] == "codes":
            a = _values(s["a"], s["as"], c["fmt"], False, torch.float64)
        else:
            e = _quant_exact(s["x"], c["fmt"], False)
            a = e["codes"] * e["scale"].t().repeat_interleave(128, 1)
        w = _values(s["w"], s["ws"], c["fmt"], c["blocks"] == "128x128", torch.float64)
        return torch.matmul(a, w.t())
    if op == "quant":
        tall, out = c["blocks"] == "128x128", {}
        if c["along"] != "columns":
            out["rows"] = _quant_exact(s["x"], c["fmt"], tall)
        if c["along"] != "rows":
            out["columns"] = _quant_exact(s["x"].t(), c["fmt"], tall)
        return out
    if op == "update":
        x = s["g"].double()
        x = x / (torch.linalg.vector_norm(x) + NS_EPS)
        a, b, k = COEFFICIENTS
        eye = torch.eye(min(x.shape), dtype=x.dtype, device=x.device)
        for _ in range(c["steps"]):
            if x.shape[0] <= x.shape[1]:
                m = x @ x.t().contiguous()
                x = (a * eye + b * m + k * m @ m) @ x
            else:
                m = x.t().contiguous() @ x
                x = x @ (a * eye + b * m + k * m @ m)
        return x
    i = s["pos"].long()
    cos, sin = s["cos"].index_select(0, i), s["sin"].index_select(0, i)
    out = {}
    for n in "qk":
        x, w = s[n].double(), s["w" + n].double()
        r = 1 / torch.sqrt((x * x).sum(2, keepdim=True) / c["dim"] + EPS)
        if op == "heads":
            out[n] = _turn64(x * r * w, cos, sin, c["style"])
        else:
            g = _turn64(s["d" + n].double(), cos, sin, c["style"], back=True)
            dot = (g * w * x).sum(2, keepdim=True)
            out["d" + n] = r * g * w - x * r ** 3 * dot / c["dim"]
            out["dw" + n] = (g * x * r).sum(1).sum(0)
    return out
