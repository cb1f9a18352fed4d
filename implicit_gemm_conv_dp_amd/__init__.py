"""Stream-K GEMM and conv-wgrad engine for MI355X (gfx950).

The compute path is the HIP library ``libskgemm.so`` (C ABI in
``include/skgemm.h``); this package only marshals torch device tensors and
streams into its calls.  PyTorch provides device memory and streams.

    import implicit_gemm_conv_dp_amd as skg
    plan = skg.gemm(A, B, C, M=..., N=..., K=..., dtype_ab="bf16", dtype_c="bf16",
                    tile="256x256x64", mode="dp_sk", reduction="tree", ctas=256)

``A`` is M x K row-major, ``B`` is K x N column-major (N rows of K), ``C`` is
M x N row-major; tensors are passed as raw storage (any torch dtype), their
element type is ``dtype_ab`` / ``dtype_c``.  ``wgrad`` takes NHWC ``x`` and
``dy`` and writes the fp32 KRSC filter gradient ``dw``.

Around the products of a layer: ``rmsnorm`` (with the residual's addition and
the output as 16-bit values, e4m3 codes with row scales, or MX blocks) and
``rmsnorm_bwd``; ``mx_quant`` / ``mx_dequant`` to and from MX blocks of e4m3 or
e2m1 (4-bit) codes; and ``gemm(dtype_ab="e2m1", scale_mode="mx",
tile="auto")`` for their product.
"""

import contextlib

from . import _lib
from ._lib import (SkgError, skg_default_pool, skg_device_info, skg_plan_gemm,  # noqa: F401
                   skg_plan_run_gemm, skg_plan_wgrad, skg_profile_events, skg_run_gemm,
                   skg_run_wgrad, skg_tile_info, skg_gemm_workspace_bytes, skg_wgrad_workspace_bytes,
                   skg_fixup_timeouts, skg_run_wgrad_static, skg_plan_fwd, skg_plan_dgrad,
                   skg_run_fwd, skg_run_dgrad, skg_run_rmsnorm, skg_run_rmsnorm_bwd,
                   skg_plan_run_rmsnorm_bwd, skg_rmsnorm_bwd_workspace_bytes,
                   skg_run_mx_quant, skg_run_mx_dequant, MODES,
                   REDUCTIONS, DTYPES, TILES, SCALE_MODES, SK_ORDERS)

__all__ = ["gemm", "wgrad", "fwd", "dgrad", "plan_gemm", "plan_wgrad", "plan_fwd", "plan_dgrad",
           "gemm_args", "wgrad_args", "conv_args",
           "workspace_for", "SkgError", "MODES", "REDUCTIONS", "DTYPES", "TILES", "SCALE_MODES",
           "SK_ORDERS",
           "skg_default_pool", "skg_device_info", "skg_plan_gemm", "skg_plan_wgrad",
           "skg_run_gemm", "skg_plan_run_gemm", "skg_run_wgrad", "skg_tile_info",
           "skg_profile_events",
           "skg_gemm_workspace_bytes", "skg_wgrad_workspace_bytes", "skg_fixup_timeouts",
           "skg_run_wgrad_static", "skg_plan_fwd", "skg_plan_dgrad", "skg_run_fwd",
           "skg_run_dgrad", "rmsnorm", "rmsnorm_bwd", "mx_quant", "mx_dequant",
           "rmsnorm_args", "rmsnorm_bwd_args", "mx_args", "skg_run_rmsnorm",
           "skg_run_rmsnorm_bwd", "skg_plan_run_rmsnorm_bwd", "skg_rmsnorm_bwd_workspace_bytes",
           "skg_run_mx_quant",
           "skg_run_mx_dequant"]


class _Names(dict):
    """The values of a table's names; whole numbers stand for themselves."""

    def __init__(self, table, what):
        super().__init__(table)
        self.what = what

    def __missing__(self, v):
        if isinstance(v, int):
            return v
        raise ValueError("unknown %s %r" % (self.what, v))


_DTYPE = _Names(DTYPES, "dtype")
_TILE = _Names(TILES, "tile")
_MODE = _Names(MODES, "mode")
_REDUCTION = _Names(REDUCTIONS, "reduction")
_SCALE_MODE = _Names(SCALE_MODES, "scale mode")
_SK_ORDER = _Names(SK_ORDERS, "stream-K order")


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def gemm_args(A=None, B=None, C=None, *, M, N, K, dtype_ab, dtype_c, lda=None, ldb=None,
              ldc=None, scale_a=None, scale_b=None, scale_mode="rowcol", tile, mode, reduction,
              ctas, sk_order="auto"):
    # Positional, in the struct's order: a call for a few tokens spends more
    # time here than on the GPU.
    return _lib.skg_gemm_args_t(
        M, N, K, _DTYPE[dtype_ab], _DTYPE[dtype_c],
        0 if A is None else A.data_ptr(), K if lda is None else lda,
        0 if B is None else B.data_ptr(), K if ldb is None else ldb,
        0 if C is None else C.data_ptr(), N if ldc is None else ldc,
        0 if scale_a is None else scale_a.data_ptr(), 0 if scale_b is None else scale_b.data_ptr(),
        _lib.TILE_AUTO if tile == "auto" else _TILE[tile], _MODE[mode], _REDUCTION[reduction],
        ctas, _SCALE_MODE[scale_mode], _SK_ORDER[sk_order])


def wgrad_args(x=None, dy=None, dw=None, *, n, h, w, c, k, r, s, stride=(1, 1), pad=(0, 0),
               groups=1, dtype, tile, mode, reduction, ctas, sk_order="auto"):
    a = _lib.skg_wgrad_args_t()
    a.n, a.h, a.w, a.c, a.k, a.r, a.s = n, h, w, c, k, r, s
    a.stride_h, a.stride_w = stride
    a.pad_h, a.pad_w = pad
    a.groups = groups
    a.dtype = _DTYPE[dtype]
    a.x, a.dy, a.dw = _ptr(x), _ptr(dy), _ptr(dw)
    a.tile_id = _TILE[tile]
    a.mode = _MODE[mode]
    a.reduction = _REDUCTION[reduction]
    a.ctas = ctas
    a.sk_order = _SK_ORDER[sk_order]
    return a


def conv_args(act=None, filt=None, out=None, *, n, h, w, c, k, r, s, stride=(1, 1), pad=(0, 0),
              groups=1, dtype, dtype_out, tile, mode, reduction, ctas, sk_order="auto"):
    """Arguments of a forward convolution (act = X, out = Y) or of its input
    gradient (act = dY, out = dX); filt is the KRSC filter W either way."""
    a = _lib.skg_conv_args_t()
    a.n, a.h, a.w, a.c, a.k, a.r, a.s = n, h, w, c, k, r, s
    a.stride_h, a.stride_w = stride
    a.pad_h, a.pad_w = pad
    a.groups = groups
    a.dtype = _DTYPE[dtype]
    a.dtype_out = _DTYPE[dtype_out]
    a.act, a.filt, a.out = _ptr(act), _ptr(filt), _ptr(out)
    a.tile_id = _TILE[tile]
    a.mode = _MODE[mode]
    a.reduction = _REDUCTION[reduction]
    a.ctas = ctas
    a.sk_order = _SK_ORDER[sk_order]
    return a


def plan_gemm(**kw):
    return skg_plan_gemm(gemm_args(**kw)).as_dict()


def plan_wgrad(**kw):
    return skg_plan_wgrad(wgrad_args(**kw)).as_dict()


def plan_fwd(**kw):
    return skg_plan_fwd(conv_args(**kw)).as_dict()


def plan_dgrad(**kw):
    return skg_plan_dgrad(conv_args(**kw)).as_dict()


def workspace_for(plan, device):
    """A device buffer large enough for ``plan`` (torch owns the memory)."""
    import torch
    return torch.empty(max(int(plan["workspace_bytes"]), 1), dtype=torch.uint8, device=device)


def _launch_stream(stream):
    import torch
    return torch.cuda.current_stream() if stream is None else stream


_current_handle = None


def _handle(stream):
    """The launch stream's handle.  Without a caller's stream that of torch's
    current one, asked for without making a Stream object where torch offers it
    (0.2 us against 2.9)."""
    global _current_handle
    if stream is not None:
        return stream.cuda_stream
    if _current_handle is None:
        import torch
        if not torch.cuda.is_initialized():
            return 0  # nothing has made another stream the current one
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        device = getattr(torch._C, "_cuda_getDevice", None)
        if raw and device:
            _current_handle = lambda: raw(device())
        else:
            _current_handle = lambda: torch.cuda.current_stream().cuda_stream
    return _current_handle()


def _pool_of(stream):
    """A context whose allocations come from the launch stream's pool: memory
    of another stream's may have been freed there by work that is still to
    run, which only that stream's own order makes safe."""
    if stream is None:
        return contextlib.nullcontext()
    import torch
    return torch.cuda.stream(stream)


def _run(run, args, plan, device, workspace, stream):
    """One run call.  A workspace the call allocates itself comes from the
    launch stream's pool, so that whatever used its memory before and uses it
    afterwards is ordered with the kernel, whichever stream the caller passed.
    A plan without one allocates nothing."""
    if workspace is not None:
        run(args, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
            _handle(stream))
    elif not plan["workspace_bytes"]:
        run(args, 0, 0, _handle(stream))
    else:
        s = _launch_stream(stream)
        with _pool_of(stream):
            ws = workspace_for(plan, device)
        ws.record_stream(s)
        run(args, ws.data_ptr(), ws.numel() * ws.element_size(), s.cuda_stream)


def gemm(A, B, C, scale_a=None, scale_b=None, workspace=None, stream=None, **kw):
    """Enqueue C = epilogue(A @ B) on ``stream`` (default: torch's current
    stream).  Returns the plan (a dict)."""
    args = gemm_args(A, B, C, scale_a=scale_a, scale_b=scale_b, **kw)
    if workspace is None:
        plan, launched = skg_plan_run_gemm(args, 0, 0, _handle(stream))
        plan = plan.as_dict()
        if launched:
            return plan
    else:
        plan = skg_plan_gemm(args).as_dict()
    _run(skg_run_gemm, args, plan, C.device, workspace, stream)
    return plan


def wgrad(x, dy, dw, workspace=None, stream=None, **kw):
    """Enqueue dw = wgrad(x, dy) on ``stream``.  Returns the plan (a dict)."""
    args = wgrad_args(x, dy, dw, **kw)
    plan = skg_plan_wgrad(args).as_dict()
    _run(skg_run_wgrad, args, plan, dw.device, workspace, stream)
    return plan


def fwd(x, filt, y, workspace=None, stream=None, **kw):
    """Enqueue the forward convolution y = conv(x, filt) on ``stream``.
    Returns the plan (a dict)."""
    args = conv_args(x, filt, y, **kw)
    plan = skg_plan_fwd(args).as_dict()
    _run(skg_run_fwd, args, plan, y.device, workspace, stream)
    return plan


def dgrad(dy, filt, dx, workspace=None, stream=None, **kw):
    """Enqueue the input gradient dx = dgrad(dy, filt) on ``stream``.
    Returns the plan (a dict)."""
    args = conv_args(dy, filt, dx, **kw)
    plan = skg_plan_dgrad(args).as_dict()
    _run(skg_run_dgrad, args, plan, dx.device, workspace, stream)
    return plan


def rmsnorm_args(x=None, y=None, *, rows, cols, dtype, dtype_y=None, weight=None, dtype_w=None,
                 residual=None, h=None, rstd=None, y_scale=None, scale_mode="rowcol", eps=1e-5,
                 ldx=None, ldr=None, ldh=None, ldy=None):
    dt = _DTYPE[dtype]
    return _lib.skg_norm_args_t(
        rows, cols, dt,
        dt if dtype_w is None else _DTYPE[dtype_w],
        dt if dtype_y is None else _DTYPE[dtype_y],
        _SCALE_MODE[scale_mode],
        0 if x is None else x.data_ptr(), cols if ldx is None else ldx,
        0 if residual is None else residual.data_ptr(), cols if ldr is None else ldr,
        0 if weight is None else weight.data_ptr(),
        0 if h is None else h.data_ptr(), cols if ldh is None else ldh,
        0 if y is None else y.data_ptr(), cols if ldy is None else ldy,
        0 if y_scale is None else y_scale.data_ptr(),
        0 if rstd is None else rstd.data_ptr(), eps)


def rmsnorm_bwd_args(dy=None, h=None, rstd=None, dx=None, *, rows, cols, dtype, weight=None,
                     dtype_w=None, dres=None, dw=None, lddy=None, ldh=None, lddres=None,
                     lddx=None):
    dt = _DTYPE[dtype]
    return _lib.skg_norm_bwd_args_t(
        rows, cols, dt, dt if dtype_w is None else _DTYPE[dtype_w],
        0 if dy is None else dy.data_ptr(), cols if lddy is None else lddy,
        0 if h is None else h.data_ptr(), cols if ldh is None else ldh,
        0 if rstd is None else rstd.data_ptr(),
        0 if weight is None else weight.data_ptr(),
        0 if dres is None else dres.data_ptr(), cols if lddres is None else lddres,
        0 if dx is None else dx.data_ptr(), cols if lddx is None else lddx,
        0 if dw is None else dw.data_ptr())


def mx_args(x=None, q=None, scales=None, *, rows, cols, dtype, dtype_q, kq=None, ldx=None,
            ldq=None, transpose=False):
    if kq is None:
        kq = ((rows if transpose else cols) + 31) // 32 * 32
    return _lib.skg_mx_args_t(
        rows, cols, kq, _DTYPE[dtype], _DTYPE[dtype_q],
        0 if x is None else x.data_ptr(), cols if ldx is None else ldx,
        0 if q is None else q.data_ptr(), kq if ldq is None else ldq,
        0 if scales is None else scales.data_ptr(), 1 if transpose else 0)


def rmsnorm(x, y, stream=None, **kw):
    """Enqueue y = norm(x + residual) * weight on ``stream``; ``h`` receives
    the sum, ``rstd`` the rows' factors for ``rmsnorm_bwd``, ``y_scale`` the
    scales of a quantised output (``dtype_y``).  MX blocks (``scale_mode="mx"``)
    take ``cols`` a multiple of 32; an MX product of them a multiple of 128."""
    skg_run_rmsnorm(rmsnorm_args(x, y, **kw), _handle(stream))


def rmsnorm_bwd(dy, h, rstd, dx, workspace=None, stream=None, **kw):
    """Enqueue the norm's gradient on ``stream``: dx (plus ``dres``) and the
    fp32 weight gradient ``dw``; either may be None."""
    args = rmsnorm_bwd_args(dy, h, rstd, dx, **kw)
    if workspace is not None:
        skg_run_rmsnorm_bwd(args, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                            _handle(stream))
        return
    need, launched = skg_plan_run_rmsnorm_bwd(args, 0, 0, _handle(stream))
    if not launched:
        import torch
        with _pool_of(stream):
            ws = torch.empty(need, dtype=torch.uint8, device=kw["dw"].device)
        skg_run_rmsnorm_bwd(args, ws.data_ptr(), need, _handle(stream))


def mx_quant(x, q, scales, stream=None, **kw):
    """Enqueue the MX quantisation of ``x`` into codes ``q`` and E8M0
    ``scales`` on ``stream``; ``transpose=True`` quantises along the columns and
    writes the codes transposed."""
    skg_run_mx_quant(mx_args(x, q, scales, **kw), _handle(stream))


def mx_dequant(q, scales, x, stream=None, **kw):
    """Enqueue x = the values of MX codes ``q`` with ``scales`` on ``stream``."""
    skg_run_mx_dequant(mx_args(x, q, scales, **kw), _handle(stream))
