"""The operators around the gated delta rule in a decoder block: the root-mean-square norm with the
residual's addition (optionally in 8 bits with a scale per row), the linear layer with its epilogue, the
gated linear unit of a feed-forward block, and their gradients (``gdn_rms_norm``, ``gdn_linear``,
``gdn_gated_linear`` and their ``_bwd`` in ``include/gdn.h``).

Argument marshalling only, as in the rest of the package: tensors are CUDA tensors, every leading
dimension is a row, the work runs on the current stream, and gradients are explicit calls.  Inputs whose
rows are contiguous are taken as they are, at any row stride (slices of a fused projection); others are
made contiguous first.  Temporary buffers come from PyTorch's allocator, so the calls can be captured
into a CUDA graph.
"""
from __future__ import annotations

import ctypes

import torch

from ._binding import GdnError, lib

GDN_F32, GDN_BF16, GDN_E4M3 = 0, 1, 2
ACTIVATIONS = {None: 0, "none": 0, "silu": 1, "gelu": 2, "gelu_tanh": 3, "relu": 4, "sigmoid": 5}
_CODE = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16, torch.float8_e4m3fn: GDN_E4M3}
_I64, _INT, _VP = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p


class GdnNormArgs(ctypes.Structure):
    _fields_ = [("rows", _I64), ("width", _INT), ("dtype", _INT), ("w_dtype", _INT), ("out_dtype", _INT),
                ("eps", ctypes.c_float), ("x", _VP), ("ldx", _I64), ("residual", _VP), ("ld_residual", _I64),
                ("weight", _VP), ("y", _VP), ("scale", _VP), ("h", _VP), ("dy", _VP), ("ld_dy", _I64), ("dh", _VP),
                ("ld_dh", _I64), ("dx", _VP), ("dweight", _VP)]


class GdnLinearArgs(ctypes.Structure):
    _fields_ = [("rows", _I64), ("out_features", _INT), ("in_features", _INT), ("dtype", _INT), ("out_dtype", _INT),
                ("act", _INT), ("x", _VP), ("ldx", _I64), ("w", _VP), ("ldw", _I64), ("x_scale", _VP), ("w_scale", _VP),
                ("bias", _VP), ("residual", _VP), ("ld_residual", _I64), ("y", _VP), ("ldy", _I64), ("dy", _VP),
                ("ld_dy", _I64), ("dx", _VP), ("dw", _VP), ("dbias", _VP)]


_bound = None


def _library():
    global _bound
    if _bound is None:
        L = lib()
        np_, lp = ctypes.POINTER(GdnNormArgs), ctypes.POINTER(GdnLinearArgs)
        for f in (L.gdn_rms_norm, L.gdn_quantize_rows):
            f.argtypes, f.restype = [np_, _VP], _INT
        L.gdn_rms_norm_bwd.argtypes, L.gdn_rms_norm_bwd.restype = [np_, _VP, ctypes.c_size_t, _VP], _INT
        L.gdn_rms_norm_bwd_workspace_size.argtypes, L.gdn_rms_norm_bwd_workspace_size.restype = [np_], ctypes.c_size_t
        for n in ("gdn_linear", "gdn_linear_bwd", "gdn_gated_linear", "gdn_gated_linear_bwd"):
            f, w = getattr(L, n), getattr(L, n + "_workspace_size")
            f.argtypes, f.restype = [lp, _VP, ctypes.c_size_t, _VP], _INT
            w.argtypes, w.restype = [lp], ctypes.c_size_t
        L.gdn_read_layer_status.argtypes, L.gdn_read_layer_status.restype = [_VP], _INT
        _bound = L
    return _bound


def _launch(what: str, device, args, workspace_size=None):
    """Call ``what`` on the current stream of ``device``, with a workspace of the size it asks for."""
    L = _library()
    index = device.index
    if index == torch.cuda.current_device():
        return _launch_here(L, what, index, args, workspace_size)
    with torch.cuda.device(device):
        return _launch_here(L, what, index, args, workspace_size)


def _launch_here(L, what, index, args, workspace_size):
    stream = torch._C._cuda_getCurrentRawStream(index)
    ref = ctypes.byref(args)
    if workspace_size is None:
        code = getattr(L, what)(ref, stream)
    else:
        need = getattr(L, workspace_size)(ref)
        if need:
            ws = torch.empty(need, dtype=torch.uint8, device=torch.device("cuda", index))
            code = getattr(L, what)(ref, ws.data_ptr(), need, stream)
        else:
            code = getattr(L, what)(ref, None, 0, stream)
    if code != 0:
        raise GdnError(code, what)


def _cuda(name, t, device=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the input on {device}")


def _rows(name, t, width, rows=None):
    """(tensor, rows, row stride) of ``t`` as a matrix of ``width`` columns: as it is when its rows are
    contiguous and evenly spaced, else a contiguous copy."""
    if t.dim() == 0 or t.shape[-1] != width:
        raise ValueError(f"{name} must have {width} columns, got shape {tuple(t.shape)}")
    n = t.numel() // width
    if rows is not None and n != rows:
        raise ValueError(f"{name} has {n} rows, expected {rows}")
    if t.dim() == 2 and t.stride(1) == 1 and t.stride(0) >= width:
        return t, n, t.stride(0)
    if t.is_contiguous():
        return t, n, width
    if t.dim() > 2 and t.stride(-1) == 1 and t.stride(-2) >= width and all(
            t.stride(i) == t.stride(i + 1) * t.shape[i + 1] for i in range(t.dim() - 2)):
        return t, n, t.stride(-2)
    return t.contiguous(), n, width


def _vector(name, t, n, device, dtypes):
    _cuda(name, t, device)
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.numel() != n:
        raise ValueError(f"{name} must have {n} elements, got {t.numel()}")
    return t.contiguous()


def _out(name, t, shape, dtype, device):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if t.shape != torch.Size(shape) or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return t


_REAL = (torch.float32, torch.bfloat16)


def _norm(x, weight, residual, eps, quant, out, residual_out):
    _cuda("x", x)
    if x.dtype not in _REAL:
        raise TypeError(f"x must be float32 or bfloat16, got {x.dtype}")
    width = x.shape[-1] if x.dim() else 0
    if width < 1:
        raise ValueError("x must have at least one column")
    dev = x.device
    xr, n, ldx = _rows("x", x, width)
    a = GdnNormArgs(n, width, _CODE[x.dtype], GDN_F32, GDN_E4M3 if quant else _CODE[x.dtype], eps, xr.data_ptr(), ldx)
    keep = [xr]
    if weight is not None:
        w = _vector("weight", weight, width, dev, _REAL)
        a.weight, a.w_dtype = w.data_ptr(), _CODE[w.dtype]
        keep.append(w)
    h = None
    if residual is not None:
        _cuda("residual", residual, dev)
        if residual.dtype != x.dtype:
            raise TypeError("x and residual must share a dtype")
        if residual.shape != x.shape:
            raise ValueError("x and residual must share a shape")
        rr, _, ldr = _rows("residual", residual, width, n)
        a.residual, a.ld_residual = rr.data_ptr(), ldr
        h = _out("residual_out", residual_out, x.shape, x.dtype, dev)
        a.h = h.data_ptr()
        keep.append(rr)
    y = _out("out", out, x.shape, torch.float8_e4m3fn if quant else x.dtype, dev)
    a.y = y.data_ptr()
    scale = None
    if quant:
        scale = torch.empty(x.shape[:-1], dtype=torch.float32, device=dev)
        a.scale = scale.data_ptr()
    _launch("gdn_rms_norm", dev, a)
    return y, scale, h


def rms_norm(x, weight=None, residual=None, eps=1e-6, *, out=None, residual_out=None):
    """Root-mean-square norm with the residual's addition in front: ``h = x + residual``,
    ``y = weight * h / sqrt(mean(h^2) + eps)`` over the last dimension, in fp32, rounded once.

    x, residual [..., D] float32 or bfloat16 (same dtype); weight [D] float32 or bfloat16, or None.
    Returns ``(y, h)``: both in x's dtype, ``h`` None without a residual.  ``residual_out`` may be
    ``residual`` itself (the residual stream updated in place)."""
    y, _, h = _norm(x, weight, residual, eps, False, out, residual_out)
    return y, h


def rms_norm_quant(x, weight=None, residual=None, eps=1e-6, *, out=None, residual_out=None):
    """:func:`rms_norm` with its output in 8 bits: returns ``(q, scale, h)``, q [..., D] float8_e4m3fn and
    scale [...] float32 with ``y ~ scale[..., None] * q`` (scale = max(max|y| / 448, 2^-126) per row)."""
    return _norm(x, weight, residual, eps, True, out, residual_out)


def quantize_rows(x, *, out=None):
    """``(q, scale)``: x [..., D] (float32 or bfloat16) in 8 bits with one scale per row, as
    :func:`rms_norm_quant` gives; for weights, once, and for activations that no norm precedes."""
    _cuda("x", x)
    if x.dtype not in _REAL:
        raise TypeError(f"x must be float32 or bfloat16, got {x.dtype}")
    width = x.shape[-1] if x.dim() else 0
    if width < 1:
        raise ValueError("x must have at least one column")
    xr, n, ldx = _rows("x", x, width)
    q = _out("out", out, x.shape, torch.float8_e4m3fn, x.device)
    scale = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    a = GdnNormArgs(n, width, _CODE[x.dtype], GDN_F32, GDN_E4M3, 0.0, xr.data_ptr(), ldx)
    a.y, a.scale = q.data_ptr(), scale.data_ptr()
    _launch("gdn_quantize_rows", x.device, a)
    return q, scale


def rms_norm_bwd(dy, h, weight=None, dh=None, eps=1e-6):
    """Gradients of :func:`rms_norm`: ``h`` is what it normalised (x + residual), ``dh`` (or None) the gradient
    that reaches h past the norm (the residual stream's).  Returns ``(dx, dweight)``: dx in h's dtype, the
    gradient of x and of residual; dweight [D] float32 (None without a weight)."""
    for name, t in (("h", h), ("dy", dy)) + ((("dh", dh),) if dh is not None else ()):
        _cuda(name, t, h.device)
        if t.dtype != h.dtype or t.shape != h.shape:
            raise ValueError(f"{name} must share h's dtype and shape")
    if h.dtype not in _REAL:
        raise TypeError(f"h must be float32 or bfloat16, got {h.dtype}")
    width = h.shape[-1] if h.dim() else 0
    if width < 1:
        raise ValueError("h must have at least one column")
    hr, n, ldh = _rows("h", h, width)
    dyr, _, ldy = _rows("dy", dy, width, n)
    a = GdnNormArgs(n, width, _CODE[h.dtype], GDN_F32, _CODE[h.dtype], eps, hr.data_ptr(), ldh)
    a.dy, a.ld_dy = dyr.data_ptr(), ldy
    if dh is not None:
        dhr, _, a.ld_dh = _rows("dh", dh, width, n)
        a.dh = dhr.data_ptr()
    dx = torch.empty(h.shape, dtype=h.dtype, device=h.device)
    a.dx = dx.data_ptr()
    dw = None
    if weight is not None:
        w = _vector("weight", weight, width, h.device, _REAL)
        a.weight, a.w_dtype = w.data_ptr(), _CODE[w.dtype]
        dw = torch.empty(width, dtype=torch.float32, device=h.device)
        a.dweight = dw.data_ptr()
    _launch("gdn_rms_norm_bwd", h.device, a, "gdn_rms_norm_bwd_workspace_size")
    return dx, dw


def _linear_args(x, weight, activation, x_scale, weight_scale, halves):
    """The inputs shared by the four calls, and the tensors that have to outlive the launch."""
    _cuda("x", x)
    dev, dt = x.device, x.dtype
    _cuda("weight", weight, dev)
    if dt not in _CODE:
        raise TypeError(f"x must be float32, bfloat16 or float8_e4m3fn, got {dt}")
    if weight.dtype != dt:
        raise TypeError("x and weight must share a dtype")
    if weight.dim() != 2 or weight.shape[0] < 1 or weight.shape[1] < 1 or weight.shape[0] % halves:
        raise ValueError(f"weight must be [{'2 F' if halves == 2 else 'N'}, K], got shape {tuple(weight.shape)}")
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {[k for k in ACTIVATIONS if k]} or None, got {activation!r}")
    N, K = weight.shape
    xr, M, ldx = _rows("x", x, K)
    wr, _, ldw = _rows("weight", weight, K)
    a = GdnLinearArgs(M, N // halves, K, _CODE[dt], GDN_F32 if dt == torch.float32 else GDN_BF16,
                      ACTIVATIONS[activation], xr.data_ptr(), ldx, wr.data_ptr(), ldw)
    keep = [xr, wr]
    if (x_scale is None) != (weight_scale is None):
        raise ValueError("x_scale and weight_scale go together")
    if x_scale is not None:
        if dt != torch.float8_e4m3fn:
            raise TypeError("scales go with float8_e4m3fn inputs")
        xs = _vector("x_scale", x_scale, M, dev, (torch.float32,))
        ws = _vector("weight_scale", weight_scale, N, dev, (torch.float32,))
        a.x_scale, a.w_scale = xs.data_ptr(), ws.data_ptr()
        keep += [xs, ws]
    return a, keep, M


def linear(x, weight, bias=None, activation=None, residual=None, *, x_scale=None, weight_scale=None, out_dtype=None,
           out=None):
    """``y = act(x weight^T + bias) + residual``, the epilogue on the fp32 sums, rounded once.

    x [..., K] and weight [N, K] bfloat16, float32 or float8_e4m3fn (with ``x_scale`` [...] and
    ``weight_scale`` [N] float32, as :func:`rms_norm_quant` and :func:`quantize_rows` give them); bias [N]
    float32; activation None, "silu", "gelu", "gelu_tanh", "relu" or "sigmoid"; residual [..., N] in the output's
    dtype.  The output is float32 for float32 inputs, else bfloat16 or, with ``out_dtype``, float32.  ``out`` may
    be ``residual`` itself."""
    a, keep, M = _linear_args(x, weight, activation, x_scale, weight_scale, 1)
    N, dev = weight.shape[0], x.device
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.float32 if x.dtype == torch.float32 else torch.bfloat16
    if out_dtype not in _REAL or (x.dtype == torch.float32 and out_dtype != torch.float32):
        raise TypeError(f"out_dtype {out_dtype} is not available for {x.dtype} inputs")
    a.out_dtype = _CODE[out_dtype]
    if bias is not None:
        b = _vector("bias", bias, N, dev, (torch.float32,))
        a.bias = b.data_ptr()
        keep.append(b)
    if residual is not None:
        _cuda("residual", residual, dev)
        if residual.dtype != out_dtype:
            raise TypeError(f"residual must be {out_dtype}, the output's dtype")
        rr, _, a.ld_residual = _rows("residual", residual, N, M)
        a.residual = rr.data_ptr()
        keep.append(rr)
    y = _out("out", out, (*x.shape[:-1], N), out_dtype, dev)
    a.y, a.ldy = y.data_ptr(), N
    _launch("gdn_linear", dev, a, "gdn_linear_workspace_size")
    return y


def linear_bwd(dy, x, weight, bias=None, activation=None, *, need_dx=True, need_dweight=True):
    """Gradients of :func:`linear` (float32 or bfloat16): returns ``(dx, dweight, dbias)`` in the dtypes of x,
    weight and float32 (dbias None without a bias; the residual's gradient is dy).  With an activation the
    pre-activation is recomputed."""
    if x.dtype not in _REAL:
        raise TypeError(f"x must be float32 or bfloat16, got {x.dtype}")
    a, keep, M = _linear_args(x, weight, activation, None, None, 1)
    N, K = weight.shape
    dev = x.device
    _cuda("dy", dy, dev)
    if dy.dtype != x.dtype:
        raise TypeError("dy and x must share a dtype")
    dyr, _, a.ld_dy = _rows("dy", dy, N, M)
    a.dy = dyr.data_ptr()
    dx = torch.empty(x.shape, dtype=x.dtype, device=dev) if need_dx else None
    dw = torch.empty((N, K), dtype=x.dtype, device=dev) if need_dweight else None
    db = None
    if bias is not None:
        b = _vector("bias", bias, N, dev, (torch.float32,))
        a.bias = b.data_ptr()
        keep.append(b)
        db = torch.empty(N, dtype=torch.float32, device=dev)
        a.dbias = db.data_ptr()
    a.dx = dx.data_ptr() if need_dx else None
    a.dw = dw.data_ptr() if need_dweight else None
    _launch("gdn_linear_bwd", dev, a, "gdn_linear_bwd_workspace_size")
    return dx, dw, db


def gated_linear(x, weight, activation="silu", *, x_scale=None, weight_scale=None, out=None):
    """Gated linear unit in one kernel: ``act(x Wg^T) * (x Wu^T)`` with weight [2F, K] = [Wg; Wu].  dtypes and
    scales as :func:`linear`; the output [..., F] is float32 for float32 inputs, else bfloat16."""
    a, keep, M = _linear_args(x, weight, activation, x_scale, weight_scale, 2)
    F = weight.shape[0] // 2
    y = _out("out", out, (*x.shape[:-1], F), torch.float32 if x.dtype == torch.float32 else torch.bfloat16, x.device)
    a.y, a.ldy = y.data_ptr(), F
    _launch("gdn_gated_linear", x.device, a, "gdn_gated_linear_workspace_size")
    return y


def gated_linear_bwd(dy, x, weight, activation="silu", *, need_dx=True, need_dweight=True, return_output=False):
    """Gradients of :func:`gated_linear` (float32 or bfloat16) from its inputs and ``dy`` [..., F]; the
    projections are recomputed.  Returns ``(dx, dweight)``, and with ``return_output`` also the recomputed
    output (the following layer's input, which then need not be kept)."""
    if x.dtype not in _REAL:
        raise TypeError(f"x must be float32 or bfloat16, got {x.dtype}")
    a, keep, M = _linear_args(x, weight, activation, None, None, 2)
    F = weight.shape[0] // 2
    dev = x.device
    _cuda("dy", dy, dev)
    if dy.dtype != x.dtype:
        raise TypeError("dy and x must share a dtype")
    dyr, _, a.ld_dy = _rows("dy", dy, F, M)
    a.dy = dyr.data_ptr()
    dx = torch.empty(x.shape, dtype=x.dtype, device=dev) if need_dx else None
    dw = torch.empty(weight.shape, dtype=x.dtype, device=dev) if need_dweight else None
    a.dx = dx.data_ptr() if need_dx else None
    a.dw = dw.data_ptr() if need_dweight else None
    y = None
    if return_output:
        y = torch.empty((*x.shape[:-1], F), dtype=x.dtype, device=dev)
        a.y, a.ldy = y.data_ptr(), F
    _launch("gdn_gated_linear_bwd", dev, a, "gdn_gated_linear_bwd_workspace_size")
    return (dx, dw, y) if return_output else (dx, dw)


def read_layer_status(device=None) -> int:
    """Synchronise the current stream; the status that device-side waits of these operators recorded since the
    last call (0, or -4 for a wait that ran out), cleared."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(dev):
        return int(_library().gdn_read_layer_status(torch.cuda.current_stream(dev).cuda_stream))
