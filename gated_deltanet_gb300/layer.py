"""The operators around the gated delta rule in a decoder block: the root-mean-square norm with the
residual's addition (optionally in 8 bits with a scale per row), the linear layer with its epilogue, the
gated linear unit of a feed-forward block, and their gradients (``gdn_rms_norm``, ``gdn_linear``,
``gdn_gated_linear`` and their ``_bwd`` in ``include/gdn.h``).

Tensors are CUDA tensors, every leading dimension is a row, the work runs on the current stream, and
gradients are explicit calls.  Inputs whose rows are contiguous are taken as they are, at any row stride
(slices of a fused projection); others are made contiguous first.  Outputs and temporary buffers come from
PyTorch's allocator, so the calls can be captured into a CUDA graph.  Argument marshalling is compiled
(``csrc/layer_binding.cpp``): a decoding step's calls are short.
"""
from __future__ import annotations

import importlib.machinery
import importlib.util
import os
import threading

import torch

from ._binding import GdnError, load_library
from . import build

ACTIVATIONS = {None: 0, "none": 0, "silu": 1, "gelu": 2, "gelu_tanh": 3, "relu": 4, "sigmoid": 5}

_lock = threading.Lock()
_module = None


def _load():
    global _module
    with _lock:
        if _module is None:
            load_library()
            p, how = build.binding_path(), "build it with `python -c 'import __graft_entry__ as g; g.build()'`"
            if not os.path.exists(p):
                raise ImportError(f"{os.path.basename(p)} not found at {p}; {how}")
            if build.built_for() != build.running():
                raise ImportError(f"{p} was built for {build.built_for()}, this is {build.running()}; {how}")
            loader = importlib.machinery.ExtensionFileLoader("_layer", p)
            m = importlib.util.module_from_spec(importlib.util.spec_from_loader("_layer", loader))
            loader.exec_module(m)
            m.set_error(GdnError)
            _module = m
    return _module


def _act(name):
    code = ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"activation must be one of {[k for k in ACTIVATIONS if k]} or None, got {name!r}")
    return code


def rms_norm(x, weight=None, residual=None, eps=1e-6, *, out=None, residual_out=None):
    """Root-mean-square norm with the residual's addition in front: ``h = x + residual``,
    ``y = weight * h / sqrt(mean(h^2) + eps)`` over the last dimension, in fp32, rounded once.

    x, residual [..., D] float32 or bfloat16 (same dtype); weight [D] float32 or bfloat16, or None.
    Returns ``(y, h)``: both in x's dtype, ``h`` None without a residual.  ``residual_out`` goes
    with a residual and may be ``residual`` itself (the residual stream updated in place)."""
    y, _, h = (_module or _load()).rms_norm(x, weight, residual, eps, False, out, residual_out)
    return y, h


def rms_norm_quant(x, weight=None, residual=None, eps=1e-6, *, out=None, residual_out=None):
    """:func:`rms_norm` with its output in 8 bits: returns ``(q, scale, h)``, q [..., D] float8_e4m3fn and
    scale [...] float32 with ``y ~ scale[..., None] * q`` (scale = max(max|y| / 448, 2^-126) per row)."""
    return (_module or _load()).rms_norm(x, weight, residual, eps, True, out, residual_out)


def quantize_rows(x, *, out=None):
    """``(q, scale)``: x [..., D] (float32 or bfloat16) in 8 bits with one scale per row, as
    :func:`rms_norm_quant` gives; for weights, once, and for activations that no norm precedes."""
    return (_module or _load()).quantize_rows(x, out)


def rms_norm_bwd(dy, h, weight=None, dh=None, eps=1e-6):
    """Gradients of :func:`rms_norm`: ``h`` is what it normalised (x + residual), ``dh`` (or None) the gradient
    that reaches h past the norm (the residual stream's).  Returns ``(dx, dweight)``: dx in h's dtype, the
    gradient of x and of residual; dweight [D] float32 (None without a weight)."""
    return (_module or _load()).rms_norm_bwd(dy, h, weight, dh, eps)


def linear(x, weight, bias=None, activation=None, residual=None, *, x_scale=None, weight_scale=None, out_dtype=None,
           out=None):
    """``y = act(x weight^T + bias) + residual``, the epilogue on the fp32 sums, rounded once.

    x [..., K] and weight [N, K] bfloat16, float32 or float8_e4m3fn (with ``x_scale`` [...] and
    ``weight_scale`` [N] float32, as :func:`rms_norm_quant` and :func:`quantize_rows` give them); bias [N]
    float32; activation None, "silu", "gelu", "gelu_tanh", "relu" or "sigmoid"; residual [..., N] in the output's
    dtype.  The output is float32 for float32 inputs, else bfloat16 or, with ``out_dtype``, float32.  ``out`` may
    be ``residual`` itself and overlap no other input."""
    f32 = None
    if out_dtype is not None:
        if out_dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"out_dtype must be float32 or bfloat16, got {out_dtype}")
        f32 = out_dtype == torch.float32
    return (_module or _load()).linear(x, weight, bias, _act(activation), residual, x_scale, weight_scale, f32, out)


def linear_bwd(dy, x, weight, bias=None, activation=None, *, need_dx=True, need_dweight=True):
    """Gradients of :func:`linear` (float32 or bfloat16): returns ``(dx, dweight, dbias)`` in the dtypes of x,
    weight and float32 (dbias None without a bias; the residual's gradient is dy).  With an activation the
    pre-activation is recomputed."""
    return (_module or _load()).linear_bwd(dy, x, weight, bias, _act(activation), need_dx, need_dweight)


def gated_linear(x, weight, activation="silu", *, x_scale=None, weight_scale=None, out=None):
    """Gated linear unit in one kernel: ``act(x Wg^T) * (x Wu^T)`` with weight [2F, K] = [Wg; Wu].  dtypes and
    scales as :func:`linear`; the output [..., F] is float32 for float32 inputs, else bfloat16."""
    return (_module or _load()).gated_linear(x, weight, _act(activation), x_scale, weight_scale, out)


def gated_linear_bwd(dy, x, weight, activation="silu", *, need_dx=True, need_dweight=True, return_output=False):
    """Gradients of :func:`gated_linear` (float32 or bfloat16) from its inputs and ``dy`` [..., F]; the
    projections are recomputed.  Returns ``(dx, dweight)``, and with ``return_output`` also the recomputed
    output (the following layer's input, which then need not be kept)."""
    got = (_module or _load()).gated_linear_bwd(dy, x, weight, _act(activation), need_dx, need_dweight, return_output)
    return got if return_output else got[:2]


def read_layer_status(device=None) -> int:
    """Synchronise the current stream; the status that device-side waits of these operators recorded since the
    last call (0, or -4 for a wait that ran out), cleared."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    return (_module or _load()).read_status(torch.cuda.current_device() if dev.index is None else dev.index)
