"""RMS norm of token rows, with the residual's addition and an MXFP8 result:
argument marshalling for ``mla_rms_norm_fwd`` and ``mla_rms_norm_bwd``
(declared in ``include/mlaq.h``).

h = x + residual, y = h rstd weight with rstd = (mean(h^2) + eps)^(-1/2), and
its gradients. The MXFP8 results are the x operands of ``fwd`` with MXFP8
weights.
"""
from __future__ import annotations

import ctypes
import math

import torch

import up_proj_gemm_gb300 as _pkg

from . import _call, _empty, _need, _ptr, _SIGS, _stream, lib

__all__ = ["NormShape", "NORM_OUTS", "rms_norm_fwd", "rms_norm_bwd"]

NORM_OUTS = {"same": 0, "mxfp8": 1, "tiled": 2}
_FLOATS = {torch.float32: 0, torch.bfloat16: 1}


class NormShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("K", ctypes.c_int64), ("ld_x", ctypes.c_int64), ("ld_res", ctypes.c_int64),
                ("ld_dy", ctypes.c_int64), ("dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32),
                ("out_mode", ctypes.c_int32), ("eps", ctypes.c_float), ("reserved", ctypes.c_int64)]


_vp, _int = ctypes.c_void_p, ctypes.c_int
_SIGS.update({
    "mla_rms_norm_fwd": (_int, [ctypes.POINTER(NormShape)] + [_vp] * 8),
    "mla_rms_norm_bwd_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(NormShape)]),
    "mla_rms_norm_bwd": (_int, [ctypes.POINTER(NormShape)] + [_vp] * 8 + [ctypes.c_size_t, _vp]),
})


def _rows(t, name, like=None):
    """A float32 or bf16 matrix with contiguous rows that do not overlap, of `like`'s type, shape and device; its row
    pitch in elements."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _FLOATS or (like is not None and t.dtype is not like.dtype):
        raise TypeError(f"{name} must be {like.dtype if like is not None else 'float32 or bfloat16'}, got {t.dtype}")
    if t.dim() != 2 or (like is not None and t.shape != like.shape):
        raise ValueError(f"{name} must be {list(like.shape) if like is not None else 'a matrix'}, got {list(t.shape)}")
    if not t.is_cuda or (like is not None and t.device != like.device):
        raise ValueError(f"{name} is on {t.device}, expected {like.device if like is not None else 'a CUDA device'}")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit inner stride")
    if rows > 1 and t.stride(0) < cols:
        raise ValueError(f"{name} must have rows that do not overlap, got a pitch of {t.stride(0)} for {cols} elements")
    return t.stride(0) if rows > 1 else cols


def _weight(w, K, dev):
    if isinstance(w, torch.Tensor) and w.dtype not in _FLOATS:
        raise TypeError(f"weight must be float32 or bfloat16, got {w.dtype}")
    _need(w, "weight", w.dtype if isinstance(w, torch.Tensor) else None, dev, shape=(K,))
    return _FLOATS[w.dtype]


def _eps(eps):
    eps = float(eps)
    if not (eps >= 0 and math.isfinite(eps)):
        raise ValueError(f"eps must be finite and not negative, got {eps}")
    return eps


def rms_norm_fwd(x, weight, eps=1e-6, residual=None, out="same", save=False, y=None, scales=None, h=None, rstd=None,
                 stream=None):
    """y = h rstd weight, h = x + residual, rstd = (mean(h^2) + eps)^(-1/2) of each row of x [T, K].

    x and residual are bf16 or float32 (one type; rows may have a pitch of K
    or more), weight [K] either. out "same": y in the type of x; "mxfp8": E4M3
    codes [T, K] and E8M0 scales [T, K/32] (uint8); "tiled": the codes and the
    scales flat in the block-scaled GEMM's tiled order, what ``fwd`` takes as
    x with weight_mode "mxfp8" and "mxfp8_tiled". Returns y; then the scales
    where there are some, h where a residual is given, and rstd [T] with
    save=True, as a tuple."""
    if out not in NORM_OUTS:
        raise ValueError(f"out must be one of {sorted(NORM_OUTS)}, got {out!r}")
    mode, eps = NORM_OUTS[out], _eps(eps)
    lib()
    c = _pkg._calls
    if c is not None and y is None and scales is None and h is None and rstd is None and stream is None:
        r = c.rms_norm_fwd(x, weight, eps, residual, mode, save)
        if r is not None:
            return r
    ld_x = _rows(x, "x")
    T, K = x.shape
    dev = x.device
    wt = _weight(weight, K, dev)
    ld_res = _rows(residual, "residual", x) if residual is not None else 0
    if residual is None and h is not None:
        raise ValueError("h is the sum with a residual: it goes with one")
    if mode == 0 and scales is not None:
        raise ValueError("scales go with an MXFP8 result")

    def result(t, name, dtype, shape):
        if t is None:
            return _empty(shape, dtype, dev, stream)
        _need(t, name, dtype, dev, shape=shape)
        return t

    outs = [result(y, "y", x.dtype if mode == 0 else torch.uint8, (T, K))]
    y = outs[0]
    if mode:
        kb = (K + 31) // 32
        n = -(-T // 128) * -(-kb // 4) * 512
        scales = result(scales, "scales", torch.uint8, (T, kb) if mode == 1 else (n,))
        outs.append(scales)
    if residual is not None:
        h = result(h, "h", x.dtype, (T, K))
        outs.append(h)
    if save or rstd is not None:
        rstd = result(rstd, "rstd", torch.float32, (T,))
        outs.append(rstd)
    s = NormShape(T, K, ld_x, ld_res, 0, _FLOATS[x.dtype], wt, mode, eps, 0)
    _call(lib().mla_rms_norm_fwd, "mla_rms_norm_fwd", ctypes.byref(s), _ptr(x), _ptr(residual), _ptr(weight), _ptr(h),
          _ptr(y), _ptr(scales), _ptr(rstd), _stream(dev, stream))
    return tuple(outs) if len(outs) > 1 else y


def rms_norm_bwd(dy, h, weight, rstd, dres=None, dx=True, dw=True, workspace=None, stream=None):
    """(dx [T, K], dw [K]) of ``rms_norm_fwd`` from dy, its h (x where it had no residual) and its rstd.

    dx is the gradient of x and of the residual alike; dres, the gradient that
    reaches h itself, is added to it. Each of dx / dw: True allocates it,
    False/None skips it (None comes back), or pass a tensor. dy, h and dres
    have one type (rows may have a pitch), dw has the weight's. The workspace
    (uint8) is allocated unless passed."""
    lib()
    c = _pkg._calls
    if c is not None and dx is True and dw is True and workspace is None and stream is None:
        r = c.rms_norm_bwd(dy, h, weight, rstd, dres)
        if r is not None:
            return r
    ld_x = _rows(h, "h")
    T, K = h.shape
    dev = h.device
    ld_dy = _rows(dy, "dy", h)
    ld_res = _rows(dres, "dres", h) if dres is not None else 0
    wt = _weight(weight, K, dev)
    _need(rstd, "rstd", torch.float32, dev, shape=(T,))
    want_dx, want_dw = (t is not None and t is not False for t in (dx, dw))
    if not (want_dx or want_dw):
        raise ValueError("no gradient is requested")
    if dres is not None and not want_dx:
        raise ValueError("dres is added to dx: it goes with one")
    outs = []
    for name, t, want, shape, dtype in (("dx", dx, want_dx, (T, K), h.dtype), ("dw", dw, want_dw, (K,), weight.dtype)):
        if not want:
            t = None
        elif t is True:
            t = _empty(shape, dtype, dev, stream)
        else:
            _need(t, name, dtype, dev, shape=shape)
        outs.append(t)
    s = NormShape(T, K, ld_x, ld_res, ld_dy, _FLOATS[h.dtype], wt, 0, 0.0, 0)
    if want_dw:
        if workspace is None:
            workspace = _empty((int(lib().mla_rms_norm_bwd_workspace_size(ctypes.byref(s))),), torch.uint8, dev, stream,
                               scratch=True)
        else:
            _need(workspace, "workspace", torch.uint8, dev, ndim=1)
    else:
        workspace = None
    _call(lib().mla_rms_norm_bwd, "mla_rms_norm_bwd", ctypes.byref(s), _ptr(dy), _ptr(h), _ptr(weight), _ptr(rstd),
          _ptr(dres), _ptr(outs[0]), _ptr(outs[1]), _ptr(workspace), 0 if workspace is None else workspace.numel(),
          _stream(dev, stream))
    return tuple(outs)
