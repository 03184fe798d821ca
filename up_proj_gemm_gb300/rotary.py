"""Rotary positions with several axes: argument marshalling for
``mla_rope_axes`` and ``mla_rope_axes_table`` (declared in ``include/mlaq.h``).

Pair i of a head (rope channels i and i + Dr/2) of token t is turned by row
``pos[axes[i], t]`` of the cos/sin tables, so the time, height and width of an
image or video token each turn their own pairs. ``axes`` is a sequence of
Dr/2 axis numbers; ``rope_sections((16, 8, 8))`` gives the one for contiguous
sections.
"""
from __future__ import annotations

import ctypes
import operator

import torch

import up_proj_gemm_gb300 as _pkg

from . import _call, _empty, _need, _ptr, _SIGS, _status, _stream, lib

__all__ = ["RopeAxesShape", "rope_sections", "rope_axes", "rope_axes_table"]


class RopeAxesShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int32), ("Dn", ctypes.c_int32), ("Dr", ctypes.c_int32),
                ("axes", ctypes.c_int32), ("cs_rows", ctypes.c_int64), ("cs_width", ctypes.c_int64),
                ("in_t", ctypes.c_int64), ("in_h", ctypes.c_int64), ("out_t", ctypes.c_int64),
                ("out_h", ctypes.c_int64), ("reserved", ctypes.c_int64)]


_vp, _int = ctypes.c_void_p, ctypes.c_int
_SIGS.update({
    "mla_rope_axes": (_int, [ctypes.POINTER(RopeAxesShape), _int, _int, _vp, _vp, _vp, _vp, ctypes.c_char_p, _vp,
                             _vp, _vp]),
    "mla_rope_axes_table": (_int, [ctypes.POINTER(RopeAxesShape), _vp, _vp, _vp, ctypes.c_char_p, _vp, _vp, _vp,
                                   _vp]),
})


def rope_sections(sections) -> bytes:
    """The axis of every pair when axis a turns the next sections[a] pairs."""
    return bytes(a for a, n in enumerate(sections) for _ in range(n))


def _axes(axes, Dr):
    """The pairs' axes as one byte each: from bytes, or a sequence of Dr/2 integers (an integer alone or an array's
    memory would be other bytes)."""
    if type(axes) is not bytes:
        axes = bytes(axes if type(axes) in (list, tuple) else [operator.index(a) for a in axes])
    if len(axes) != Dr // 2:
        raise ValueError(f"axes must name the axis of each of the {Dr // 2} pairs, got {len(axes)}")
    return axes


_bf16, _f32, _i32 = torch.bfloat16, torch.float32, torch.int32


def _refuse_tables(cos, sin, pos, T, dev):
    """Name what is wrong with the tables or the positions [A, T]."""
    _need(cos, "cos", _f32, dev, ndim=2)
    _need(sin, "sin", _f32, dev, shape=cos.shape)
    _need(pos, "pos", _i32, dev, ndim=2)
    if pos.shape[1] != T:
        raise ValueError(f"pos must be [axes, {T}], got {list(pos.shape)}")


def _tables_ok(cos, sin, pos, T, dev):
    """The checks of _refuse_tables in one expression: a call's checks cost as much as its launch."""
    return (isinstance(cos, torch.Tensor) and isinstance(sin, torch.Tensor) and isinstance(pos, torch.Tensor)
            and cos.dtype is _f32 and sin.dtype is _f32 and pos.dtype is _i32 and cos.dim() == 2
            and sin.shape == cos.shape and pos.dim() == 2 and pos.shape[1] == T
            and cos.is_cuda and sin.is_cuda and pos.is_cuda
            and cos.device == dev and sin.device == dev and pos.device == dev
            and cos.is_contiguous() and sin.is_contiguous() and pos.is_contiguous())


def _refuse_x(x, Dr, inverse, sum_heads):
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if x.dtype not in (_bf16, _f32):
        raise TypeError(f"x must be bfloat16 or float32, got {x.dtype}")
    if not x.is_cuda or x.dim() != 3 or (x.shape[2] > 1 and x.stride(2) != 1):
        raise ValueError("x must be a 3-D CUDA tensor [T, H, D] with unit inner stride")
    if sum_heads and not inverse:
        raise ValueError("sum_heads sums gradients: it needs inverse=True")
    raise ValueError(f"Dr must be in 1..{x.shape[2]}, got {Dr}")


def rope_axes(x, cos, sin, pos, axes, Dr, inverse=False, sum_heads=False, out=None, status=None, stream=None):
    """x [T, H, D] (bf16 or float32, any token and head strides, contiguous
    channels) with the last Dr channels of every head rotated; the others are
    copied.

    pos: int32 [A, T]; axes: the axis of each of the Dr/2 pairs, as bytes or a
    sequence of integers. ``inverse`` applies the Jacobian transpose (the
    gradient), ``sum_heads`` (with inverse) the transpose of the heads' sum,
    [T, 1, D]: the gradient of a key part that all heads share. ``out`` may be
    a strided view."""
    axes = _axes(axes, Dr)
    c = _pkg._calls
    if c is not None and out is None and status is None and stream is None and (inverse or not sum_heads):
        out = c.rope_axes(x, cos, sin, pos, axes, Dr, (2 if sum_heads else 1) if inverse else 0)
        if out is not None:
            return out
    if not (isinstance(x, torch.Tensor) and (x.dtype is _bf16 or x.dtype is _f32) and x.is_cuda and x.dim() == 3
            and (x.shape[2] <= 1 or x.stride(2) == 1) and (inverse or not sum_heads) and 0 < Dr <= x.shape[2]):
        _refuse_x(x, Dr, inverse, sum_heads)
    T, H, D = x.shape
    in_t, in_h, _ = x.stride()
    dev = x.device
    if not _tables_ok(cos, sin, pos, T, dev):
        _refuse_tables(cos, sin, pos, T, dev)
    if status is not None:
        _status(status, dev)
    Ho = 1 if sum_heads else H
    if out is None:
        out = _empty((T, Ho, D), x.dtype, dev, stream)
        out_t, out_h = Ho * D, D
    else:
        if not isinstance(out, torch.Tensor) or out.dtype is not x.dtype:
            raise TypeError(f"out must be a {x.dtype} tensor")
        if tuple(out.shape) != (T, Ho, D):
            raise ValueError(f"out must be {[T, Ho, D]}, got {list(out.shape)}")
        if not out.is_cuda or out.device != dev or (D > 1 and out.stride(2) != 1):
            raise ValueError(f"out must be on {dev} with unit inner stride")
        out_t, out_h = out.stride(0), out.stride(1)
    rows, width = cos.shape
    s = RopeAxesShape(T, H, D - Dr, Dr, pos.shape[0], rows, width, in_t if T > 1 else 0, in_h if H > 1 else 0,
                      out_t if T > 1 else 0, out_h if Ho > 1 else 0, 0)
    _call(lib().mla_rope_axes, "mla_rope_axes", ctypes.byref(s), 0 if x.dtype is _f32 else 1,
          (2 if sum_heads else 1) if inverse else 0, x.data_ptr(), cos.data_ptr(), sin.data_ptr(), pos.data_ptr(),
          axes, out.data_ptr(), _ptr(status), _stream(dev, stream))
    return out


def rope_axes_table(cos, sin, pos, axes, Dr, cos_out=None, sin_out=None, status=None, stream=None):
    """(cos, sin) float32 [T, Dr] of every token for positions with several
    axes: the tables to give fwd, bwd_dgrad, bwd_wgrad, bwd_mxfp8 and kv_fwd
    (with pos=None), which then rotate by several axes."""
    axes = _axes(axes, Dr)
    c = _pkg._calls
    if c is not None and cos_out is None and sin_out is None and status is None and stream is None:
        r = c.rope_axes_table(cos, sin, pos, axes, Dr)
        if r is not None:
            return r
    if not isinstance(pos, torch.Tensor) or pos.dim() != 2:
        raise ValueError("pos must be an int32 tensor [A, T]")
    dev = pos.device
    A, T = pos.shape
    if not _tables_ok(cos, sin, pos, T, dev):
        _refuse_tables(cos, sin, pos, T, dev)
    if status is not None:
        _status(status, dev)
    if cos_out is None:
        cos_out = _empty((T, Dr), _f32, dev, stream)
    else:
        _need(cos_out, "cos_out", _f32, dev, shape=(T, Dr))
    if sin_out is None:
        sin_out = _empty((T, Dr), _f32, dev, stream)
    else:
        _need(sin_out, "sin_out", _f32, dev, shape=(T, Dr))
    rows, width = cos.shape
    s = RopeAxesShape(T, 1, 0, Dr, A, rows, width, 0, 0, 0, 0, 0)
    _call(lib().mla_rope_axes_table, "mla_rope_axes_table", ctypes.byref(s), cos.data_ptr(), sin.data_ptr(),
          pos.data_ptr(), axes, cos_out.data_ptr(), sin_out.data_ptr(), _ptr(status), _stream(dev, stream))
    return cos_out, sin_out
