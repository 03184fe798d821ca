"""Gated feed-forward block: argument marshalling for ``mla_gated_ffn_fwd``
and ``mla_gated_ffn_bwd`` (declared in ``include/mlaq.h``).

y = (act(x Wg^T) * (x Wu^T)) Wd^T with Wg and Wu stacked in ``w_gate_up``
[2F, K], and its gradients.
"""
from __future__ import annotations

import ctypes

import torch

import up_proj_gemm_gb300 as _pkg

from . import _call, _empty, _need, _ptr, _SIGS, _status, _stream, lib

__all__ = ["FfnShape", "ACTIVATIONS", "gated_ffn_fwd", "gated_ffn_bwd"]

ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}
_bf16 = torch.bfloat16


class FfnShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("K", ctypes.c_int64), ("F", ctypes.c_int64), ("ld_x", ctypes.c_int64),
                ("act", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_vp, _int = ctypes.c_void_p, ctypes.c_int
_SIGS.update({
    "mla_gated_ffn_fwd": (_int, [ctypes.POINTER(FfnShape)] + [_vp] * 8),
    "mla_gated_ffn_bwd": (_int, [ctypes.POINTER(FfnShape)] + [_vp] * 12),
})


def _rows(t, name, dev=None, T=None, K=None):
    """A bf16 matrix with contiguous rows; its row pitch in elements."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != _bf16:
        raise TypeError(f"{name} must be {_bf16}, got {t.dtype}")
    if t.dim() != 2 or (T is not None and tuple(t.shape) != (T, K)):
        raise ValueError(f"{name} must be {[T, K] if T is not None else 'a matrix'}, got {list(t.shape)}")
    if not t.is_cuda or (dev is not None and t.device != dev):
        raise ValueError(f"{name} is on {t.device}, expected {dev or 'a CUDA device'}")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit inner stride")
    if rows > 1 and t.stride(0) < cols:  # a row for all tokens, too: pitch 0 would say dense
        raise ValueError(f"{name} must have rows that do not overlap, got a pitch of {t.stride(0)} for {cols} elements")
    return t.stride(0) if rows > 1 else cols


def _act(act):
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}, got {act!r}")
    return ACTIVATIONS[act]


def gated_ffn_fwd(x, w_gate_up, w_down, act="silu", save=False, gate_up=None, h=None, y=None, status=None,
                  stream=None):
    """y [T, K] bf16 = (act(g) * u) w_down^T with [g | u] = x w_gate_up^T.

    x [T, K] bf16 (rows may have a pitch of K or more), w_gate_up [2F, K] bf16 (F gate
    rows, then F up rows), w_down [K, F] bf16; act "silu", "gelu" or
    "gelu_tanh". save=True returns (y, gate_up [T, 2F], h [T, F]), what
    gated_ffn_bwd needs. h is also the scratch of the second product."""
    a = _act(act)
    c = _pkg._calls
    if c is not None and gate_up is None and h is None and y is None and status is None and stream is None:
        r = c.ffn_fwd(x, w_gate_up, w_down, a, save)
        if r is not None:
            return r
    ld = _rows(x, "x")
    T, K = x.shape
    dev = x.device
    _need(w_down, "w_down", _bf16, dev, ndim=2)
    F = w_down.shape[1]
    _need(w_down, "w_down", _bf16, dev, shape=(K, F))
    _need(w_gate_up, "w_gate_up", _bf16, dev, shape=(2 * F, K))
    _status(status, dev)
    if y is None:
        y = _empty((T, K), _bf16, dev, stream)
    else:
        _need(y, "y", _bf16, dev, shape=(T, K))
    if h is None:
        h = _empty((T, F), _bf16, dev, stream, scratch=not save)
    else:
        _need(h, "h", _bf16, dev, shape=(T, F))
    if gate_up is not None:
        _need(gate_up, "gate_up", _bf16, dev, shape=(T, 2 * F))
    elif save:
        gate_up = _empty((T, 2 * F), _bf16, dev, stream)
    s = FfnShape(T, K, F, ld, a, 0)
    _call(lib().mla_gated_ffn_fwd, "mla_gated_ffn_fwd", ctypes.byref(s), _ptr(x), _ptr(w_gate_up), _ptr(w_down),
          _ptr(gate_up), _ptr(h), _ptr(y), _ptr(status), _stream(dev, stream))
    return (y, gate_up, h) if save else y


def gated_ffn_bwd(dy, x, w_gate_up, w_down, gate_up, h, act="silu", dx=True, dw_gate_up=True, dw_down=True,
                  dgate_up=None, status=None, stream=None):
    """(dx [T, K], dw_gate_up [2F, K], dw_down [K, F]) in bf16 from dy [T, K]
    bf16, the forward's inputs and its saved gate_up and h.

    Each of dx / dw_gate_up / dw_down: True allocates it, False/None skips it
    (None comes back), or pass a tensor. Inputs that no requested gradient
    needs may be None: w_gate_up without dx, x without dw_gate_up, h without
    dw_down, w_down and gate_up without both dx and dw_gate_up. ``dgate_up``
    [T, 2F], the gradient of gate_up, is allocated unless passed."""
    a = _act(act)
    c = _pkg._calls
    if (c is not None and dx is True and dw_gate_up is True and dw_down is True and dgate_up is None and status is None
            and stream is None):
        r = c.ffn_bwd(dy, x, w_gate_up, w_down, gate_up, h, a)
        if r is not None:
            return r
    if not isinstance(dy, torch.Tensor) or dy.dim() != 2:
        raise ValueError("dy must be a bf16 CUDA matrix [T, K]")
    T, K = dy.shape
    dev = dy.device
    _need(dy, "dy", _bf16, ndim=2)
    want_dx, want_gu, want_d = (t is not None and t is not False for t in (dx, dw_gate_up, dw_down))
    if not (want_dx or want_gu or want_d):
        raise ValueError("no gradient is requested")
    hidden = want_dx or want_gu
    if hidden:
        _need(w_down, "w_down", _bf16, dev, ndim=2)
        F = w_down.shape[1]
        _need(w_down, "w_down", _bf16, dev, shape=(K, F))
        _need(gate_up, "gate_up", _bf16, dev, shape=(T, 2 * F))
    else:
        _need(h, "h", _bf16, dev, ndim=2)
        F = h.shape[1]
    ld = 0
    if want_dx:
        _need(w_gate_up, "w_gate_up", _bf16, dev, shape=(2 * F, K))
    if want_gu:
        ld = _rows(x, "x", dev, T, K)
    if want_d:
        _need(h, "h", _bf16, dev, shape=(T, F))
    _status(status, dev)
    if hidden:
        if dgate_up is None:
            dgate_up = _empty((T, 2 * F), _bf16, dev, stream, scratch=True)
        else:
            _need(dgate_up, "dgate_up", _bf16, dev, shape=(T, 2 * F))
    outs = []
    for name, t, want, shape in (("dx", dx, want_dx, (T, K)), ("dw_gate_up", dw_gate_up, want_gu, (2 * F, K)),
                                 ("dw_down", dw_down, want_d, (K, F))):
        if not want:
            t = None
        elif t is True:
            t = _empty(shape, _bf16, dev, stream)
        else:
            _need(t, name, _bf16, dev, shape=shape)
        outs.append(t)
    s = FfnShape(T, K, F, ld, a, 0)
    _call(lib().mla_gated_ffn_bwd, "mla_gated_ffn_bwd", ctypes.byref(s), _ptr(dy), _ptr(x if want_gu else None),
          _ptr(w_gate_up if want_dx else None), _ptr(w_down if hidden else None), _ptr(gate_up if hidden else None),
          _ptr(h if want_d else None), _ptr(dgate_up if hidden else None), _ptr(outs[0]), _ptr(outs[1]),
          _ptr(outs[2]), _ptr(status), _stream(dev, stream))
    return tuple(outs)
