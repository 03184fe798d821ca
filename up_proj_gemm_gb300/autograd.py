"""Autograd face of the fused query up-projection (argument marshalling only).

TransformerEngine PR "Add a backwards linear function to be used with the
fused mla q up-proj": the layer is a PyTorch autograd function whose
backward runs the RoPE backward and then the linear backward with the saved
input. Megatron-LM PR "Fix fused MLA YaRN RoPE query kernel corrupting
upstream tensor in-place", discussion: the weight gradient uses the linear's
saved input x, not its output.

``q_up_proj(x, W, cos, sin, H, Dn, Dr, bias=None, pos=None)`` returns
q [T, H, Dn + Dr] bf16 = RoPE(x W^T + b). Its backward calls the library's
dgrad and wgrad entry points; dgrad hands the rotated rope channels to
wgrad. Only the gradients autograd asks for are computed. Every step runs in
the library's CUDA kernels; this module only moves tensors.

``q_up_proj_mxfp8(...)`` is the same layer with the MXFP8 query the pages'
module hands to attention (TransformerEngine PR "Add support for fused Q
Up-Proj GEMM/RoPE/Quant", flowchart: the fused up-projection emits an MXFP8
query, its scales go to the BHSD transpose and the GEMM swizzle, attention
may return a BF16 dQ). E4M3 codes and E8M0 scales are integer tensors that
autograd cannot differentiate, so the result is an ``Mxfp8Query``: the codes,
the scales (in the out_mode's layout) and an ``anchor``, a 0-d float tensor
that carries the graph. The consumer hands back the bf16 gradient of the
query with ``query.backward(dq)``; that runs this layer's backward, like
``q.backward(dq)`` on the bf16 face.

``rope_axes(x, cos, sin, pos, axes, Dr, heads=None)`` rotates by positions
with several axes; with ``heads`` one shared head becomes that many, and its
gradient is the inverse rotation of the heads' sum.

``gated_ffn(x, w_gate_up, w_down, act)`` is the gated feed-forward block; it
keeps x, the gate and up products and the hidden activations for its backward.

``rms_norm(x, weight, eps, residual)`` is the norm of x, or of x + residual,
which it then gives too; it keeps that sum and a number per row.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch
from torch.autograd.function import once_differentiable

from . import bwd_dgrad, bwd_wgrad, fwd
from . import gated_ffn_bwd, gated_ffn_fwd
from . import rms_norm_bwd, rms_norm_fwd
from . import rope_axes as _rope_axes
from .rotary import _axes

__all__ = ["QUpProj", "q_up_proj", "Mxfp8Query", "q_up_proj_mxfp8", "RopeAxes", "rope_axes", "GatedFfn",
           "gated_ffn", "RmsNorm", "rms_norm"]


def _dense(g):
    """An upstream gradient as the kernels take it: contiguous, on 16 bytes. (A part of a concatenation's gradient is a
    slice that may start anywhere.)"""
    g = g.contiguous()
    return g.clone() if g.data_ptr() % 16 else g


def _layer_backward(ctx, dq):
    """dx, dW, db of the layer for the upstream gradient dq [T, H, D] bf16,
    only those autograd asks for."""
    x, W, cos, sin, pos = ctx.saved_tensors
    H, Dn, Dr = ctx.shape
    need_x, need_w, need_b = ctx.needs_input_grad[0], ctx.needs_input_grad[1], ctx.needs_input_grad[2]
    dq = _dense(dq)
    dx = dW = db = None
    rope = None
    if need_x:
        # dgrad also stores the rotated rope channels when wgrad follows
        if need_w or need_b:
            rope = torch.empty((x.shape[0], H, Dr), dtype=torch.bfloat16, device=dq.device)
        dx = bwd_dgrad(dq, W, cos, sin, H, Dn, Dr, pos=pos, dq_pre_rope=rope)
    if need_w or need_b:
        dW, db = bwd_wgrad(dq, x, cos, sin, H, Dn, Dr, pos=pos, db=ctx.has_bias and need_b, dq_pre_rope=rope)
    return dx if need_x else None, dW if need_w else None, db if need_b else None


class QUpProj(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, W, bias, cos, sin, pos, H, Dn, Dr):
        q = fwd(x, W, cos, sin, H, Dn, Dr, bias=bias, pos=pos, out_mode="bf16")
        ctx.save_for_backward(x, W, cos, sin, pos)
        ctx.shape = (H, Dn, Dr)
        ctx.has_bias = bias is not None
        return q

    @staticmethod
    @once_differentiable
    def backward(ctx, dq):
        dx, dW, db = _layer_backward(ctx, dq)
        return dx, dW, db, None, None, None, None, None, None


def q_up_proj(x, W, cos, sin, H, Dn, Dr, bias=None, pos=None):
    """q = RoPE(x W^T + b) as bf16 [T, H, Dn + Dr], differentiable in x, W and b."""
    return QUpProj.apply(x, W, bias, cos, sin, pos, H, Dn, Dr)


class _GradBox:
    """Holds the query gradient the consumer hands in until the backward runs."""

    def __init__(self):
        self.dq = None


class _QUpProjMxfp8(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, W, bias, cos, sin, pos, H, Dn, Dr, out_mode, box):
        codes, scales = fwd(x, W, cos, sin, H, Dn, Dr, bias=bias, pos=pos, out_mode=out_mode)
        ctx.save_for_backward(x, W, cos, sin, pos)
        ctx.shape = (H, Dn, Dr)
        ctx.has_bias = bias is not None
        ctx.box = box
        ctx.mark_non_differentiable(codes, scales)
        anchor = torch.zeros((), dtype=torch.float32, device=x.device)
        return codes, scales, anchor

    @staticmethod
    @once_differentiable
    def backward(ctx, g_codes, g_scales, g_anchor):
        dq = ctx.box.dq
        if dq is None:
            raise RuntimeError("the MXFP8 query's backward needs its bf16 gradient: call query.backward(dq)")
        ctx.box.dq = None
        dx, dW, db = _layer_backward(ctx, dq)
        return dx, dW, db, None, None, None, None, None, None, None, None


@dataclass
class Mxfp8Query:
    """The MXFP8 query of q_up_proj_mxfp8: codes uint8 [T, H, D] (E4M3),
    scales uint8 (E8M0; [T, H, ceil(D/32)] for out_mode "mxfp8", [H, T,
    ceil(D/32)] for "mxfp8_bhsd", each head in the GEMM's tiled order for
    "mxfp8_bhsd_swizzled"), and the anchor of the layer's autograd graph."""

    codes: torch.Tensor
    scales: torch.Tensor
    anchor: torch.Tensor
    _box: _GradBox

    def backward(self, dq: torch.Tensor) -> None:
        """Run the layer's backward for the query gradient dq (bf16 [T, H, D],
        e.g. the BF16 dQ of attention): dx, dW and db accumulate into the
        inputs' .grad like any autograd backward."""
        if dq.dtype != torch.bfloat16 or tuple(dq.shape) != tuple(self.codes.shape):
            raise ValueError(f"dq must be bf16 {list(self.codes.shape)}, got {dq.dtype} {list(dq.shape)}")
        self._box.dq = dq
        self.anchor.backward()


def q_up_proj_mxfp8(x, W, cos, sin, H, Dn, Dr, bias=None, pos=None, out_mode="mxfp8") -> Mxfp8Query:
    """The layer with an MXFP8 query (out_mode "mxfp8", "mxfp8_bhsd" or
    "mxfp8_bhsd_swizzled"), differentiable in x, W and b through
    Mxfp8Query.backward(dq)."""
    if out_mode not in ("mxfp8", "mxfp8_bhsd", "mxfp8_bhsd_swizzled"):
        raise ValueError(f"out_mode must be an MXFP8 mode, got {out_mode!r}")
    box = _GradBox()
    codes, scales, anchor = _QUpProjMxfp8.apply(x, W, bias, cos, sin, pos, H, Dn, Dr, out_mode, box)
    return Mxfp8Query(codes, scales, anchor, box)


class RopeAxes(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, cos, sin, pos, axes, Dr, heads):
        ctx.save_for_backward(cos, sin, pos)
        ctx.axes, ctx.Dr, ctx.shared = axes, Dr, heads is not None
        return _rope_axes(x if heads is None else x.expand(-1, heads, -1), cos, sin, pos, axes, Dr)

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        cos, sin, pos = ctx.saved_tensors
        if g.shape[2] > 1 and g.stride(2) != 1:
            g = g.contiguous()
        dx = _rope_axes(g, cos, sin, pos, ctx.axes, ctx.Dr, inverse=True, sum_heads=ctx.shared)
        return dx, None, None, None, None, None, None


def rope_axes(x, cos, sin, pos, axes, Dr, heads=None):
    """x [T, H, D] with the last Dr channels of every head rotated by several
    axes, differentiable in x. heads: x holds one head [T, 1, D] that this
    many heads share; the result is [T, heads, D]."""
    if heads is not None and x.shape[1] != 1:
        raise ValueError(f"a shared head is [T, 1, D], got {list(x.shape)}")
    # as bytes: a list that changes until the backward would turn the gradient otherwise
    return RopeAxes.apply(x, cos, sin, pos, _axes(axes, Dr), Dr, heads)


class GatedFfn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate_up, w_down, act):
        ctx.act = act
        if not any(ctx.needs_input_grad):
            return gated_ffn_fwd(x, w_gate_up, w_down, act=act)
        y, gate_up, h = gated_ffn_fwd(x, w_gate_up, w_down, act=act, save=True)
        ctx.save_for_backward(x, w_gate_up, w_down, gate_up, h)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w_gate_up, w_down, gate_up, h = ctx.saved_tensors
        need = ctx.needs_input_grad
        return (*gated_ffn_bwd(_dense(dy), x, w_gate_up, w_down, gate_up, h, act=ctx.act, dx=need[0],
                               dw_gate_up=need[1], dw_down=need[2]), None)


def gated_ffn(x, w_gate_up, w_down, act="silu"):
    """(act(g) * u) w_down^T with [g | u] = x w_gate_up^T as bf16 [T, K],
    differentiable in x, w_gate_up and w_down."""
    if not torch.is_grad_enabled():  # nothing to keep for a backward; a Function sees the inputs' flags only
        return gated_ffn_fwd(x, w_gate_up, w_down, act=act)
    return GatedFfn.apply(x, w_gate_up, w_down, act)


def _plain_rows(g):
    """An upstream gradient with unit inner stride and rows that do not overlap (an expanded one is copied)."""
    return g if g.stride(1) == 1 and (g.shape[0] <= 1 or g.stride(0) >= g.shape[1]) else g.contiguous()


class RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        ctx.set_materialize_grads(False)
        if not any(ctx.needs_input_grad):
            return rms_norm_fwd(x, weight, eps=eps, residual=residual)
        r = rms_norm_fwd(x, weight, eps=eps, residual=residual, save=True)
        ctx.save_for_backward(x if residual is None else r[1], weight, r[-1])
        return r[0] if residual is None else (r[0], r[1])

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh=None):
        h, weight, rstd = ctx.saved_tensors
        need_x, need_w, need_r = ctx.needs_input_grad[:3]
        if dy is None:  # h alone was used
            return dh if need_x else None, torch.zeros_like(weight) if need_w else None, dh if need_r else None, None
        need = need_x or need_r
        dx, dw = rms_norm_bwd(_plain_rows(dy), h, weight, rstd, dres=None if dh is None or not need else _plain_rows(dh),
                              dx=need, dw=need_w)
        return dx if need_x else None, dw, dx if need_r else None, None


def rms_norm(x, weight, eps=1e-6, residual=None):
    """The RMS norm of x [T, K], differentiable in x and weight; with a
    residual (y, h): the norm of h = x + residual, and h for the next block,
    differentiable in the residual too."""
    if not torch.is_grad_enabled():
        return rms_norm_fwd(x, weight, eps=eps, residual=residual)
    return RmsNorm.apply(x, weight, residual, eps)
