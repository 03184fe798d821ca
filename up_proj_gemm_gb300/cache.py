"""Keys and values in a paged 8-bit cache, and the attention that reads them:
argument marshalling for ``mla_kv_cache_write``, ``mla_kv_cache_read`` and
``mla_cache_attn`` (declared in ``include/mlaq.h``).

``KvCache`` holds the pages. ``kv_cache_write`` quantizes what ``kv_fwd`` gives
(or the latents and rotary keys it starts from) as it is appended,
``kv_cache_read`` gives it back, and ``cache_attn`` takes a query over it: single
tokens, drafts of a few, or a prompt's chunk. Over keys and values of the heads
that is the query that ``fwd`` gives. Over latents the caller multiplies the key
weights into the query and the value weights into the result.
"""
from __future__ import annotations

import ctypes
import math

import torch

import up_proj_gemm_gb300 as _pkg

from . import _call, _empty, _need, _ptr, _SIGS, _status, _stream, lib

__all__ = ["KvCache", "KvCacheShape", "AttnShape", "kv_cache_write", "kv_cache_read", "cache_attn"]

_u8, _bf16, _f32, _i32 = torch.uint8, torch.bfloat16, torch.float32, torch.int32


class KvCacheShape(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_int64)] + [(n, ctypes.c_int32) for n in ("page", "block", "H", "Dk", "Dv", "reserved")] + [
        (n, ctypes.c_void_p) for n in ("k", "k_scales", "v", "v_scales")]


class AttnShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("T", "B", "q_t", "q_h", "table_width")] + [
        ("Hq", ctypes.c_int32), ("scale", ctypes.c_float), ("reserved", ctypes.c_int64)]


_vp, _int, _i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
_cache = ctypes.POINTER(KvCacheShape)
_SIGS.update({
    "mla_kv_cache_write": (_int, [_cache, _vp, _i64, _i64, _vp, _i64, _i64, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _vp]),
    "mla_kv_cache_read": (_int, [_cache, _vp, _vp, _int, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _vp]),
    "mla_cache_attn_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(AttnShape), _cache]),
    "mla_cache_attn": (_int, [ctypes.POINTER(AttnShape), _cache] + [_vp] * 7 + [ctypes.c_size_t, _vp, _vp]),
})


class KvCache:
    """Pages of E4M3 codes with an E8M0 scale for each block of tokens and head.

    k uint8 [pages, H, page, Dk] with k_scales uint8 [pages, H, page / block];
    v [pages, H, page, Dv] and v_scales alike, or None: the values are then the
    first Dv channels of the keys (a latent cache; Dv defaults to all). page
    is a power of two from 16 to 1024, block one from 1 to page, Dk and Dv
    multiples of 16, and there is a page at least. ``KvCache.empty`` allocates
    one. Pages need no particular contents until they are written."""

    def __init__(self, k, k_scales, v=None, v_scales=None, Dv=None):
        self.k, self.k_scales, self.v, self.v_scales = k, k_scales, v, v_scales
        own = isinstance(v, torch.Tensor) and v.dim() == 4
        if Dv is None:
            Dv = v.shape[3] if own else k.shape[3] if isinstance(k, torch.Tensor) and k.dim() == 4 else 0
        self.Dv = int(Dv)
        self.check()

    @classmethod
    def empty(cls, pages, page, heads, Dk, Dv, block=32, shared=False, device="cuda"):
        """A cache of `pages` pages of `page` tokens; shared: the values are the first Dv channels of the keys."""
        def codes(D):
            return torch.empty((pages, heads, page, D), dtype=_u8, device=device)

        def scales():
            return torch.empty((pages, heads, page // block), dtype=_u8, device=device)

        return cls(codes(Dk), scales(), None if shared else codes(Dv), None if shared else scales(), Dv)

    def check(self):
        """Raise where the tensors are not a cache."""
        _need(self.k, "cache.k", _u8, ndim=4)
        pages, H, page, Dk = self.k.shape
        dev = self.k.device
        _need(self.k_scales, "cache.k_scales", _u8, dev, ndim=3)
        per = self.k_scales.shape[2]
        if pages < 1:
            raise ValueError("a cache has a page at least")
        if page < 16 or page > 1024 or page & (page - 1):
            raise ValueError(f"a page must hold a power of two of 16 to 1024 tokens, got {page}")
        if per < 1 or page % per or (per & (per - 1)):
            raise ValueError(f"a page's {page} tokens must be a power of two of blocks, got {per}")
        _need(self.k_scales, "cache.k_scales", _u8, dev, shape=(pages, H, per))
        if (self.v is None) != (self.v_scales is None):
            raise ValueError("values and their scales go together")
        if self.v is None:
            if not 0 < self.Dv <= Dk:
                raise ValueError(f"values in the keys have 1 to {Dk} channels, got {self.Dv}")
        else:
            _need(self.v, "cache.v", _u8, dev, shape=(pages, H, page, self.Dv))
            _need(self.v_scales, "cache.v_scales", _u8, dev, shape=(pages, H, per))

    def _shape(self):
        self.check()
        pages, H, page, Dk = self.k.shape
        at = [None if t is None or not t.numel() else t.data_ptr() for t in (self.k, self.k_scales, self.v, self.v_scales)]
        return KvCacheShape(pages, page, page // self.k_scales.shape[2], H, Dk, self.Dv, 0, *at)


def _sequences(table, at, name, cu, T, dev):
    """Check the table [B, width], the positions [B] and the rows' bounds [B + 1]; B."""
    _need(table, "table", _i32, dev, ndim=2)
    B = table.shape[0]
    _need(at, name, _i32, dev, shape=(B,))
    if cu is not None:
        _need(cu, "cu", _i32, dev, shape=(B + 1,))
    elif T != B:
        raise ValueError(f"without cu every sequence has one row: {T} rows for {B} sequences")
    return B


def _dense(t, name, dev, H, D, T=None):
    """Rows [T, H, D] in bf16 with any strides outside the channels; their strides as the library takes them."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != _bf16:
        raise TypeError(f"{name} must be {_bf16}, got {t.dtype}")
    if t.dim() != 3 or tuple(t.shape[1:]) != (H, D) or (T is not None and t.shape[0] != T):
        raise ValueError(f"{name} must be {['T' if T is None else T, H, D]}, got {list(t.shape)}")
    if not t.is_cuda or t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if D > 1 and t.stride(2) != 1:
        raise ValueError(f"{name} must have unit inner stride")
    return t.stride(0) if t.shape[0] > 1 else 0, t.stride(1) if H > 1 else 0


def kv_cache_write(cache, k, v, table, start, cu=None, status=None, stream=None):
    """Append tokens: row cu[b] + i of k [T, H, Dk] and v [T, H, Dv] (bf16, any
    token and head strides; v None for a cache without values of its own) goes
    to position start[b] + i of sequence b, quantized.

    table int32 [B, width]: the pages of every sequence's positions; start
    int32 [B]; cu int32 [B + 1], or None where every sequence brings one
    token. A block's scale is the smallest power of two that holds its finite
    elements; a block that is continued keeps its scale or raises it, and its
    older codes are then rounded again. Positions behind the new ones are no
    longer valid. Pages that are written belong to one sequence of the call."""
    if not isinstance(cache, KvCache):
        raise TypeError("cache must be a KvCache")
    lib()
    c = _pkg._calls
    if c is not None and status is None and stream is None and c.kv_cache_write(
            cache.k, cache.k_scales, cache.v, cache.v_scales, cache.Dv, k, v, table, start, cu):
        return
    s = cache._shape()
    dev = cache.k.device
    k_t, k_h = _dense(k, "k", dev, s.H, s.Dk)
    T = k.shape[0]
    v_t = v_h = 0
    if cache.v is not None:
        v_t, v_h = _dense(v, "v", dev, s.H, s.Dv, T)
    elif v is not None:
        raise ValueError("the cache's values are in its keys: v must be None")
    B = _sequences(table, start, "start", cu, T, dev)
    _status(status, dev)
    _call(lib().mla_kv_cache_write, "mla_kv_cache_write", ctypes.byref(s), _ptr(k), k_t, k_h, _ptr(v), v_t, v_h, T, B,
          _ptr(table), table.shape[1], _ptr(start), _ptr(cu), _ptr(status), _stream(dev, stream))


def kv_cache_read(cache, table, start, tokens, cu=None, dtype=torch.bfloat16, k=None, v=None, status=None, stream=None):
    """(k [tokens, H, Dk], v [tokens, H, Dv] or None): row cu[b] + i is position
    start[b] + i of sequence b, as bf16 or float32. Rows behind the last
    sequence's are left as they are. See ``kv_cache_write`` for the arguments."""
    if not isinstance(cache, KvCache):
        raise TypeError("cache must be a KvCache")
    if dtype not in (_bf16, _f32):
        raise TypeError(f"dtype must be bfloat16 or float32, got {dtype}")
    tokens = int(tokens)
    if tokens < 0:
        raise ValueError(f"tokens must not be negative, got {tokens}")
    lib()
    c = _pkg._calls
    if c is not None and k is None and v is None and status is None and stream is None:
        r = c.kv_cache_read(cache.k, cache.k_scales, cache.v, cache.v_scales, cache.Dv, table, start, tokens, cu,
                            1 if dtype is _bf16 else 0)
        if r is not None:
            return r
    s = cache._shape()
    dev = cache.k.device
    B = _sequences(table, start, "start", cu, tokens, dev)
    _status(status, dev)
    if cache.v is None and v is not None:
        raise ValueError("the cache's values are in its keys: v must be None")
    outs = []
    for name, t, D in (("k", k, s.Dk), ("v", v, s.Dv)):
        if name == "v" and cache.v is None:
            t = None
        elif t is None:
            t = _empty((tokens, s.H, D), dtype, dev, stream)
        else:
            _need(t, name, dtype, dev, shape=(tokens, s.H, D))
        outs.append(t)
    _call(lib().mla_kv_cache_read, "mla_kv_cache_read", ctypes.byref(s), _ptr(outs[0]), _ptr(outs[1]),
          0 if dtype is _f32 else 1, tokens, B, _ptr(table), table.shape[1], _ptr(start), _ptr(cu), _ptr(status),
          _stream(dev, stream))
    return tuple(outs)


def cache_attn(q, cache, table, length, cu=None, scale=None, lse=False, out=None, workspace=None, status=None, stream=None):
    """out [T, Hq, Dv] bf16 = softmax(scale q k^T) v over the cache, for q [T, Hq, Dk] bf16 (any token and head strides).

    Sequence b has length[b] positions (int32 [B], its new tokens counted);
    rows cu[b] to cu[b + 1] - 1 of q are its last ones, and each sees the
    positions up to its own (cu None: one row for each sequence). Query head h
    reads head h / (Hq / H) of the cache. scale defaults to Dk^-1/2. lse=True
    (or a float32 tensor [T, Hq]) also gives the scores' log-sum-exp, as
    (out, lse). A row that sees nothing gives zeros and -inf; rows behind the
    last sequence's are left as they are. The workspace (uint8) is allocated
    unless passed."""
    if not isinstance(cache, KvCache):
        raise TypeError("cache must be a KvCache")
    lib()
    if scale is not None and not math.isfinite(scale):
        raise ValueError(f"scale must be finite, got {scale}")
    c = _pkg._calls
    if c is not None and out is None and workspace is None and status is None and stream is None and (
            lse is True or lse is False):
        r = c.cache_attn(q, cache.k, cache.k_scales, cache.v, cache.v_scales, cache.Dv, table, length, cu,
                         math.nan if scale is None else scale, lse)
        if r is not None:
            return r
    s = cache._shape()
    dev = cache.k.device
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a bf16 CUDA tensor [T, Hq, Dk]")
    T, Hq, _ = q.shape
    if Hq < 1 or Hq % s.H:
        raise ValueError(f"the {Hq} query heads must be a multiple of the cache's {s.H}")
    q_t, q_h = _dense(q, "q", dev, Hq, s.Dk)
    B = _sequences(table, length, "length", cu, T, dev)
    _status(status, dev)
    scale = s.Dk ** -0.5 if scale is None else float(scale)
    if out is None:
        out = _empty((T, Hq, s.Dv), _bf16, dev, stream)
    else:
        _need(out, "out", _bf16, dev, shape=(T, Hq, s.Dv))
    if lse is True:
        lse = _empty((T, Hq), _f32, dev, stream)
    elif lse is False:
        lse = None
    elif lse is not None:
        _need(lse, "lse", _f32, dev, shape=(T, Hq))
    a = AttnShape(T, B, q_t, q_h, table.shape[1], Hq, scale, 0)
    if workspace is None:
        workspace = _empty((int(lib().mla_cache_attn_workspace_size(ctypes.byref(a), ctypes.byref(s))),), _u8, dev, stream,
                           scratch=True)
    else:
        _need(workspace, "workspace", _u8, dev, ndim=1)
    _call(lib().mla_cache_attn, "mla_cache_attn", ctypes.byref(a), ctypes.byref(s), _ptr(q), _ptr(table), _ptr(length),
          _ptr(cu), _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(), _ptr(status), _stream(dev, stream))
    return out if lse is None else (out, lse)
