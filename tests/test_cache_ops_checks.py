"""Refusals of the norm, the 8-bit cache and the attention over it without a GPU: the C entry points with fake device
addresses, the binding with CPU tensors that report themselves as CUDA tensors, and the memory of calls on another
stream than the current one."""
import contextlib
import ctypes
import math

import pytest
import torch

import up_proj_gemm_gb300 as mlaq
from up_proj_gemm_gb300 import _build, cache, norm

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="a valid call would use the fake addresses")
S = mlaq.STATUS
OK, INV, AL, ALIAS, UNSUP, NO_GPU = (S[n] for n in ("MLA_OK", "MLA_ERR_INVALID_ARG", "MLA_ERR_ALIGNMENT", "MLA_ERR_ALIAS",
                                                    "MLA_ERR_UNSUPPORTED", "MLA_ERR_CUDA"))
bf16, f32, u8, i32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
FAKE = 0x40000000


@pytest.fixture(scope="module")
def L():
    _build.build()
    return mlaq.lib()


def p(i, off=0):
    return ctypes.c_void_p(FAKE * (i + 1) + off)


# ------------------------------------------------------------ C entry points
def norm_fwd(L, T=64, K=64, ld_x=0, ld_res=0, dtype=1, w_dtype=1, mode=0, eps=1e-6, reserved=0, **kw):
    s = norm.NormShape(T, K, ld_x, ld_res, 0, dtype, w_dtype, mode, eps, reserved)
    a = dict(x=p(0), res=p(1), w=p(2), h=p(3), y=p(4), sc=None, rstd=p(6))
    a.update(kw)
    return L.mla_rms_norm_fwd(ctypes.byref(s), *[a[n] for n in ("x", "res", "w", "h", "y", "sc", "rstd")], None)


def test_norm_forward_refusals(L):
    mx = dict(mode=1, sc=p(5))
    assert norm_fwd(L) == NO_GPU and norm_fwd(L, **mx) == NO_GPU and norm_fwd(L, mode=2, sc=p(5)) == NO_GPU
    for kw in (dict(T=-1), dict(K=0), dict(K=-8), dict(dtype=2), dict(dtype=-1), dict(w_dtype=2), dict(mode=3), dict(mode=-1),
               dict(eps=-1e-6), dict(eps=math.nan), dict(eps=math.inf), dict(reserved=1), dict(ld_x=56), dict(ld_res=-64),
               dict(T=2 ** 31), dict(x=None), dict(w=None), dict(y=None), dict(h=None), dict(res=None), dict(sc=p(5)), dict(mode=1),
               dict(T=2 ** 30, ld_x=2 ** 40)):
        assert norm_fwd(L, **kw) == INV, kw
    assert norm_fwd(L, K=2 ** 15 + 8) == UNSUP and norm_fwd(L, K=2 ** 15) == NO_GPU
    assert norm_fwd(L, K=48, **mx) == UNSUP
    for kw in (dict(x=p(0, 1)), dict(w=p(2, 1)), dict(w_dtype=0, w=p(2, 2)), dict(h=p(3, 1)), dict(rstd=p(6, 2)), dict(y=p(4, 4), **mx)):
        assert norm_fwd(L, **kw) == AL, kw
    for kw in (dict(y=p(0)), dict(h=p(1)), dict(h=p(4)), dict(rstd=p(4, 64 * 64 * 2 - 4)), dict(y=p(2)), dict(mode=1, sc=p(4, 64 * 64 - 2))):
        assert norm_fwd(L, **kw) == ALIAS, kw
    # a pitched x spans (T - 1) ld + K elements
    assert norm_fwd(L, ld_x=128, y=p(0, (63 * 128 + 64) * 2)) == NO_GPU
    assert norm_fwd(L, ld_x=128, y=p(0, (63 * 128 + 64) * 2 - 2)) == ALIAS
    assert norm_fwd(L, T=0, x=None, res=None, h=None, y=None, rstd=None) == OK
    assert norm_fwd(L, T=0, w=None) == INV
    assert L.mla_rms_norm_fwd(None, *[None] * 8) == INV


def norm_bwd(L, T=64, K=64, dtype=1, w_dtype=0, mode=0, size=1 << 24, **kw):
    s = norm.NormShape(T, K, 0, 0, 0, dtype, w_dtype, mode, 0.0, 0)
    a = dict(dy=p(0), h=p(1), w=p(2), rstd=p(3), dh=p(4), dx=p(5), dw=p(6), ws=p(7))
    a.update(kw)
    return L.mla_rms_norm_bwd(ctypes.byref(s), *[a[n] for n in ("dy", "h", "w", "rstd", "dh", "dx", "dw", "ws")], size, None)


def test_norm_backward_refusals(L):
    assert norm_bwd(L) == NO_GPU and norm_bwd(L, dw=None, size=0) == NO_GPU and norm_bwd(L, dx=None, dh=None) == NO_GPU
    for kw in (dict(dx=None, dw=None), dict(dx=None), dict(dy=None), dict(h=None), dict(w=None), dict(rstd=None), dict(mode=1)):
        assert norm_bwd(L, **kw) == INV, kw
    for kw in (dict(dx=p(0)), dict(dx=p(4)), dict(dw=p(5)), dict(dw=p(2)), dict(dx=p(7)), dict(dw=p(3))):
        assert norm_bwd(L, **kw) == ALIAS, kw
    for kw in (dict(dy=p(0, 1)), dict(dw=p(6, 2)), dict(ws=p(7, 8))):
        assert norm_bwd(L, **kw) == AL, kw
    assert norm_bwd(L, T=0, dw=None) == OK
    s = norm.NormShape(4, 0, 0, 0, 0, 1, 1, 0, 0.0, 0)
    assert L.mla_rms_norm_bwd_workspace_size(ctypes.byref(s)) == 0 and L.mla_rms_norm_bwd_workspace_size(None) == 0


def cache_shape(pages=8, page=64, block=32, H=2, Dk=64, Dv=32, reserved=0, k=p(0), ks=p(1), v=p(2), vs=p(3)):
    return cache.KvCacheShape(pages, page, block, H, Dk, Dv, reserved, k, ks, v, vs)


BAD_CACHES = [(dict(pages=-1), INV), (dict(page=8), INV), (dict(page=96), INV), (dict(page=2048), INV), (dict(block=0), INV),
              (dict(block=3), INV), (dict(block=128), INV), (dict(H=0), INV), (dict(Dk=0), INV), (dict(Dv=-16), INV),
              (dict(reserved=1), INV), (dict(k=None), INV), (dict(ks=None), INV), (dict(v=None), INV), (dict(vs=None), INV),
              (dict(v=None, vs=None, Dv=80), INV), (dict(pages=2 ** 31), INV), (dict(Dk=72), UNSUP), (dict(Dv=24), UNSUP),
              (dict(k=p(0, 8)), AL), (dict(v=p(2, 4)), AL)]


def write(L, c=None, T=100, B=3, width=4, k_t=128, k_h=64, v_t=64, v_h=32, **kw):
    a = dict(k=p(4), v=p(5), table=p(6), start=p(7), cu=p(8), st=None)
    a.update(kw)
    return L.mla_kv_cache_write(ctypes.byref(cache_shape(**(c or {}))), a["k"], k_t, k_h, a["v"], v_t, v_h, T, B, a["table"],
                                width, a["start"], a["cu"], a["st"], None)


def read(L, c=None, T=100, B=3, width=4, dtype=1, **kw):
    a = dict(k=p(4), v=p(5), table=p(6), start=p(7), cu=p(8), st=None)
    a.update(kw)
    return L.mla_kv_cache_read(ctypes.byref(cache_shape(**(c or {}))), a["k"], a["v"], dtype, T, B, a["table"], width,
                               a["start"], a["cu"], a["st"], None)


def test_cache_refusals(L):
    shared = dict(v=None, vs=None)
    for f in (write, read):
        assert f(L) == NO_GPU and f(L, shared, v=None) == NO_GPU and f(L, T=3, cu=None) == NO_GPU
        for c, want in BAD_CACHES:
            assert f(L, c, **(dict(v=None) if c.get("v", 1) is None else {})) == want, c
        for kw in (dict(T=-1), dict(B=-1), dict(T=2 ** 31), dict(B=0), dict(cu=None), dict(k=None), dict(v=None), dict(start=None),
                   dict(table=None), dict(width=-1), dict(width=2 ** 31)):
            assert f(L, **kw) == INV, kw
        assert f(L, shared) == INV  # v without values in the cache
        for kw in (dict(k=p(4, 1)), dict(v=p(5, 1)), dict(start=p(7, 2)), dict(cu=p(8, 1)), dict(table=p(6, 2)), dict(st=p(9, 2))):
            assert f(L, **kw) == AL, kw
        assert f(L, T=2 ** 31 - 1) in (UNSUP, NO_GPU, INV, ALIAS) and f(L, dict(H=65535, pages=1), T=2 ** 30, B=1) != OK
        assert f(L, T=0, k=None, v=None) == OK and f(L, T=0, B=0, cu=None, start=None, table=None) == OK
    for kw in (dict(k=p(0)), dict(k=p(1)), dict(v=p(2, 8 * 2 * 64 * 32 - 2)), dict(table=p(0)), dict(start=p(3)), dict(st=p(2)), dict(cu=p(0))):
        assert write(L, **kw) == ALIAS, kw
    for kw in (dict(k_t=-1), dict(v_h=-32), dict(k_t=2 ** 62)):
        assert write(L, **kw) == INV, kw
    assert write(L, k_t=0, k_h=0) == NO_GPU  # one row for all
    assert write(L, k=p(4, 2), v=p(5, 2)) == NO_GPU
    # the dense side spans (T - 1) k_t + (H - 1) k_h + Dk elements
    end = (99 * 128 + 64 + 64) * 2
    assert write(L, v=p(4, end)) == NO_GPU and write(L, dict(k=p(4, end + 0))) == NO_GPU and write(L, dict(k=p(4, end - 16))) == ALIAS
    assert read(L, dtype=2) == INV and read(L, dtype=-1) == INV
    assert read(L, k=p(4, 8)) == AL
    for kw in (dict(k=p(0)), dict(v=p(4)), dict(k=p(1)), dict(v=p(6)), dict(st=p(4)), dict(st=p(7))):
        assert read(L, **kw) == ALIAS, kw
    assert L.mla_kv_cache_write(None, *[None, 0, 0, None, 0, 0, 0, 0, None, 0, None, None, None, None]) == INV
    assert L.mla_kv_cache_read(None, None, None, 1, 0, 0, None, 0, None, None, None, None) == INV


def attn(L, c=None, T=10, B=3, q_t=512, q_h=64, width=4, Hq=8, scale=0.1, reserved=0, size=1 << 28, **kw):
    s = cache.AttnShape(T, B, q_t, q_h, width, Hq, scale, reserved)
    a = dict(q=p(4), table=p(5), length=p(6), cu=p(7), out=p(8), lse=p(9), ws=p(10), st=None)
    a.update(kw)
    return L.mla_cache_attn(ctypes.byref(s), ctypes.byref(cache_shape(**(c or {}))),
                            *[a[n] for n in ("q", "table", "length", "cu", "out", "lse", "ws")], size, a["st"], None)


def test_attention_refusals(L):
    shared = dict(v=None, vs=None)
    assert attn(L) == NO_GPU and attn(L, shared) == NO_GPU and attn(L, lse=None) == NO_GPU and attn(L, T=3, cu=None) == NO_GPU
    for c, want in BAD_CACHES:
        assert attn(L, c) == want, c
    for kw in (dict(T=-1), dict(T=2 ** 31), dict(B=-1), dict(B=0), dict(Hq=0), dict(Hq=7), dict(Hq=-2), dict(scale=math.nan),
               dict(scale=math.inf), dict(scale=-math.inf), dict(reserved=1), dict(q_t=-1), dict(q_h=-64), dict(q_t=2 ** 62),
               dict(cu=None), dict(q=None), dict(out=None), dict(length=None), dict(table=None), dict(width=-1), dict(width=0),
               dict(width=2 ** 31)):
        assert attn(L, **kw) == INV, kw
    assert attn(L, dict(pages=0)) == INV
    for c in (dict(Dk=272), dict(Dv=272), dict(Dk=656, Dv=512, **shared), dict(Dk=640, Dv=528, **shared)):
        assert attn(L, c, q_t=8 * 656, q_h=656) == UNSUP, c
    assert attn(L, dict(Dk=640, Dv=512, **shared), q_t=8 * 640, q_h=640) == NO_GPU
    assert attn(L, T=2 ** 29, q_t=0, q_h=0) == UNSUP  # more than 2^31 - 1 rows of heads
    for kw in (dict(q=p(4, 1)), dict(out=p(8, 1)), dict(lse=p(9, 2)), dict(length=p(6, 1)), dict(cu=p(7, 2)), dict(ws=p(10, 8)),
               dict(st=p(11, 1)), dict(table=p(5, 2))):
        assert attn(L, **kw) == AL, kw
    for kw in (dict(out=p(4)), dict(out=p(0)), dict(lse=p(8, 16)), dict(ws=p(8)), dict(ws=p(5)), dict(out=p(2)), dict(lse=p(7)),
               dict(st=p(6)), dict(out=p(10))):
        assert attn(L, **kw) == ALIAS, kw
    assert attn(L, T=0, q=None, out=None, length=None, size=0) == OK
    s = cache.AttnShape(10, 3, 512, 64, 4, 8, 0.1, 0)
    assert L.mla_cache_attn_workspace_size(None, ctypes.byref(cache_shape())) == 0
    assert L.mla_cache_attn_workspace_size(ctypes.byref(s), None) == 0
    assert L.mla_cache_attn(None, ctypes.byref(cache_shape()), *[None] * 7, 0, None, None) == INV
    assert L.mla_cache_attn(ctypes.byref(s), None, *[None] * 7, 0, None, None) == INV


# ------------------------------------------------------------------ binding
class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Log:
    def __init__(self):
        self.current = Stream(0)
        self.names = []     # entry points that were called
        self.made = {}      # address: the stream that was current when it was allocated
        self.recorded = {}  # address: the stream that it was recorded on


@pytest.fixture
def log(L, monkeypatch):
    log, empty = Log(), torch.empty

    def make(*a, **kw):
        t = empty(*a, **kw)
        log.made[t.data_ptr()] = log.current.cuda_stream
        return t

    @contextlib.contextmanager
    def on(stream):
        before, log.current = log.current, stream
        yield
        log.current = before

    monkeypatch.setattr(mlaq, "_calls", None)
    for m in (cache, norm):
        monkeypatch.setattr(m, "_call", lambda fn, what, *args: log.names.append(what))
        monkeypatch.setattr(m, "_stream", lambda device, stream: None)
    # the sizes of workspaces ask the device
    for name in ("mla_cache_attn_workspace_size", "mla_rms_norm_bwd_workspace_size"):
        monkeypatch.setattr(mlaq.lib(), name, lambda *a: 4096)
    monkeypatch.setattr(torch, "empty", make)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: log.recorded.__setitem__(t.data_ptr(), s.cuda_stream))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: log.current)
    monkeypatch.setattr(torch.cuda, "stream", on)
    return log


def refused(f, *a, **kw):
    with pytest.raises((TypeError, ValueError)):
        f(*a, **kw)


def test_norm_binding(log):
    T, K = 6, 64
    x, w = torch.zeros(T, K, dtype=bf16), torch.ones(K, dtype=bf16)
    f, b = mlaq.rms_norm_fwd, mlaq.rms_norm_bwd
    assert f(x, w).shape == (T, K)
    y, h, rstd = f(torch.zeros(T, K + 8, dtype=bf16)[:, :K], w.float(), residual=x, save=True)
    codes, scales = f(x, w, out="mxfp8")
    assert codes.dtype == u8 and scales.shape == (T, K // 32) and f(x, w, out="tiled")[1].shape == (512,)
    n = len(log.names)
    for bad in ((None, w), (x, None), (x.double(), w), (x[0], w), (x.t(), w), (x, w[1:]), (x, w.double()), (x, w[None]),
                (x[:1].expand(T, K), w)):
        refused(f, *bad)
    for kw in (dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(out="e4m3"), dict(residual=x.float()), dict(residual=x[1:]),
               dict(y=y.float()), dict(y=y[1:]), dict(h=h), dict(scales=scales), dict(rstd=rstd.to(bf16)), dict(rstd=rstd[1:])):
        refused(f, x, w, **kw)
    refused(f, x, w, out="mxfp8", scales=scales[1:])
    refused(f, x, w, out="mxfp8", y=y)
    assert len(log.names) == n
    dx, dw = b(x, h, w, rstd)
    assert dx.shape == (T, K) and dw.shape == (K,) and dw.dtype == bf16
    assert b(x, h, w, rstd, dx=False)[0] is None and b(x, h, w, rstd, dw=None)[1] is None
    n = len(log.names)
    for bad in ((x.float(), h, w, rstd), (x[1:], h, w, rstd), (x, h, w[1:], rstd), (x, h, w, rstd[1:]), (x, h, w, rstd.double()),
                (x, h, w, None), (None, h, w, rstd), (x, None, w, rstd)):
        refused(b, *bad)
    for kw in (dict(dx=False, dw=False), dict(dres=x, dx=False), dict(dres=x.float()), dict(dx=x[1:]), dict(dw=w.float()),
               dict(workspace=torch.zeros(8))):
        refused(b, x, h, w, rstd, **kw)
    assert len(log.names) == n


def sequences(B=2, width=4):
    return torch.zeros(B, width, dtype=i32), torch.zeros(B, dtype=i32), torch.zeros(B + 1, dtype=i32)


def test_cache_binding(log):
    own = mlaq.KvCache.empty(8, 64, 2, 64, 32, device="cpu")
    latent = mlaq.KvCache.empty(8, 64, 1, 64, 48, shared=True, device="cpu")
    assert own.Dv == 32 and latent.v is None and latent.Dv == 48
    u = lambda *s: torch.zeros(s, dtype=u8)  # noqa: E731
    assert mlaq.KvCache(u(8, 2, 64, 48), u(8, 2, 2)).Dv == 48
    for bad in ((u(8, 2, 64), u(8, 2, 2)), (u(8, 2, 64, 48).float(), u(8, 2, 2)), (u(8, 2, 64, 48), u(8, 2, 3)),
                (u(8, 2, 64, 48), u(8, 1, 2)), (u(8, 2, 96, 48), u(8, 2, 2)), (u(8, 2, 8, 48), u(8, 2, 1)),
                (u(8, 2, 2048, 16), u(8, 2, 1)), (u(8, 2, 64, 48), u(8, 2, 2), u(8, 2, 64, 48)), (None, u(8, 2, 2)),
                (u(8, 2, 64, 48), None), (u(8, 2, 64, 48), u(8, 2, 2), u(8, 2, 32, 48), u(8, 2, 2)), (u(0, 2, 64, 48), u(0, 2, 2)),
                (u(8, 2, 64, 48), u(8, 2, 2), u(8, 2, 64, 48), u(8, 2, 1)), (u(8, 2, 64, 48), u(8, 2, 0))):
        refused(mlaq.KvCache, *bad)
    refused(mlaq.KvCache, u(8, 2, 64, 48), u(8, 2, 2), Dv=64)
    refused(mlaq.KvCache, u(8, 2, 64, 48), u(8, 2, 2), Dv=-1)
    table, start, cu = sequences()
    T = 5
    k, v = torch.zeros(T, 2, 64, dtype=bf16), torch.zeros(T, 2, 32, dtype=bf16)
    w, r = mlaq.kv_cache_write, mlaq.kv_cache_read
    w(own, k, v, table, start, cu=cu)
    w(own, k[:2], v[:2], table, start)
    w(own, k.transpose(0, 1).contiguous().transpose(0, 1), torch.zeros(T, 2, 96, dtype=bf16)[..., :32], table, start, cu=cu)
    w(latent, k[:, :1], None, table, start, cu=cu)
    assert [t.shape for t in r(own, table, start, T, cu=cu)] == [(T, 2, 64), (T, 2, 32)]
    a, b = r(latent, table, start, T, cu=cu, dtype=f32)
    assert a.dtype == f32 and b is None
    n = len(log.names)
    refused(w, None, k, v, table, start, cu)
    for bad in ((k, v, table, start), (k.float(), v, table, start, cu), (k, None, table, start, cu), (None, v, table, start, cu),
                (k, v[1:], table, start, cu), (k[:, :1], v, table, start, cu), (k, v, table[0], start, cu), (k, v, table.long(), start, cu),
                (k, v, table, start[1:], cu), (k, v, table, start.long(), cu), (k, v, table, start, cu[1:]), (k, v, table, start, cu.long()),
                (torch.zeros(T, 2, 128, dtype=bf16)[..., ::2], v, table, start, cu), (k, v, None, start, cu), (k, v, table, None, cu)):
        refused(w, own, *bad)
    refused(w, latent, k[:, :1], k[:, :1], table, start, cu)
    refused(w, own, k, v, table, start, cu, status=torch.zeros(1))
    for kw in (dict(dtype=torch.float16), dict(k=k[1:]), dict(v=v.float()), dict(status=torch.zeros(1))):
        refused(r, own, table, start, T, cu=cu, **kw)
    refused(r, own, table, start, -1, cu=cu)
    refused(r, own, table, start, T)
    refused(r, latent, table, start, T, cu=cu, v=v)
    assert len(log.names) == n


def test_attention_binding(log):
    own = mlaq.KvCache.empty(8, 64, 2, 64, 32, device="cpu")
    table, length, cu = sequences()
    T = 5
    q = torch.zeros(T, 6, 64, dtype=bf16)
    f = mlaq.cache_attn
    out = f(q, own, table, length, cu=cu)
    assert out.shape == (T, 6, 32) and f(q[:2], own, table, length).shape == (2, 6, 32)
    out, lse = f(q, own, table, length, cu=cu, lse=True)
    assert lse.shape == (T, 6) and lse.dtype == f32
    o, l = f(q, own, table, length, cu=cu, lse=lse)  # a result that is passed, alone and with the other
    assert l is lse
    o, l = f(q, own, table, length, cu=cu, lse=lse, out=out)
    assert o is out and l is lse
    assert f(q, own, table, length, cu=cu, lse=None).shape == (T, 6, 32)
    n = len(log.names)
    refused(f, q, None, table, length, cu=cu)
    for bad in ((None, own, table, length), (q[0], own, table, length), (q.float(), own, table, length), (q[:, :5], own, table, length),
                (q[..., :32], own, table, length), (q, own, table[:1], length), (q, own, table.long(), length), (q, own, table, length[1:]),
                (q, own, table, length.long()), (q, own, table, None), (torch.zeros(T, 6, 128, dtype=bf16)[..., ::2], own, table, length)):
        refused(f, *bad, cu=cu)
    refused(f, q, own, table, length)
    for kw in (dict(scale=math.nan), dict(scale=math.inf), dict(scale="1"), dict(out=out.float()), dict(out=out[1:]), dict(lse=lse[1:]),
               dict(lse=lse.double()), dict(lse=1), dict(workspace=torch.zeros(8)), dict(status=torch.zeros(1)), dict(cu=cu[1:])):
        refused(f, q, own, table, length, **{"cu": cu, **kw})
    own.v_scales = own.v_scales[1:]  # a cache that was changed
    refused(f, q, own, table, length, cu=cu)
    assert len(log.names) == n


def test_memory_of_another_stream(log):
    """What a call on stream 7 allocates comes from that stream; what the caller keeps may be read on the current one."""
    own = mlaq.KvCache.empty(8, 64, 2, 64, 32, device="cpu")
    table, length, cu = sequences()
    x, w, rstd = torch.zeros(6, 64, dtype=bf16), torch.ones(64), torch.zeros(6)
    for f, scratch in ((lambda s: mlaq.rms_norm_fwd(x, w, residual=x, save=True, stream=s), 0),
                       (lambda s: mlaq.rms_norm_bwd(x, x, w, rstd, stream=s), 1),
                       (lambda s: mlaq.kv_cache_read(own, table, length, 5, cu=cu, stream=s), 0),
                       (lambda s: mlaq.cache_attn(torch.zeros(5, 6, 64, dtype=bf16), own, table, length, cu=cu, lse=True, stream=s), 1)):
        log.made.clear(), log.recorded.clear()
        kept = f(Stream(7))
        assert len(log.made) == len(kept) + scratch and set(log.made.values()) == {7}
        assert {t.data_ptr(): 0 for t in kept} == log.recorded and log.current.cuda_stream == 0
        log.made.clear(), log.recorded.clear()
        f(Stream(0))  # the current one by name
        assert set(log.made.values()) == {0} and not log.recorded
