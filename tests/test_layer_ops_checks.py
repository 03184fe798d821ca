"""Refusals of the layer operators (feed-forward block, rotary axes, AdamW) without a GPU: the C entry points with
fake device addresses, and the binding with CPU tensors that report themselves as CUDA tensors."""
import contextlib
import ctypes

import pytest
import torch

import up_proj_gemm_gb300 as mlaq
from up_proj_gemm_gb300 import _build, ffn, optim, rotary

S = mlaq.STATUS
bf16, f32, u8, i32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
FAKE = 0x40000000


@pytest.fixture(scope="module")
def L():
    _build.build()
    return mlaq.lib()


def p(i, off=0):
    return ctypes.c_void_p(FAKE * (i + 1) + off)


# ------------------------------------------------------------ C entry points
def ffn_fwd(L, T=64, K=64, F=128, ld=0, act=0, reserved=0, **kw):
    s = mlaq.FfnShape(T, K, F, ld, act, reserved)
    a = dict(x=p(0), wgu=p(1), wd=p(2), gu=p(3), h=p(4), y=p(5), st=None)
    a.update(kw)
    return L.mla_gated_ffn_fwd(ctypes.byref(s), a["x"], a["wgu"], a["wd"], a["gu"], a["h"], a["y"], a["st"], None)


def test_ffn_forward_refusals(L):
    inv, al, alias = S["MLA_ERR_INVALID_ARG"], S["MLA_ERR_ALIGNMENT"], S["MLA_ERR_ALIAS"]
    assert ffn_fwd(L) in (S["MLA_ERR_CUDA"], S["MLA_OK"])  # valid: refused for want of a device only
    for kw in (dict(T=-1), dict(K=0), dict(F=0), dict(act=3), dict(act=-1), dict(reserved=1), dict(ld=56), dict(ld=-8),
               dict(T=2**31), dict(x=None), dict(wgu=None), dict(wd=None), dict(h=None), dict(y=None)):
        assert ffn_fwd(L, **kw) == inv, kw
    for kw in (dict(K=60), dict(F=132), dict(ld=68), dict(x=p(0, 8)), dict(h=p(4, 2)), dict(gu=p(3, 4)), dict(st=p(6, 2))):
        assert ffn_fwd(L, **kw) == al, kw
    for kw in (dict(h=p(0)), dict(y=p(4)), dict(gu=p(4, 16)), dict(y=p(2, 64 * 128 * 2 - 16)), dict(st=p(1))):
        assert ffn_fwd(L, **kw) == alias, kw
    # a pitched x spans (T - 1) ld + K elements
    assert ffn_fwd(L, ld=128, y=p(0, (63 * 128 + 64) * 2)) != alias
    assert ffn_fwd(L, ld=128, y=p(0, (63 * 128 + 64) * 2 - 16)) == alias
    assert ffn_fwd(L, T=0, x=None, wgu=None, wd=None, gu=None, h=None, y=None) == S["MLA_OK"]
    assert L.mla_gated_ffn_fwd(None, *[None] * 8) == inv


def ffn_bwd(L, T=64, K=64, F=128, **kw):
    s = mlaq.FfnShape(T, K, F, 0, 0, 0)
    a = dict(dy=p(0), x=p(1), wgu=p(2), wd=p(3), gu=p(4), h=p(5), dgu=p(6), dx=p(7), dwgu=p(8), dwd=p(9), st=None)
    a.update(kw)
    return L.mla_gated_ffn_bwd(ctypes.byref(s), *[a[n] for n in ("dy", "x", "wgu", "wd", "gu", "h", "dgu", "dx", "dwgu",
                                                                 "dwd", "st")], None)


def test_ffn_backward_refusals(L):
    inv, alias = S["MLA_ERR_INVALID_ARG"], S["MLA_ERR_ALIAS"]
    ok = (S["MLA_ERR_CUDA"], S["MLA_OK"])
    assert ffn_bwd(L) in ok
    assert ffn_bwd(L, dx=None, dwgu=None, dwd=None) == inv
    for n in ("dy", "x", "wgu", "wd", "gu", "h", "dgu"):
        assert ffn_bwd(L, **{n: None}) == inv, n
    assert ffn_bwd(L, dx=None, dwgu=None, x=None, wgu=None, wd=None, gu=None, dgu=None) in ok
    assert ffn_bwd(L, dwd=None, dwgu=None, x=None, h=None) in ok
    assert ffn_bwd(L, dwd=None, dx=None, wgu=None, h=None) in ok
    for kw in (dict(dx=p(0)), dict(dgu=p(4)), dict(dwd=p(8)), dict(dwgu=p(2))):
        assert ffn_bwd(L, **kw) == alias, kw
    assert ffn_bwd(L, dwd=p(9, 8)) == S["MLA_ERR_ALIGNMENT"]


def rope(L, T=8, H=4, Dn=16, Dr=32, axes=3, rows=64, width=32, strides=None, dtype=1, mode=0, pair=None, reserved=0, **kw):
    D = Dn + Dr
    st = strides or (H * D, D, H * D, D)
    s = mlaq.RopeAxesShape(T, H, Dn, Dr, axes, rows, width, *st, reserved)
    a = dict(x=p(0), cos=p(1), sin=p(2), pos=p(3), out=p(4), st=None)
    a.update(kw)
    pair = bytes([i % 3 for i in range(Dr // 2)]) if pair is None else pair
    return L.mla_rope_axes(ctypes.byref(s), dtype, mode, a["x"], a["cos"], a["sin"], a["pos"], pair, a["out"], a["st"], None)


def test_rope_axes_refusals(L):
    inv, al, alias = S["MLA_ERR_INVALID_ARG"], S["MLA_ERR_ALIGNMENT"], S["MLA_ERR_ALIAS"]
    ok = (S["MLA_ERR_CUDA"], S["MLA_OK"])
    assert rope(L) in ok
    for kw in (dict(T=-1), dict(H=0), dict(Dr=31), dict(Dr=0), dict(axes=0), dict(dtype=2), dict(mode=3), dict(mode=-1),
               dict(reserved=1), dict(axes=2), dict(x=None), dict(cos=None), dict(pos=None), dict(out=None),
               dict(strides=(192, 48, 192, 40)), dict(strides=(192, 48, 100, 48)), dict(strides=(-1, 48, 192, 48)),
               dict(T=2**30, H=4)):
        assert rope(L, **kw) == inv, kw
    assert rope(L, width=31) == S["MLA_ERR_ROPE_WIDTH"]
    assert rope(L, rows=0) == S["MLA_ERR_POS_RANGE"]
    assert rope(L, Dr=258, width=258) == S["MLA_ERR_UNSUPPORTED"]
    assert rope(L, Dn=8192) == S["MLA_ERR_UNSUPPORTED"]
    for kw in (dict(x=p(0, 1)), dict(out=p(4, 1)), dict(cos=p(1, 2)), dict(pos=p(3, 2)), dict(dtype=0, x=p(0, 2))):
        assert rope(L, **kw) == al, kw
    for kw in (dict(out=p(0)), dict(out=p(0, 8 * 192 * 2 - 2)), dict(out=p(1)), dict(out=p(3, 92)), dict(st=p(0))):
        assert rope(L, **kw) == alias, kw
    assert rope(L, out=p(3, 96)) in ok                              # right behind the positions
    assert rope(L, strides=(48, 8 * 48, 48, 8 * 48)) in ok          # head-major on both sides
    assert rope(L, strides=(192, 0, 192, 48)) in ok                 # one head for all
    assert rope(L, mode=2, strides=(192, 48, 48, 0)) in ok          # one head comes out
    assert rope(L, mode=2, strides=(192, 48, 40, 0)) == inv
    assert rope(L, T=0, x=None, cos=None, sin=None, pos=None, out=None) == S["MLA_OK"]


def test_rope_table_refusals(L):
    s = mlaq.RopeAxesShape(8, 1, 0, 32, 3, 64, 32, 0, 0, 0, 0, 0)
    pair = bytes([i % 3 for i in range(16)])
    f = lambda *a: L.mla_rope_axes_table(ctypes.byref(s), *a)  # noqa: E731
    assert f(p(1), p(2), p(3), pair, p(4), p(5), None, None) in (S["MLA_ERR_CUDA"], S["MLA_OK"])
    assert f(p(1), p(2), p(3), pair, None, p(5), None, None) == S["MLA_ERR_INVALID_ARG"]
    assert f(p(1), p(2), p(3), pair, p(4, 8), p(5), None, None) == S["MLA_ERR_ALIGNMENT"]
    assert f(p(1), p(2), p(3), pair, p(4), p(4), None, None) == S["MLA_ERR_ALIAS"]
    assert f(p(1), p(2), p(3), pair, p(1), p(5), None, None) == S["MLA_ERR_ALIAS"]


def plan(L, rows, pt=1, gt=1, bits=32, size=None):
    a = (optim._Tensor * len(rows))(*[optim._Tensor(*r) for r in rows])
    n = int(L.mla_adamw_plan_bytes(a, len(rows)))
    buf = ctypes.create_string_buffer(max(n, 64))
    return L.mla_adamw_plan_build(a, len(rows), pt, gt, bits, ctypes.addressof(buf), n if size is None else size), buf, n


def a(i, off=0):
    return FAKE * (i + 1) + off


def test_adamw_refusals(L):
    inv, al, alias = S["MLA_ERR_INVALID_ARG"], S["MLA_ERR_ALIGNMENT"], S["MLA_ERR_ALIAS"]
    one = (a(0), a(1), a(2), a(3), None, None, None, 100)
    eight = (a(0), a(1), a(2), a(3), a(4), a(5), None, 100)
    assert plan(L, [one])[0] == S["MLA_OK"] and plan(L, [eight], bits=8)[0] == S["MLA_OK"]
    for kw in (dict(pt=2), dict(gt=-1), dict(bits=16)):
        assert plan(L, [one], **kw)[0] == inv, kw
    assert plan(L, [eight])[0] == inv and plan(L, [one], bits=8)[0] == inv
    assert plan(L, [one], size=8)[0] == S["MLA_ERR_WORKSPACE"]
    for i in range(4):
        assert plan(L, [one[:i] + (None,) + one[i + 1:]])[0] == inv, i
    assert plan(L, [one[:7] + (-1,)])[0] == inv
    assert plan(L, [(None,) * 7 + (0,), one])[0] == S["MLA_OK"]                # an empty tensor needs nothing
    assert plan(L, [(a(0, 1),) + one[1:]])[0] == al and plan(L, [one[:2] + (a(2, 2),) + one[3:]])[0] == al
    assert plan(L, [one[:6] + (a(0, 100), 100)])[0] == alias                   # the master inside the parameter
    assert plan(L, [one[:6] + (a(0, 200), 100)])[0] == S["MLA_OK"]             # and right behind it
    assert plan(L, [one, one])[0] == alias                                     # a tensor listed twice
    two = (a(6), a(1), a(7), a(8), None, None, None, 100)
    assert plan(L, [one, two])[0] == S["MLA_OK"]                               # gradients may share memory
    assert plan(L, [one, (a(6), a(0, 50), a(7), a(8), None, None, None, 4)])[0] == alias  # a gradient inside a parameter
    _, buf, n = plan(L, [one])
    step = lambda host=ctypes.addressof(buf), dev=a(20), gs=None, **kw: L.mla_adamw_step(  # noqa: E731
        host, dev, ctypes.byref(optim._Args(**{**dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=1,
                                                      stochastic=0, seed=0), **kw})), gs, None)
    assert step() in (S["MLA_ERR_CUDA"], S["MLA_OK"])
    for kw in (dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1.0), dict(step=0), dict(lr=float("nan")), dict(stochastic=2),
               dict(host=None), dict(dev=None)):
        assert step(**kw) == inv, kw
    assert step(dev=a(20, 8)) == al and step(gs=a(21, 2)) == al
    junk = ctypes.create_string_buffer(64)
    assert step(host=ctypes.addressof(junk)) == inv
    assert L.mla_adamw_plan_bytes(None, 1) == 0 and L.mla_adamw_plan_bytes((optim._Tensor * 1)(), 0) == 0


# ------------------------------------------------------------------ binding
@pytest.fixture
def calls(L, monkeypatch):
    log = []
    for m in (ffn, rotary, optim):
        real = m._call

        def call(fn, what, *args, real=real):
            if what == "mla_adamw_plan_build":
                return real(fn, what, *args)
            log.append(what)

        monkeypatch.setattr(m, "_call", call)
        monkeypatch.setattr(m, "_stream", lambda device, stream: None)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: FakeStream())
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    return log


class FakeStream:
    cuda_stream = 0

    def record_event(self):
        return None


def refused(f, *a, **kw):
    with pytest.raises((TypeError, ValueError)):
        f(*a, **kw)


def test_ffn_binding(calls):
    T, K, F = 5, 16, 24
    x, wgu, wd = torch.zeros(T, K, dtype=bf16), torch.zeros(2 * F, K, dtype=bf16), torch.zeros(K, F, dtype=bf16)
    wide = torch.zeros(T, K + 8, dtype=bf16)[:, :K]
    f = mlaq.gated_ffn_fwd
    y, gu, h = f(wide, wgu, wd, save=True)
    assert calls == ["mla_gated_ffn_fwd"] and y.shape == (T, K) and gu.shape == (T, 2 * F) and h.shape == (T, F)
    f(x, wgu, wd, act="gelu", y=y, h=h, gate_up=gu)
    for bad in ((x.float(), wgu, wd), (x[0], wgu, wd), (x.t(), wgu, wd), (x, wgu[1:], wd), (x, wgu, wd[:, 1:]),
                (x, wgu.float(), wd), (x, wgu, wd.t()), (None, wgu, wd), (x, None, wd), (x, wgu, None)):
        refused(f, *bad)
    for kw in (dict(act="tanh"), dict(y=y[1:]), dict(h=h.float()), dict(gate_up=h), dict(status=torch.zeros(1))):
        refused(f, x, wgu, wd, **kw)
    b, dy = mlaq.gated_ffn_bwd, torch.zeros(T, K, dtype=bf16)
    n = len(calls)
    dx, dwgu, dwd = b(dy, x, wgu, wd, gu, h)
    assert len(calls) == n + 1 and dx.shape == x.shape and dwgu.shape == wgu.shape and dwd.shape == wd.shape
    b(dy, None, None, None, None, h, dx=False, dw_gate_up=False)
    refused(b, dy, x, wgu, wd, gu, h, dx=False, dw_gate_up=False, dw_down=False)
    for bad in ((dy.float(), x, wgu, wd, gu, h), (dy[1:], x, wgu, wd, gu, h), (dy, x[1:], wgu, wd, gu, h),
                (dy, x, wgu[1:], wd, gu, h), (dy, x, wgu, wd[1:], gu, h), (dy, x, wgu, wd, gu[:, 1:], h),
                (dy, x, wgu, wd, gu, h[1:]), (dy, None, wgu, wd, gu, h), (dy, x, wgu, wd, None, h)):
        refused(b, *bad)
    refused(b, dy, x, wgu, wd, gu, h, dx=dx[1:])
    refused(b, dy, x, wgu, wd, gu, h, dgate_up=h)
    assert len(calls) == n + 2


def test_rope_binding(calls):
    T, H, Dr = 6, 3, 8
    x = torch.zeros(T, H, 12, dtype=bf16)
    cos = torch.zeros(32, 8)
    pos, axes = torch.zeros(2, T, dtype=i32), [0, 0, 1, 1]
    f = mlaq.rope_axes
    assert f(x, cos, cos, pos, axes, Dr).shape == x.shape
    assert f(x, cos, cos, pos, axes, Dr, inverse=True, sum_heads=True).shape == (T, 1, 12)
    assert f(x[:, :1].expand(T, 5, 12), cos, cos, pos, axes, Dr).shape == (T, 5, 12)
    f(x, cos, cos, pos, bytes(axes), Dr, out=torch.zeros(T, H, 20, dtype=bf16)[:, :, 8:])
    assert mlaq.rope_sections((2, 1, 1)) == bytes([0, 0, 1, 2])
    n = len(calls)
    for bad in ((None, cos, cos, pos, axes, Dr), (x.double(), cos, cos, pos, axes, Dr), (x[0], cos, cos, pos, axes, Dr),
                (x.transpose(1, 2), cos, cos, pos, axes, Dr), (x, cos, cos, pos, axes, 14), (x, cos, cos, pos, axes, 0),
                (x, cos.double(), cos, pos, axes, Dr), (x, cos, cos[1:], pos, axes, Dr), (x, cos, cos, pos[0], axes, Dr),
                (x, cos, cos, pos[:, 1:], axes, Dr), (x, cos, cos, pos.long(), axes, Dr),
                (x, cos, cos, pos, axes[1:], Dr), (x, cos.t(), cos.t(), pos, axes, Dr), (x, None, cos, pos, axes, Dr)):
        refused(f, *bad)
    for kw in (dict(sum_heads=True), dict(out=x.float()), dict(out=x[1:]), dict(status=torch.zeros(1))):
        refused(f, x, cos, cos, pos, axes, Dr, **kw)
    g = mlaq.rope_axes_table
    c, s = g(cos, cos, pos, axes, Dr)
    assert c.shape == s.shape == (T, Dr)
    for bad in ((cos, cos, pos[0], axes, Dr), (cos, cos, None, axes, Dr), (cos, cos, pos, axes[1:], Dr)):
        refused(g, *bad)
    refused(g, cos, cos, pos, axes, Dr, cos_out=c[1:])
    assert len(calls) == n + 1


def test_adamw_binding(calls):
    p, g, m, v = ([torch.zeros(5, 7), torch.zeros(40)] for _ in range(4))
    q = mlaq.adamw_plan(p, g, m, v)
    mlaq.adamw_step(q, 1, lr=1e-3)
    assert calls == ["mla_adamw_step"]
    codes = lambda: [torch.zeros(5, 7, dtype=u8), torch.zeros(40, dtype=u8)]  # noqa: E731
    scales = lambda: [torch.zeros(2, dtype=u8), torch.zeros(2, dtype=u8)]  # noqa: E731
    mlaq.adamw_plan([t.to(bf16) for t in p], [t.to(bf16) for t in g], codes(), codes(), masters=m,
                    exp_avg_scales=scales(), exp_avg_sq_scales=scales())
    for bad in (([], [], [], []), (p, g[1:], m, v), (p, [t[1:] for t in g], m, v), (p, g, m, [t.to(bf16) for t in v]),
                ([t.double() for t in p], g, m, v), ([p[0].t(), p[1]], g, m, v), (p, [g[0], g[1].to(bf16)], m, v),
                (p, g, codes(), codes())):
        refused(mlaq.adamw_plan, *bad)
    refused(mlaq.adamw_plan, p, g, m, v, exp_avg_scales=scales(), exp_avg_sq_scales=scales())
    refused(mlaq.adamw_plan, p, g, codes(), codes(), exp_avg_scales=[t[1:] for t in scales()], exp_avg_sq_scales=scales())
    refused(mlaq.adamw_plan, p, g, m, v, masters=[t.to(bf16) for t in m])
    with pytest.raises(mlaq.MlaError):
        mlaq.adamw_plan(p, g, m, m)  # the moments overlap
    refused(mlaq.adamw_step, None, 1, lr=1e-3)
    refused(mlaq.adamw_step, q, 1, lr=1e-3, grad_scale=torch.zeros(2))
    refused(mlaq.AdamW, p, 1e-3, state_bits=16)
    opt = mlaq.AdamW([torch.nn.Parameter(t) for t in p], 1e-3)
    refused(opt.step)
