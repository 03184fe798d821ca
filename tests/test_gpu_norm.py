"""RMS norm on the GPU against its formula in 64 bits: types, row pitches, odd widths, the residual's sum, the MXFP8
results and the gradient.

Tolerances. Sums of K squares in float32, each thread's at most 32 terms and then a tree: below 64 roundings of 2^-24,
halved by the root; rstd and two products add three: with r = 2^-18 everything before the last rounding is covered. A
result in type t then is off by half a step, eps(t) / 2 of its value (an E4M3 code by 2^-4, or half the smallest step).
The gradient subtracts a mean: r times the sum of what it subtracts."""
import numpy as np
import pytest
import torch

import oracle
import up_proj_gemm_gb300 as mlaq
from up_proj_gemm_gb300 import autograd

pytestmark = pytest.mark.gpu
bf16, f32, f64 = torch.bfloat16, torch.float32, torch.float64
R = 2.0 ** -18


def half(t):
    return torch.finfo(t).eps / 2


def rows(T, K, dtype, pitch, seed, dev, std=1.0, shift=0):
    g = torch.Generator().manual_seed(seed)
    t = torch.randn((T, K + pitch), generator=g) * std * torch.exp(torch.randn((T, 1), generator=g))
    return t.to(dtype).to(dev)[:, shift:shift + K]


def formula(x, w, eps, residual=None):
    h = x.to(f64) if residual is None else x.to(f64) + residual.to(f64)
    rstd = (h.square().mean(1) + eps).rsqrt()
    return h, rstd, h * rstd[:, None] * w.to(f64)


def near(got, want, tol, what=""):
    d = (got.to(f64) - want).abs()
    bad = d > tol
    assert not bad.any(), (what, int(bad.sum()), float((d - tol).max()), got.shape)


# widths that take each way through the kernel: a warp to a row (1, 2, 4 and 8 granules), blocks of one to eight
SHAPES = [(1, 1), (1, 8), (3, 7), (1, 1536), (5, 33), (700, 64), (1300, 500), (2000, 1000), (1500, 1536), (2500, 2048),
          (40, 4096), (400, 4100), (310, 7168), (3, 16384), (2, 20000), (1, 32768), (320, 12288)]


@pytest.mark.parametrize("T,K", SHAPES)
@pytest.mark.parametrize("dtype,wtype,pitch,residual", [(bf16, bf16, 0, False), (bf16, f32, 24, True), (f32, f32, 4, True),
                                                        (f32, bf16, 3, False), (bf16, f32, 5, True)])
def test_forward(cuda_device, T, K, dtype, wtype, pitch, residual):
    x = rows(T, K, dtype, pitch, 1, cuda_device)
    w = (1 + rows(1, K, f32, 0, 2, cuda_device, 0.1)[0]).to(wtype)
    r = rows(T, K, dtype, 0, 3, cuda_device) if residual else None
    got = mlaq.rms_norm_fwd(x, w, eps=1e-5, residual=r, save=True)
    h, rstd, y = formula(x, w, 1e-5, r)
    near(got[-1], rstd, R * rstd, "rstd")
    near(got[0], y, (half(dtype) + R) * y.abs() + 1e-38, "y")
    if residual:
        near(got[1], h, half(dtype) * h.abs() + 2.0 ** -24 * (x.to(f64).abs() + r.to(f64).abs()), "h")
    again = mlaq.rms_norm_fwd(x, w, eps=1e-5, residual=r)
    assert torch.equal(again[0] if residual else again, got[0])


@pytest.mark.parametrize("T,K", [(1, 32), (1, 1536), (130, 96), (257, 1536), (2000, 1024), (300, 7168), (129, 160)])
@pytest.mark.parametrize("dtype,pitch,shift", [(bf16, 0, 0), (bf16, 576, 0), (f32, 5, 3)])
def test_mxfp8(cuda_device, T, K, dtype, pitch, shift):
    x = rows(T, K, dtype, pitch, 4, cuda_device, shift=shift)
    w = 1 + rows(1, K, f32, 0, 5, cuda_device, 0.2)[0]
    codes, scales, rstd = mlaq.rms_norm_fwd(x, w, out="mxfp8", save=True)
    _, _, y = formula(x, w, 1e-6)
    b = y.view(T, K // 32, 32)
    e = scales.to(torch.int32) - 127
    amax = b.abs().amax(2)
    top = torch.ldexp(torch.full_like(amax, 448.0), e)
    assert (amax <= top * (1 + R)).all() and (amax > top / 2 * (1 - R)).all()
    got = torch.ldexp(codes.view(torch.float8_e4m3fn).to(f64).view_as(b), e[..., None])
    near(got, b, 2.0 ** -4 * b.abs() + torch.ldexp(torch.full_like(amax, 2.0 ** -10), e)[..., None] + R * b.abs())
    tiled = mlaq.rms_norm_fwd(x, w, out="tiled")
    assert torch.equal(tiled[0], codes)
    assert np.array_equal(tiled[1].cpu().numpy(), oracle.mxfp8_swizzle_scales(scales.cpu().numpy()))


def test_special_values(cuda_device):
    """NaN and Inf stay in their row (and, as MXFP8, in their block); rows of zeros give zeros; eps 0."""
    x = rows(6, 256, bf16, 0, 6, cuda_device).clone()
    x[1, 7], x[2, 9], x[4] = float("nan"), float("inf"), 0
    w = torch.ones(256, device=cuda_device)
    y, rstd = mlaq.rms_norm_fwd(x, w, save=True)
    for t in (0, 3, 5):
        near(y[t:t + 1], formula(x[t:t + 1], w, 1e-6)[2], (half(bf16) + R) * formula(x[t:t + 1], w, 1e-6)[2].abs())
    assert y[1].isnan().all() and y[2, 9].isnan() and (y[2, :9] == 0).all() and (y[4] == 0).all()
    codes, scales = mlaq.rms_norm_fwd(x, w, out="mxfp8")
    assert (scales[1] == 255).all() and scales[2].tolist() == [255] + [0] * 7 and (scales[4] == 0).all()
    assert torch.equal(codes[[0, 3, 5]], mlaq.rms_norm_fwd(x[[0, 3, 5]], w, out="mxfp8")[0])
    assert mlaq.rms_norm_fwd(x[4:5], w, eps=0.0).isnan().all()  # 0 / 0
    assert mlaq.rms_norm_fwd(x[:0], w).shape == (0, 256)
    assert [tuple(t.shape) for t in mlaq.rms_norm_fwd(x[:0], w, residual=x[:0], out="tiled", save=True)] == [
        (0, 256), (0,), (0, 256), (0,)]


@pytest.mark.parametrize("T,K", SHAPES)
@pytest.mark.parametrize("dtype,wtype,pitch,dres", [(bf16, bf16, 0, False), (bf16, f32, 24, True), (f32, f32, 4, True),
                                                    (f32, bf16, 3, False)])
def test_gradient(cuda_device, T, K, dtype, wtype, pitch, dres):
    h = rows(T, K, dtype, pitch, 7, cuda_device)
    dy = rows(T, K, dtype, 2 * pitch, 8, cuda_device)
    w = (1 + rows(1, K, f32, 0, 9, cuda_device, 0.1)[0]).to(wtype)
    dh = rows(T, K, dtype, pitch, 10, cuda_device) if dres else None
    _, rstd = mlaq.rms_norm_fwd(h, w, save=True)
    dx, dw = mlaq.rms_norm_bwd(dy, h, w, rstd, dres=dh)
    r = rstd.to(f64)[:, None]
    n, g = h.to(f64) * r, dy.to(f64) * w.to(f64)
    mean, size = (g * n).mean(1, keepdim=True), (g * n).abs().mean(1, keepdim=True)
    want = r * (g - n * mean) + (0 if dh is None else dh.to(f64))
    slack = R * r * (g.abs() + n.abs() * size) + 2.0 ** -22 * want.abs() + (0 if dh is None else 2.0 ** -22 * dh.to(f64).abs())
    near(dx, want, half(dtype) * want.abs() + slack, "dx")
    # dw: T products in float32, at most T / 152 + 64 of them in a row
    want, size = (dy.to(f64) * n).sum(0), (dy.to(f64) * n).abs().sum(0)
    near(dw, want, half(wtype) * want.abs() + (T / 152 + 70) * 2.0 ** -24 * size + 1e-38, "dw")
    alone = mlaq.rms_norm_bwd(dy, h, w, rstd, dres=dh, dw=False)
    assert alone[1] is None and torch.equal(alone[0], dx)
    alone = mlaq.rms_norm_bwd(dy, h, w, rstd, dx=False)
    assert alone[0] is None and torch.equal(alone[1], dw)


def test_no_rows(cuda_device):
    z = torch.zeros((0, 96), dtype=bf16, device=cuda_device)
    dx, dw = mlaq.rms_norm_bwd(z, z, torch.ones(96, device=cuda_device), torch.zeros(0, device=cuda_device))
    assert dx.shape == (0, 96) and (dw == 0).all()


@pytest.mark.parametrize("residual", [False, True])
def test_autograd(cuda_device, residual):
    """Against the formula's derivatives by autograd in 64 bits, and against differences."""
    T, K = 33, 80
    x, r = (rows(T, K, f32, 0, s, cuda_device).clone().requires_grad_() for s in (11, 12))
    w = (1 + rows(1, K, f32, 0, 13, cuda_device, 0.1)[0]).clone().requires_grad_()
    cy, ch = rows(T, K, f32, 0, 14, cuda_device), rows(T, K, f32, 0, 15, cuda_device)

    def loss(x, w, r, y_of):
        y = y_of(x, w, r)
        return (y[0] * cy.to(y[0].dtype)).sum() + (y[1] * ch.to(y[1].dtype)).sum() if residual else (y * cy.to(y.dtype)).sum()

    def exact(x, w, r):
        h, _, y = formula(x, w, 1e-6, r if residual else None)
        return (y, h) if residual else y

    loss(x, w, r, lambda x, w, r: autograd.rms_norm(x, w, residual=r if residual else None)).backward()
    ref = [t.detach().to(f64).requires_grad_() for t in (x, w, r)]
    loss(*ref, exact).backward()
    for got, want in zip((x, w, r), ref):
        if want.grad is None:
            assert got.grad is None
            continue
        assert (got.grad.to(f64) - want.grad).norm() <= 1e-5 * want.grad.norm()
    d = torch.randn(x.shape, generator=torch.Generator().manual_seed(16)).to(cuda_device).to(f64)
    step = 1e-5
    with torch.no_grad():
        a, b = (loss(ref[0] + s * d, ref[1], ref[2], exact) for s in (step, -step))
    assert abs((a - b) / (2 * step) - (x.grad.to(f64) * d).sum()) <= 1e-4 * x.grad.to(f64).norm() * d.norm()


def test_autograd_parts(cuda_device):
    """Only what is asked for; expanded and strided upstream gradients; h used alone; no graph without gradients."""
    x = rows(9, 64, bf16, 0, 17, cuda_device).clone().requires_grad_()
    w = torch.ones(64, dtype=bf16, device=cuda_device)
    y = autograd.rms_norm(x, w)
    y.sum().backward()  # an expanded gradient
    assert x.grad.shape == x.shape and w.grad is None
    r = torch.ones_like(x).requires_grad_()
    y, h = autograd.rms_norm(x.detach(), w, residual=r)
    h.float().sum().backward()
    assert (r.grad == 1).all()
    with torch.no_grad():
        assert not autograd.rms_norm(x, w).requires_grad
    y = autograd.rms_norm(x, w)
    (g,) = torch.autograd.grad(y, x, torch.ones_like(y).t().contiguous().t(), create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_feeds_the_projection(cuda_device):
    """The MXFP8 results are the projection's operands, row-major and tiled alike."""
    T, K, H, Dn, Dr = 200, 256, 2, 64, 64
    x = rows(T, K, bf16, 64, 18, cuda_device)
    w = 1 + rows(1, K, f32, 0, 19, cuda_device, 0.1)[0]
    W, Ws = mlaq.mxfp8_quantize_rows(rows(H * (Dn + Dr), K, bf16, 0, 20, cuda_device, 0.05))
    cos, sin = torch.ones((T, Dr), device=cuda_device), torch.zeros((T, Dr), device=cuda_device)
    codes, scales = mlaq.rms_norm_fwd(x, w, out="mxfp8")
    q = mlaq.fwd(codes, W, cos, sin, H, Dn, Dr, weight_mode="mxfp8", x_scales=scales, w_scales=Ws, out_mode="bf16")
    G = mlaq.w_scale_group(T, K, H, Dn, Dr, T, Dr)
    tiled, ts = mlaq.rms_norm_fwd(x, w, out="tiled")
    q2 = mlaq.fwd(tiled, W, cos, sin, H, Dn, Dr, weight_mode="mxfp8_tiled", x_scales=ts,
                  w_scales=mlaq.mxfp8_swizzle_scales(Ws, group=G), out_mode="bf16")
    assert torch.equal(q, q2)

    def value(c, s):
        return torch.ldexp(c.view(torch.float8_e4m3fn).to(f64).unflatten(1, (-1, 32)), (s.to(torch.int32) - 127)[..., None]).flatten(1)

    a, b = value(codes, scales), value(W, Ws)
    near(q.flatten(1), a @ b.t(), half(bf16) * (a @ b.t()).abs() + K * 2.0 ** -22 * (a.abs() @ b.abs().t()))
