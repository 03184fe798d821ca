"""Gated feed-forward block against its formulas in 64 bits, stage by stage:
each product is checked on the bf16 operands the kernels used (g and u, h and
[dg | du] are read back), so every bound is one product's.

Bounds: a float32 sum of n products is off by at most (n + 8) * 2^-23 of the
sum of magnitudes, in any order; the activation's exp, erfc and division by 32
units of 2^-24 (|g| < 16). A bf16 result is the rounding of some value inside its
bound, and rounding is monotone: it lies between the roundings of the two ends.
"""
import pytest
import torch

import up_proj_gemm_gb300 as mlaq
from up_proj_gemm_gb300 import autograd as mlaq_grad

pytestmark = pytest.mark.gpu
bf16, f64 = torch.bfloat16, torch.float64
U = 2.0 ** -24


def make(T, K, F, pitch=0, seed=0, dev="cuda:0"):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g) * std).to(bf16).to(dev)

    return (normal(T, K + pitch)[:, :K], normal(2 * F, K, std=K ** -0.5), normal(K, F, std=F ** -0.5),
            normal(T, K, std=0.1))


def act64(g, act):
    g = g.clone().requires_grad_()
    with torch.enable_grad():
        a = (g * torch.sigmoid(g) if act == "silu" else
             torch.nn.functional.gelu(g, approximate="none" if act == "gelu" else "tanh"))
        (da,) = torch.autograd.grad(a.sum(), g)
    return a.detach(), da


def check(out, ref, bound, what):
    bound = bound + ref.abs() * U  # 64 bits are rounded to bf16 by way of float32
    out = out.to(f64)
    bad = (out < (ref - bound).to(bf16).to(f64)) | (out > (ref + bound).to(bf16).to(f64)) | ~torch.isfinite(out)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside their bounds"


def product(a, b):
    """a b^T in 64 bits and its bound."""
    a, b = a.to(f64), b.to(f64)
    return a @ b.t(), (a.shape[1] + 8) * 2 * U * (a.abs() @ b.abs().t())


def check_forward(x, wgu, wd, act, y, gu, h):
    F = wd.shape[1]
    ref, e = product(x, wgu)
    check(gu, ref, e, "gate_up")
    g, u, eg, eu = ref[:, :F], ref[:, F:], e[:, :F], e[:, F:]
    a, _ = act64(g, act)
    # |act'| <= 1.13 for the three of them
    check(h, a * u, eu * (a.abs() + 1.13 * eg) + 1.13 * eg * u.abs() + 32 * U * (a * u).abs() + 32 * U * u.abs() * g.abs() * 1e-3,
          "h")
    check(y, *product(h, wd), "y")


# T: one token, around the tile and step sizes; K, F: below, at and off the 64-element steps and 128/256 tiles
SHAPES = [(1, 64, 128), (1, 8, 8), (2, 136, 72), (17, 256, 520), (63, 64, 64), (64, 512, 256), (65, 72, 264),
          (127, 128, 136), (129, 200, 384), (255, 328, 128), (257, 1024, 8), (300, 8, 640), (700, 264, 392)]


@pytest.mark.parametrize("T,K,F", SHAPES)
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_forward(cuda_device, T, K, F, act):
    x, wgu, wd, _ = make(T, K, F, pitch=8 if T % 2 else 0, seed=T)
    st = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    y, gu, h = mlaq.gated_ffn_fwd(x, wgu, wd, act=act, save=True, status=st)
    mlaq.check_status(st)
    check_forward(x, wgu, wd, act, y, gu, h)
    assert torch.equal(mlaq.gated_ffn_fwd(x, wgu, wd, act=act), y)  # without saving: the same bits


@pytest.mark.parametrize("T,K,F", SHAPES)
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_backward(cuda_device, T, K, F, act):
    x, wgu, wd, dy = make(T, K, F, pitch=16 if T % 2 else 0, seed=T + 1)
    _, gu, h = mlaq.gated_ffn_fwd(x, wgu, wd, act=act, save=True)
    dgu = torch.empty((T, 2 * F), dtype=bf16, device=cuda_device)
    st = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    dx, dwgu, dwd = mlaq.gated_ffn_bwd(dy, x, wgu, wd, gu, h, act=act, dgate_up=dgu, status=st)
    mlaq.check_status(st)
    dh, e = product(dy, wd.t())
    g, u = gu.to(f64).split(F, 1)
    a, da = act64(g, act)
    check(dgu[:, :F], dh * u * da, e * (u * da).abs() + 64 * U * (dh * u).abs() * (1 + g.abs()), "dg")
    check(dgu[:, F:], dh * a, e * a.abs() + 64 * U * (dh * a).abs() + 32 * U * (dh * g).abs() * 1e-3, "du")
    check(dx, *product(dgu, wgu.t()), "dx")
    check(dwgu, *product(dgu.t(), x.t()), "dw_gate_up")
    check(dwd, *product(dy.t(), h.t()), "dw_down")


def test_parts_of_the_backward(cuda_device):
    """Each gradient alone: the same bits as all together, and only its own inputs are needed."""
    x, wgu, wd, dy = make(130, 136, 200)
    _, gu, h = mlaq.gated_ffn_fwd(x, wgu, wd, save=True)
    dx, dwgu, dwd = mlaq.gated_ffn_bwd(dy, x, wgu, wd, gu, h)
    a = mlaq.gated_ffn_bwd(dy, None, wgu, wd, gu, None, dw_gate_up=False, dw_down=False)
    b = mlaq.gated_ffn_bwd(dy, x, None, wd, gu, None, dx=False, dw_down=False)
    c = mlaq.gated_ffn_bwd(dy, None, None, None, None, h, dx=False, dw_gate_up=False)
    assert a[1] is a[2] is b[0] is b[2] is c[0] is c[1] is None
    assert torch.equal(a[0], dx) and torch.equal(b[1], dwgu) and torch.equal(c[2], dwd)


def test_no_tokens(cuda_device):
    x, wgu, wd, dy = make(0, 64, 128)
    y, gu, h = mlaq.gated_ffn_fwd(x, wgu, wd, save=True)
    assert y.shape == (0, 64) and gu.shape == (0, 256) and h.shape == (0, 128)
    dwgu = torch.full((256, 64), 7.0, dtype=bf16, device=cuda_device)
    dx, dwgu, dwd = mlaq.gated_ffn_bwd(dy, x, wgu, wd, gu, h, dw_gate_up=dwgu)
    assert dx.shape == (0, 64) and not dwgu.any() and not dwd.any()


def test_large_activations(cuda_device):
    """Gates far in the tails: finite, and the limits of the activations."""
    x, wgu, wd, dy = make(70, 64, 128)
    x, wgu = x.clone(), wgu.clone()
    wgu[:128] = 0
    wgu[:64, 0], wgu[64:128, 0] = 1.0, -1.0
    x[:, 0] = 20000.0
    for act in ("silu", "gelu", "gelu_tanh"):
        y, gu, h = mlaq.gated_ffn_fwd(x, wgu, wd, act=act, save=True)
        assert (gu[:, :64] == 20000.0 // 128 * 128).all() and not h[:, 64:].any()
        ref = gu[:, :64].to(f64) * (x.to(f64) @ wgu[128:192].to(f64).t())
        assert ((h[:, :64].to(f64) - ref).abs() <= 2.0 ** -7 * ref.abs().clamp(min=2.0 ** -7 * 20000 * 64)).all()
        for t in mlaq.gated_ffn_bwd(dy, x, wgu, wd, gu, h, act=act):
            assert torch.isfinite(t).all()


def test_a_nan_row_stays_in_its_row(cuda_device):
    x, wgu, wd, _ = make(200, 72, 136)
    y0 = mlaq.gated_ffn_fwd(x, wgu, wd)
    x = x.clone()
    x[150, 3] = float("nan")
    y = mlaq.gated_ffn_fwd(x, wgu, wd)
    assert torch.isnan(y[150]).all()
    keep = torch.arange(200, device=cuda_device) != 150
    assert torch.equal(y[keep], y0[keep])


def test_stays_inside_its_buffers(cuda_device):
    """Outputs handed in between guard rows: nothing around them is written."""
    T, K, F = 131, 72, 200
    x, wgu, wd, dy = make(T, K, F)

    def guarded(rows, cols):
        b = torch.full((rows + 2, cols), 7.0, dtype=bf16, device=cuda_device)
        return b, b[1:-1]

    bufs = [guarded(T, K), guarded(T, 2 * F), guarded(T, F), guarded(T, K), guarded(2 * F, K), guarded(K, F),
            guarded(T, 2 * F)]
    (_, y), (_, gu), (_, h), (_, dx), (_, dwgu), (_, dwd), (_, dgu) = bufs
    mlaq.gated_ffn_fwd(x, wgu, wd, save=True, y=y, gate_up=gu, h=h)
    check_forward(x, wgu, wd, "silu", y, gu, h)
    mlaq.gated_ffn_bwd(dy, x, wgu, wd, gu, h, dx=dx, dw_gate_up=dwgu, dw_down=dwd, dgate_up=dgu)
    check(dx, *product(dgu, wgu.t()), "dx")
    for b, _ in bufs:
        assert (b[0] == 7.0).all() and (b[-1] == 7.0).all()


def test_another_stream_and_repeatability(cuda_device):
    x, wgu, wd, dy = make(515, 264, 520)
    s = torch.cuda.Stream(cuda_device)
    s.wait_stream(torch.cuda.current_stream())
    y, gu, h = mlaq.gated_ffn_fwd(x, wgu, wd, save=True)
    torch.cuda.synchronize()
    out = torch.empty_like(y)
    mlaq.gated_ffn_fwd(x, wgu, wd, y=out, h=torch.empty_like(h), stream=s)
    s.synchronize()
    assert torch.equal(out, y)
    a = mlaq.gated_ffn_bwd(dy, x, wgu, wd, gu, h)
    b = mlaq.gated_ffn_bwd(dy, x, wgu, wd, gu, h)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gradients_against_differences(cuda_device, act):
    """Directional differences of the 64-bit formula. The kernels' gradients hold at most four bf16 roundings in a row
    (g and u, [dg | du], the result; 2^-8 each), so a directional derivative is off by at most 2^-6 of |grad| |dir|."""
    x, wgu, wd, dy = make(40, 64, 72, seed=3)

    def loss(x, wgu, wd):
        g, u = (x @ wgu.t()).split(72, 1)
        return ((act64(g, act)[0] * u) @ wd.t() * dy.to(f64)).sum()

    leaves = [t.clone().requires_grad_() for t in (x, wgu, wd)]
    mlaq_grad.gated_ffn(*leaves, act=act).backward(dy)
    wide = [t.to(f64) for t in (x, wgu, wd)]
    for i, leaf in enumerate(leaves):
        gen = torch.Generator().manual_seed(i)
        d = torch.randn(leaf.shape, generator=gen).to(f64).to(cuda_device)
        eps = 1e-5
        hi = loss(*[t + eps * d if j == i else t for j, t in enumerate(wide)])
        lo = loss(*[t - eps * d if j == i else t for j, t in enumerate(wide)])
        got = (leaf.grad.to(f64) * d).sum()
        assert abs(float(got - (hi - lo) / (2 * eps))) <= 2.0 ** -6 * float(leaf.grad.to(f64).norm() * d.norm())


# few tokens: padded counts around 16s, reductions split over 1, 2, 4 and 8 CTAs, ragged channel tiles and splits
FEW = [(1, 2048, 8), (1, 1032, 2000), (3, 520, 72), (8, 264, 10008), (16, 2056, 136), (17, 640, 328), (31, 1544, 64),
       (48, 72, 3000), (64, 1000, 1000), (80, 2048, 200), (96, 136, 136), (100, 1288, 520), (112, 64, 1032),
       (128, 776, 264)]


@pytest.mark.parametrize("T,K,F", FEW)
def test_few_tokens(cuda_device, T, K, F):
    x, wgu, wd, dy = make(T, K, F, pitch=24 if T % 2 else 0, seed=T + K)
    st = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    y, gu, h = mlaq.gated_ffn_fwd(x, wgu, wd, save=True, status=st)
    check_forward(x, wgu, wd, "silu", y, gu, h)
    dgu = torch.empty((T, 2 * F), dtype=bf16, device=cuda_device)
    dx, dwgu, dwd = mlaq.gated_ffn_bwd(dy, x, wgu, wd, gu, h, dgate_up=dgu, status=st)
    mlaq.check_status(st)
    dh, e = product(dy, wd.t())
    g, u = gu.to(f64).split(F, 1)
    a, da = act64(g, "silu")
    check(dgu[:, :F], dh * u * da, e * (u * da).abs() + 64 * U * (dh * u).abs() * (1 + g.abs()), "dg")
    check(dgu[:, F:], dh * a, e * a.abs() + 64 * U * (dh * a).abs() + 32 * U * (dh * g).abs() * 1e-3, "du")
    check(dx, *product(dgu, wgu.t()), "dx")
    check(dwgu, *product(dgu.t(), x.t()), "dw_gate_up")
    check(dwd, *product(dy.t(), h.t()), "dw_down")


def test_few_tokens_back_to_back(cuda_device):
    """Calls that reuse the same scratch and outputs, one behind the other: each product waits for the one it reads."""
    T, K, F = 4, 1024, 2048
    sets = [make(T, K, F, seed=i) for i in range(4)]
    want = [mlaq.gated_ffn_fwd(x, wgu, wd) for x, wgu, wd, _ in sets]
    torch.cuda.synchronize()
    h = torch.empty((T, F), dtype=bf16, device=cuda_device)
    ys = [torch.empty((T, K), dtype=bf16, device=cuda_device) for _ in range(40)]
    for i, y in enumerate(ys):
        x, wgu, wd, _ = sets[i % 4]
        mlaq.gated_ffn_fwd(x, wgu, wd, y=y, h=h)
    for i, y in enumerate(ys):
        assert torch.equal(y, want[i % 4])


def test_few_tokens_in_a_graph(cuda_device):
    x, wgu, wd, _ = make(5, 512, 1024)
    y = mlaq.gated_ffn_fwd(x, wgu, wd)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mlaq.gated_ffn_fwd(x, wgu, wd)
    x.copy_(torch.roll(x, 1, 0))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, torch.roll(y, 1, 0))


# many tokens: 256 x 256 tiles and their edges, reductions whole and split over 2, 3 and 4 pairs, tiles in several waves
MANY = [(1025, 264, 392), (1030, 1288, 520), (1100, 2056, 264), (1281, 136, 4104), (1111, 72, 5000), (2049, 520, 264),
        (1300, 1096, 1032), (5000, 8, 72), (3001, 136, 328)]


@pytest.mark.parametrize("T,K,F", MANY)
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_many_tokens(cuda_device, T, K, F, act):
    x, wgu, wd, dy = make(T, K, F, pitch=8, seed=T + K)
    st = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    y, gu, h = mlaq.gated_ffn_fwd(x, wgu, wd, act=act, save=True, status=st)
    check_forward(x, wgu, wd, act, y, gu, h)
    assert torch.equal(mlaq.gated_ffn_fwd(x, wgu, wd, act=act), y)
    dgu = torch.empty((T, 2 * F), dtype=bf16, device=cuda_device)
    dx, dwgu, dwd = mlaq.gated_ffn_bwd(dy, x, wgu, wd, gu, h, act=act, dgate_up=dgu, status=st)
    mlaq.check_status(st)
    dh, e = product(dy, wd.t())
    g, u = gu.to(f64).split(F, 1)
    a, da = act64(g, act)
    check(dgu[:, :F], dh * u * da, e * (u * da).abs() + 64 * U * (dh * u).abs() * (1 + g.abs()), "dg")
    check(dgu[:, F:], dh * a, e * a.abs() + 64 * U * (dh * a).abs() + 32 * U * (dh * g).abs() * 1e-3, "du")
    check(dx, *product(dgu, wgu.t()), "dx")
    check(dwgu, *product(dgu.t(), x.t()), "dw_gate_up")
    check(dwd, *product(dy.t(), h.t()), "dw_down")


def test_many_tokens_parts_and_guards(cuda_device):
    """Each gradient alone gives the bits of all together, between guard rows that stay."""
    T, K, F = 1111, 328, 520
    x, wgu, wd, dy = make(T, K, F)

    def guarded(rows, cols):
        b = torch.full((rows + 2, cols), 7.0, dtype=bf16, device=cuda_device)
        return b, b[1:-1]

    bufs = [guarded(T, K), guarded(T, 2 * F), guarded(T, F), guarded(T, K), guarded(2 * F, K), guarded(K, F),
            guarded(T, 2 * F)]
    (_, y), (_, gu), (_, h), (_, dx), (_, dwgu), (_, dwd), (_, dgu) = bufs
    mlaq.gated_ffn_fwd(x, wgu, wd, save=True, y=y, gate_up=gu, h=h)
    mlaq.gated_ffn_bwd(dy, x, wgu, wd, gu, h, dx=dx, dw_gate_up=dwgu, dw_down=dwd, dgate_up=dgu)
    check_forward(x, wgu, wd, "silu", y, gu, h)
    for b, _ in bufs:
        assert (b[0] == 7.0).all() and (b[-1] == 7.0).all()
    a = mlaq.gated_ffn_bwd(dy, None, wgu, wd, gu, None, dw_gate_up=False, dw_down=False)
    b = mlaq.gated_ffn_bwd(dy, x, None, wd, gu, None, dx=False, dw_down=False)
    c = mlaq.gated_ffn_bwd(dy, None, None, None, None, h, dx=False, dw_gate_up=False)
    assert torch.equal(a[0], dx) and torch.equal(b[1], dwgu) and torch.equal(c[2], dwd)


@pytest.mark.parametrize("T,K,F", [(1100, 512, 1024), (300, 2048, 512), (90, 512, 1024), (7, 264, 2048), (5000, 1024, 2048), (2000, 2000, 264)])
def test_weight_gradients_run_beside_dx(cuda_device, T, K, F):
    """The weights' gradients start before dx is finished: dx is whole for whoever comes after, call after call, and
    every bit is the one that a call for it alone gives."""
    g = torch.Generator().manual_seed(4)
    x, dy = ((torch.randn((T, K), generator=g)).to(torch.bfloat16).to(cuda_device) for _ in range(2))
    wgu, wd = (torch.randn(s, generator=g).mul(s[-1] ** -0.5).to(torch.bfloat16).to(cuda_device)
               for s in ((2 * F, K), (K, F)))
    y, gu, h = mlaq.gated_ffn_fwd(x, wgu, wd, save=True)
    alone = [mlaq.gated_ffn_bwd(dy, x, wgu, wd, gu, h, dx=i == 0, dw_gate_up=i == 1, dw_down=i == 2)[i] for i in range(3)]
    torch.cuda.synchronize()
    out = [torch.empty_like(t) for t in alone]
    kept = []
    for _ in range(8):
        for t in out:
            t.fill_(float("nan"))
        mlaq.gated_ffn_bwd(dy, x, wgu, wd, gu, h, dx=out[0], dw_gate_up=out[1], dw_down=out[2])
        kept.append([t.clone() for t in out])
    # and read by a kernel that itself starts under the last one: dx as the next call's dy
    got = mlaq.gated_ffn_bwd(out[0], x, wgu, wd, gu, h)
    torch.cuda.synchronize()
    want = mlaq.gated_ffn_bwd(alone[0], x, wgu, wd, gu, h)
    assert all(torch.equal(a, b) for k in kept for a, b in zip(k, alone))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T,K,F", [(1290, 2568, 1664), (1290, 3328, 2600), (1290, 2568, 3328)])
def test_last_wave_split(cuda_device, T, K, F):
    """A few tiles more than full waves of the gate and up, the down or dh product: these tiles' reductions are split, in
    a grid beside the others', and the bits are the same call after call."""
    x, wgu, wd, dy = make(T, K, F, seed=8)
    y, gu, h = mlaq.gated_ffn_fwd(x, wgu, wd, save=True)
    check_forward(x, wgu, wd, "silu", y, gu, h)
    dgu = torch.empty((T, 2 * F), dtype=bf16, device=cuda_device)
    grads = mlaq.gated_ffn_bwd(dy, x, wgu, wd, gu, h, dgate_up=dgu)
    dh, e = product(dy, wd.t())
    g, u = gu.to(f64).split(F, 1)
    a, da = act64(g, "silu")
    check(dgu[:, :F], dh * u * da, e * (u * da).abs() + 64 * U * (dh * u).abs() * (1 + g.abs()), "dg")
    check(dgu[:, F:], dh * a, e * a.abs() + 64 * U * (dh * a).abs() + 32 * U * (dh * g).abs() * 1e-3, "du")
    check(grads[0], *product(dgu, wgu.t()), "dx")
    for _ in range(4):
        assert torch.equal(mlaq.gated_ffn_fwd(x, wgu, wd), y)
        again = mlaq.gated_ffn_bwd(dy, x, wgu, wd, gu, h)
        assert all(torch.equal(b, c) for b, c in zip(grads, again))
