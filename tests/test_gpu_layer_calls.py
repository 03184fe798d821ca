"""The compiled calls of the layer operators and their Python face: the same results, and the same refusals on real
CUDA tensors, whichever of the two serves the call."""
import pytest
import torch

import up_proj_gemm_gb300 as mlaq

pytestmark = pytest.mark.gpu
bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(params=["compiled", "python"])
def face(request, monkeypatch):
    mlaq.lib()
    if request.param == "python":
        monkeypatch.setattr(mlaq, "_calls", None)
    elif mlaq._calls is None:
        pytest.skip("calls.cpp was not built here")
    return request.param


def tensors(dev):
    g = torch.Generator().manual_seed(1)

    def normal(*s, dtype=bf16):
        return torch.randn(s, generator=g).to(dtype).to(dev)

    T, K, F = 9, 64, 72
    return dict(x=normal(T, K), wgu=normal(2 * F, K), wd=normal(K, F), dy=normal(T, K), q=normal(T, 3, 24),
                cos=normal(32, 16, dtype=f32), sin=normal(32, 16, dtype=f32),
                pos=torch.randint(0, 32, (2, T), generator=g).to(i32).to(dev), axes=[0, 1] * 4)


def results(d, calls):
    """Every operator once, by the compiled calls or not."""
    keep = mlaq._calls
    mlaq._calls = calls
    try:
        y, gu, h = mlaq.gated_ffn_fwd(d["x"], d["wgu"], d["wd"], act="gelu", save=True)
        out = [y, gu, h, mlaq.gated_ffn_fwd(d["x"], d["wgu"], d["wd"])]
        out += mlaq.gated_ffn_bwd(d["dy"], d["x"], d["wgu"], d["wd"], gu, h, act="gelu")
        r = (d["cos"], d["sin"], d["pos"], d["axes"], 16)
        out += [mlaq.rope_axes(d["q"], *r), mlaq.rope_axes(d["q"], *r, inverse=True),
                mlaq.rope_axes(d["q"].float(), *r, inverse=True, sum_heads=True),
                mlaq.rope_axes(d["q"][:, :1].expand(-1, 5, -1), *r), mlaq.rope_axes(d["q"].transpose(0, 1)[:, :2].transpose(
                    0, 1), *r[:2], d["pos"][:, :2].contiguous(), *r[3:])]
        out += mlaq.rope_axes_table(*r)
        p = [torch.full((50,), 0.5, device=d["x"].device), torch.ones(3, device=d["x"].device)]
        s = [[torch.zeros_like(t) for t in p] for _ in range(2)]
        plan = mlaq.adamw_plan(p, [torch.ones_like(t) for t in p], *s)
        mlaq.adamw_step(plan, 1, lr=0.1, grad_scale=torch.full((1,), 0.5, device=d["x"].device))
        mlaq.adamw_step(plan, 2, lr=0.1, seed=3)
        return out + p + s[0] + s[1]
    finally:
        mlaq._calls = keep


def test_both_faces_give_the_same_bits(cuda_device):
    mlaq.lib()
    if mlaq._calls is None:
        pytest.skip("calls.cpp was not built here")
    d = tensors(cuda_device)
    a, b = results(d, mlaq._calls), results(d, None)
    assert len(a) == len(b)
    for i, (s, t) in enumerate(zip(a, b)):
        assert s.shape == t.shape and s.dtype == t.dtype and s.stride() == t.stride() and torch.equal(s, t), i
        assert not s.requires_grad


def test_refusals(cuda_device, face):
    d = tensors(cuda_device)
    x, wgu, wd = d["x"], d["wgu"], d["wd"]
    for bad in ((x.float(), wgu, wd), (x[0], wgu, wd), (x, wgu[1:], wd), (x, wgu, wd[:, 1:]), (x.cpu(), wgu, wd),
                (x, wgu.cpu(), wd), (None, wgu, wd), (x, wgu, wd.t().contiguous())):
        with pytest.raises((TypeError, ValueError)):
            mlaq.gated_ffn_fwd(*bad)
    with pytest.raises(ValueError):
        mlaq.gated_ffn_fwd(x, wgu, wd, act="relu")
    with pytest.raises(mlaq.MlaError):  # 63 channels: rows off the 16-byte grid
        mlaq.gated_ffn_fwd(x[:, :63].contiguous(), wgu[:, :63].contiguous(), wd[:63].contiguous())
    y, gu, h = mlaq.gated_ffn_fwd(x, wgu, wd, save=True)
    for bad in ((d["dy"], x[1:], wgu, wd, gu, h), (d["dy"], x, wgu, wd, gu[:, 1:], h), (d["dy"], x, wgu, wd, gu, h.float())):
        with pytest.raises((TypeError, ValueError)):
            mlaq.gated_ffn_bwd(*bad)
    q, cos, sin, pos, axes = (d[n] for n in ("q", "cos", "sin", "pos", "axes"))
    for bad in ((q.double(), cos, sin, pos, axes, 16), (q, cos, sin[1:], pos, axes, 16), (q, cos, sin, pos.long(), axes, 16),
                (q, cos, sin, pos[:, 1:], axes, 16), (q, cos, sin, pos, axes[1:], 16), (q, cos, sin, pos.cpu(), axes, 16),
                (q, cos, sin, pos, axes, 26), (q.cpu(), cos, sin, pos, axes, 16)):
        with pytest.raises((TypeError, ValueError)):
            mlaq.rope_axes(*bad)
    with pytest.raises(ValueError):
        mlaq.rope_axes(q, cos, sin, pos, axes, 16, sum_heads=True)
    with pytest.raises(mlaq.MlaError) as e:  # an axis that pos does not have
        mlaq.rope_axes(q, cos, sin, pos, [2] * 8, 16)
    assert e.value.status == mlaq.STATUS["MLA_ERR_INVALID_ARG"]
    with pytest.raises(mlaq.MlaError) as e:
        mlaq.rope_axes(q, cos[:, :8].contiguous(), sin[:, :8].contiguous(), pos, axes, 16)
    assert e.value.status == mlaq.STATUS["MLA_ERR_ROPE_WIDTH"]
    with pytest.raises((TypeError, ValueError)):
        mlaq.rope_axes_table(cos, sin, pos[0], axes, 16)
    p = [torch.ones(4, device=cuda_device)]
    plan = mlaq.adamw_plan(p, [torch.ones_like(p[0])], [torch.zeros_like(p[0])], [torch.zeros_like(p[0])])
    with pytest.raises(mlaq.MlaError):
        mlaq.adamw_step(plan, 0, lr=0.1)
    with pytest.raises((TypeError, ValueError)):
        mlaq.adamw_step(plan, 1, lr=0.1, grad_scale=torch.ones(2, device=cuda_device))
    assert torch.equal(p[0], torch.ones_like(p[0]))


def test_current_stream_is_used(cuda_device, face):
    """Work goes to the current stream: a long kernel before it on that stream is waited for."""
    d = tensors(cuda_device)
    want = mlaq.rope_axes(d["q"], d["cos"], d["sin"], d["pos"], d["axes"], 16)
    torch.cuda.synchronize()
    side = torch.cuda.Stream(cuda_device)
    q = torch.zeros_like(d["q"])
    with torch.cuda.stream(side):
        a = torch.randn((4096, 4096), device=cuda_device)
        for _ in range(8):
            a = a @ a
            a = a / a.norm()
        q.copy_(d["q"])
        out = mlaq.rope_axes(q, d["cos"], d["sin"], d["pos"], d["axes"], 16)
    side.synchronize()
    assert torch.equal(out, want)


def test_overlapped_launches_keep_the_order(cuda_device):
    """Launches start under the ones before them; what they read and write stays in order: parameters are stepped and
    used by the next product, its output rotated, buffers reused, many times in a row and in a graph."""
    dev = cuda_device
    g = torch.Generator().manual_seed(2)
    T, K, F = 6, 256, 512
    w = [torch.randn(s, generator=g).to(dev) * s[-1] ** -0.5 for s in ((2 * F, K), (K, F))]
    x = torch.randn((T, K), generator=g).to(bf16).to(dev)
    cos, sin = torch.randn((64, 32), generator=g).to(dev), torch.randn((64, 32), generator=g).to(dev)
    pos = torch.randint(0, 64, (3, T), generator=g).to(i32).to(dev)
    axes = [i % 3 for i in range(16)]

    def chain(sync):
        p = [t.to(bf16) for t in w]
        grad = [torch.full_like(t, 1e-2) for t in p]
        m, v = ([torch.zeros(t.shape, device=dev) for t in p] for _ in range(2))
        plan = mlaq.adamw_plan(p, grad, m, v)
        h, y = torch.empty((T, F), dtype=bf16, device=dev), torch.empty((T, K), dtype=bf16, device=dev)
        z, outs = x.clone(), []
        wait = torch.cuda.synchronize if sync else (lambda: None)
        for step in range(1, 31):
            mlaq.adamw_step(plan, step, lr=1e-2, weight_decay=0.0)
            wait()
            mlaq.gated_ffn_fwd(z, p[0], p[1], y=y, h=h)
            wait()
            mlaq.rope_axes(y.view(T, 8, 32), cos, sin, pos, axes, 32, out=z.view(T, 8, 32))
            wait()
            z = z.float().clamp(-2, 2).to(bf16) if step % 7 == 0 else z
            outs.append(mlaq.rope_axes(z.view(T, 8, 32), cos, sin, pos, axes, 32, inverse=True, sum_heads=True))
            wait()
        return outs + [z] + p

    want, got = chain(True), chain(False)
    torch.cuda.synchronize()
    assert all(torch.equal(a.nan_to_num(), b.nan_to_num()) for a, b in zip(want, got))
