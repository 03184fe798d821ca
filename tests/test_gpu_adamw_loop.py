"""AdamW as a training loop uses it."""
import numpy as np
import pytest
import torch

import oracle
import up_proj_gemm_gb300 as mlaq

pytestmark = pytest.mark.gpu
bf16 = torch.bfloat16
E4M3 = np.array([oracle.e4m3_decode(c) for c in range(256)])


def test_a_moved_parameter_is_stepped(cuda_device):
    """p.data is another buffer from the second step on, the gradient's stays: the visible parameter moves, the buffer
    it left does not."""
    p = torch.nn.Parameter(torch.ones(1000, device=cuda_device))
    p.grad = torch.ones_like(p)
    opt = mlaq.AdamW([p], lr=0.25, weight_decay=0.0)
    opt.step()
    left = p.data
    kept = left.clone()
    p.data = left.clone()
    opt.step()
    # two steps of lr each on gradients of one: off by 16 * 2^-24 of a step each and 3 * 2^-24 of the parameter
    assert ((p.detach().double() - 0.5).abs() <= 40 * 2.0 ** -24).all()
    assert torch.equal(left, kept)


@pytest.mark.parametrize("name", ["exp_avg", "exp_avg_sq", "masters"])
def test_replaced_state_is_stepped(cuda_device, name):
    """A state that is put back by replacing its tensors is the one that the next step reads and writes."""
    p = torch.nn.Parameter(torch.ones(500, device=cuda_device, dtype=bf16))
    p.grad = torch.ones_like(p)
    opt = mlaq.AdamW([p], lr=0.25, weight_decay=0.0, masters=True)
    opt.step()
    left = getattr(opt, name)[0]
    kept = left.clone()
    fresh = left.clone()
    getattr(opt, name)[0] = fresh
    opt.step()
    assert torch.equal(left, kept) and not torch.equal(fresh, kept)


def test_gradients_are_not_kept(cuda_device):
    """With p.grad = None after a step, the gradients' memory is free: only parameters, moments and a plan remain."""
    n = 1 << 22
    p = torch.nn.Parameter(torch.ones(n, device=cuda_device))
    opt = mlaq.AdamW([p], lr=1e-3)
    before = torch.cuda.memory_allocated(cuda_device)
    for _ in range(3):
        p.grad = torch.ones_like(p)
        opt.step()
        p.grad = None
        assert torch.cuda.memory_allocated(cuda_device) - before < n  # the gradient is 4 n bytes


def decoded(codes, scales):
    e = np.repeat(scales.cpu().numpy().astype(np.int64) - 127, 32)[:codes.numel()]
    return E4M3[codes.cpu().numpy()] * np.exp2(e.astype(np.float64))


def test_default_rounding_of_8_bit_moments_trains(cuda_device):
    """Gradients of unit variance, default arguments: the corrected root of v is 1. Rounding at random leaves a root's
    mean where it is and adds its variance to v: a step moves v by a thousandth, so the root stands f of a code step
    (2^-3 to 2^-4 of it) away from a code with f about 0.0005 / 0.09, which adds f 0.09^2 to v each step and 5% of v
    over the 1000 steps of the average. To nearest, v would stay where it is."""
    n = 16384
    g = torch.Generator(device=cuda_device).manual_seed(3)
    p = torch.zeros(n, device=cuda_device)
    grad = torch.zeros(n, device=cuda_device)
    opt = mlaq.AdamW([p], lr=1e-3, state_bits=8)
    for t in range(1, 601):
        grad.normal_(generator=g)
        opt.step([grad])
        if t in (50, 200, 600):
            v = np.square(decoded(opt.exp_avg_sq[0], opt.exp_avg_sq_scales[0])).mean() / (1 - 0.999 ** t)
            assert abs(v ** 0.5 - 1) <= 0.06, (t, v ** 0.5)


def test_random_bits_of_consecutive_steps(cuda_device):
    """Equal values between two codes, the same before each step: whether place i is rounded up at one step says nothing
    of place i + lag at the next, within 6 standard errors."""
    n = 1 << 18
    p, grad = torch.zeros(n, device=cuda_device), torch.zeros(n, device=cuda_device)
    opt = mlaq.AdamW([p], lr=0.0, betas=(0.9, 0.95), weight_decay=0.0, state_bits=8, seed=11)
    m, ms = mlaq.mxfp8_quantize_rows(torch.full((n // 32, 32), 0.875, device=cuda_device))
    v, vs = mlaq.mxfp8_quantize_rows(torch.full((n // 32, 32), 1.0, device=cuda_device))
    ups = []
    for _ in range(3):
        for to, t in ((opt.exp_avg, m), (opt.exp_avg_scales, ms), (opt.exp_avg_sq, v), (opt.exp_avg_sq_scales, vs)):
            to[0].copy_(t.reshape(-1))
        opt.step([grad])
        ups.append([t.double() - t.double().mean() for t in (opt.exp_avg[0], opt.exp_avg_sq[0])])
    for a, b in zip(ups, ups[1:]):
        for s, t in zip(a, b):
            assert float(s.var()) > 0
            for lag in (0, 1, 2, 3, 8, 32, 64):
                bound = 6 * float(s.std() * t.std()) / n ** 0.5
                assert abs(float((s[:n - lag] * t[lag:]).mean())) <= bound, lag
                assert abs(float((s[lag:] * t[:n - lag]).mean())) <= bound, -lag


def test_a_captured_step_outlives_other_gradients(cuda_device):
    """A graph of a step replays on its own buffers after eager steps on other gradients."""
    n = 3000
    p = torch.nn.Parameter(torch.ones(n, device=cuda_device))
    opt = mlaq.AdamW([p], lr=0.125, betas=(0.0, 0.0), weight_decay=0.0)  # a step is lr times the gradient's sign
    p.grad = torch.ones_like(p)
    opt.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step()
    p.grad = -torch.ones_like(p)
    opt.step()
    p.grad = None
    junk = [torch.full((1 << 16,), 255, dtype=torch.uint8, device=cuda_device) for _ in range(8)]
    junk += [torch.full((n,), float("nan"), device=cuda_device) for _ in range(8)]
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert ((p.detach().double() - (1 - 0.125 * 3)).abs() <= 100 * 2.0 ** -24).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_an_overflowing_second_moment_stops_its_element(cuda_device, bits):
    """v' is infinite in float32: its root is, the quotient is zero and the parameter stays, as the formula says; the
    others step on. (The 8-bit root itself is kept as the largest float32's, in a block of its own here.)"""
    n = 64
    p = torch.ones(n, device=cuda_device)
    g = torch.ones(n, device=cuda_device)
    g[:32] = torch.tensor([1e30, -1e25], device=cuda_device).repeat(16)
    opt = mlaq.AdamW([p], lr=0.25, betas=(0.9, 0.95), weight_decay=0.0, state_bits=bits)
    opt.step([g])
    assert (p[:32] == 1.0).all()
    assert ((p[32:].double() - 0.75).abs() <= 20 * 2.0 ** -24).all()
    if bits == 8:
        assert 255 not in opt.exp_avg_sq_scales[0].tolist()


@pytest.mark.parametrize("compiled", [True, False])
def test_gradients_of_another_stream(cuda_device, monkeypatch, compiled):
    """Steps on a busy side stream, by its context or by name, with gradients of the main stream that are dropped right
    away: what the main stream allocates and fills then is not what the steps read."""
    mlaq.lib()
    if not compiled:
        monkeypatch.setattr(mlaq, "_calls", None)
    elif mlaq._calls is None:
        pytest.skip("calls.cpp was not built here")
    n = 1 << 20
    p = torch.nn.Parameter(torch.ones(n, device=cuda_device))
    opt = mlaq.AdamW([p], lr=0.125, betas=(0.0, 0.0), weight_decay=0.0)  # a step is lr times the gradient's sign
    side, main = torch.cuda.Stream(cuda_device), torch.cuda.current_stream(cuda_device)
    busy = torch.randn((2048, 2048), device=cuda_device)
    for i in range(4):
        p.grad = torch.ones_like(p)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            for _ in range(8):
                busy = busy @ busy
                busy = busy / busy.norm()
            if i % 2:
                opt.step()
        if i % 2 == 0:
            opt.step(stream=side)
        p.grad = None
        fill = [torch.full((n,), -1.0, device=cuda_device) for _ in range(4)]
        main.wait_stream(side)
        assert ((p.detach().double() - (1 - 0.125 * (i + 1))).abs() <= 40 * (i + 1) * 2.0 ** -24).all()
        del fill
