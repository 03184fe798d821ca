"""The example that runs the layer operators together: it trains, with float32 and with MXFP8 moments, and a step's
gradients agree with the block written in plain torch operations."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("video_block", os.path.join(ROOT, "examples", "video_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("bits", [32, 8])
def test_training_lowers_the_loss(cuda_device, example, bits):
    losses = example.train(steps=30, state_bits=bits)
    assert all(map(torch.isfinite, map(torch.tensor, losses)))
    assert losses[-1] < 0.5 * losses[0]


def plain(block, x, e):
    """The block in float64, every rotation written out."""
    w = {n: getattr(block, n).detach().double().requires_grad_() for n in
         ("w_q", "w_k", "w_v", "w_rope", "w_out", "w_gate_up", "w_down")}
    T = x.shape[0]
    rows = block.pos.long()[torch.tensor(list(block.axes) * 2, device=x.device)].t()
    cos, sin = (t.double().gather(0, rows)[:, None] for t in (block.cos, block.sin))

    def turn(v):
        a, b = v.chunk(2, -1)
        h = e.DR // 2
        return torch.cat([a * cos[..., :h] - b * sin[..., :h], b * cos[..., h:] + a * sin[..., h:]], -1)

    x = x.double()
    q = (x @ w["w_q"].t()).view(T, e.H, e.DN + e.DR)
    q = torch.cat([q[..., :e.DN], turn(q[..., e.DN:])], -1)
    k_rope = turn((x @ w["w_rope"].t()).view(T, 1, e.DR)).expand(-1, e.H, -1)
    k = torch.cat([(x @ w["w_k"].t()).view(T, e.H, e.DN), k_rope], -1)
    v = (x @ w["w_v"].t()).view(T, e.H, e.DV)
    p = (torch.einsum("qhd,khd->hqk", q, k) * (e.DN + e.DR) ** -0.5).softmax(-1)
    x = x + torch.einsum("hqk,khd->qhd", p, v).reshape(T, -1) @ w["w_out"].t()
    g, u = (x @ w["w_gate_up"].t()).chunk(2, -1)
    return x + (torch.nn.functional.silu(g) * u) @ w["w_down"].t(), w


def test_gradients_of_the_block(cuda_device, example):
    block = example.Block(cuda_device)
    g = torch.Generator().manual_seed(5)
    x = torch.randn((256, example.K), generator=g).to(torch.bfloat16).to(cuda_device)
    dy = torch.randn((256, example.K), generator=g).to(cuda_device)
    y = block(x)
    y.backward(dy.to(torch.bfloat16))
    ref, w = plain(block, x, example)
    ref.backward(dy.to(torch.bfloat16).double())
    # a chain of about ten bf16 roundings of 2^-9 rms each, on both sides of every product: 2^-5 of the norm
    y, ref = y.detach().double(), ref.detach()
    assert float((y - ref).norm() / ref.norm()) <= 2.0 ** -5
    for n, t in w.items():
        got = getattr(block, n).grad.double()
        assert float((got - t.grad).norm() / t.grad.norm()) <= 2.0 ** -5, n
