"""The autograd faces of the layer operators without a GPU: what they ask the calls for."""
import pytest
import torch

from up_proj_gemm_gb300 import autograd

bf16 = torch.bfloat16
T, K, F = 4, 8, 16


@pytest.fixture
def ffn(monkeypatch):
    """Calls that list what is asked for and return tensors of the right shapes."""
    log = []

    def fwd(x, wgu, wd, act="silu", save=False):
        log.append(("fwd", save))
        y = torch.ones((T, K), dtype=bf16)
        return (y, torch.ones((T, 2 * F), dtype=bf16), torch.ones((T, F), dtype=bf16)) if save else y

    def bwd(dy, x, wgu, wd, gu, h, act="silu", dx=True, dw_gate_up=True, dw_down=True):
        log.append(("bwd", dy.is_contiguous() and dy.data_ptr() % 16 == 0, dy.clone()))
        return tuple(torch.ones_like(t) if want else None for t, want in ((x, dx), (wgu, dw_gate_up), (wd, dw_down)))

    monkeypatch.setattr(autograd, "gated_ffn_fwd", fwd)
    monkeypatch.setattr(autograd, "gated_ffn_bwd", bwd)
    return log


def tensors(grad=True):
    return [torch.ones(s, dtype=bf16, requires_grad=grad) for s in ((T, K), (2 * F, K), (K, F))]


def test_nothing_is_saved_without_a_gradient(ffn):
    """Evaluation does not write the gate and up products, though the weights would have gradients."""
    x, wgu, wd = tensors()
    with torch.no_grad():
        y = autograd.gated_ffn(x, wgu, wd)
    assert ffn == [("fwd", False)] and not y.requires_grad
    with torch.inference_mode():
        autograd.gated_ffn(x, wgu, wd)
    autograd.gated_ffn(*tensors(grad=False))
    assert ffn == [("fwd", False)] * 3
    assert autograd.gated_ffn(x.detach(), wgu.detach(), wd).requires_grad  # one gradient is enough
    assert ffn[3:] == [("fwd", True)]


def test_a_gradient_off_the_16_byte_grid(ffn):
    """The gradient of one part of a concatenation is a slice: contiguous, but anywhere. It reaches the call aligned."""
    x, wgu, wd = tensors()
    y = autograd.gated_ffn(x, wgu, wd)
    out = torch.cat([torch.zeros(3, dtype=bf16), y.flatten()])
    g = torch.arange(out.numel()).to(bf16)
    out.backward(g)
    what, aligned, dy = ffn[-1]
    assert what == "bwd" and aligned and torch.equal(dy.flatten(), g[3:])


def test_a_query_gradient_off_the_16_byte_grid(monkeypatch):
    """The same for the projection's query."""
    seen = []

    def dgrad(dq, W, *a, **kw):
        seen.append(dq.is_contiguous() and dq.data_ptr() % 16 == 0)
        return torch.ones((3, K), dtype=bf16)

    monkeypatch.setattr(autograd, "fwd", lambda x, W, *a, **kw: torch.ones((3, 2, 4), dtype=bf16))
    monkeypatch.setattr(autograd, "bwd_dgrad", dgrad)
    monkeypatch.setattr(autograd, "bwd_wgrad", lambda dq, *a, **kw: (seen.append(dq.data_ptr() % 16 == 0) or
                                                                     torch.ones((8, K), dtype=bf16), None))
    x, W = torch.ones((3, K), dtype=bf16, requires_grad=True), torch.ones((8, K), dtype=bf16, requires_grad=True)
    q = autograd.q_up_proj(x, W, torch.ones(3, 4), torch.ones(3, 4), 2, 0, 4)
    out = torch.cat([torch.zeros(1, dtype=bf16), q.flatten()])
    out.backward(torch.ones_like(out))
    assert seen == [True, True]


def test_second_derivatives_are_refused(ffn, monkeypatch):
    """The backward is not differentiable itself: a penalty on a gradient raises instead of counting for nothing."""
    monkeypatch.setattr(autograd, "_rope_axes", lambda x, *a, **kw: x * 1.0)
    monkeypatch.setattr(autograd, "fwd", lambda x, W, *a, **kw: torch.ones((3, 2, 4), dtype=bf16))
    monkeypatch.setattr(autograd, "bwd_dgrad", lambda dq, W, *a, **kw: torch.ones((3, K), dtype=bf16))
    monkeypatch.setattr(autograd, "bwd_wgrad", lambda dq, *a, **kw: (torch.ones((8, K), dtype=bf16), None))
    t = torch.ones(3, 4)

    def rope():
        x = torch.ones(3, 2, 4, requires_grad=True)
        return x, autograd.rope_axes(x, t, t, torch.zeros(1, 3, dtype=torch.int32), [0, 0], 4)

    def block():
        x, wgu, wd = tensors()
        return x, autograd.gated_ffn(x, wgu, wd)

    def query():
        x, W = (torch.ones(s, dtype=bf16, requires_grad=True) for s in ((3, K), (8, K)))
        return x, autograd.q_up_proj(x, W, t, t, 2, 0, 4)

    for make in (rope, block, query):
        x, y = make()
        (g,) = torch.autograd.grad((y.float() ** 2).sum(), x, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            (y.float().sum() + (g.float() ** 2).sum()).backward()
