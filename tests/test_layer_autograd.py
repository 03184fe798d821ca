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
