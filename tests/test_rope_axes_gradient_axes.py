"""The gradient of a rotation turns by the axes of its forward, whatever becomes of the list that named them."""
import torch

from up_proj_gemm_gb300 import autograd


def test_a_list_that_changes(monkeypatch):
    seen = []

    def rope(x, cos, sin, pos, axes, Dr, **kw):
        seen.append((bytes(axes), kw))
        return x.clone()

    monkeypatch.setattr(autograd, "_rope_axes", rope)
    x, axes = torch.ones(3, 2, 8, requires_grad=True), [0, 1, 1, 0]
    y = autograd.rope_axes(x, torch.ones(4, 8), torch.ones(4, 8), torch.zeros(2, 3, dtype=torch.int32), axes, 8)
    axes[0] = 1
    y.sum().backward()
    assert seen == [(bytes([0, 1, 1, 0]), {}), (bytes([0, 1, 1, 0]), dict(inverse=True, sum_heads=False))]
