"""AdamW as a training loop uses it."""
import pytest
import torch

import up_proj_gemm_gb300 as mlaq

pytestmark = pytest.mark.gpu
bf16 = torch.bfloat16


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
