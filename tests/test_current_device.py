"""Tensors on another GPU than the current one, and streams of another GPU than the tensors', are refused on the host:
the library launches on the current device, and default streams have the same handle everywhere."""
import pytest
import torch

import up_proj_gemm_gb300 as mlaq


class Stream:
    def __init__(self, handle, device):
        self.cuda_stream, self.device_index = handle, device


@pytest.fixture
def current(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i)


def test_stream_of_a_call(current):
    assert mlaq._stream(torch.device("cuda:1"), None).value == 101
    assert mlaq._stream(torch.device("cuda"), None).value == 101
    assert mlaq._stream(torch.device("cuda:1"), Stream(7, 1)).value == 7
    for device, stream in (("cuda:0", None), ("cuda:2", None), ("cuda:0", Stream(7, 0)), ("cuda:0", Stream(7, 1)),
                           ("cuda:1", Stream(7, 0)), ("cuda", Stream(0, 0))):
        with pytest.raises(ValueError, match="cuda:"):
            mlaq._stream(torch.device(device), stream)


@pytest.mark.gpu
def test_calls_elsewhere(cuda_device, monkeypatch):
    """The Python face on real tensors, while another device counts as current."""
    mlaq.lib()
    monkeypatch.setattr(mlaq, "_calls", None)
    b = lambda *s: torch.ones(s, dtype=torch.bfloat16, device=cuda_device)  # noqa: E731
    x, wgu, wd = b(4, 16), b(48, 16), b(16, 24)
    p = [torch.ones(8, device=cuda_device) for _ in range(4)]
    plan = mlaq.adamw_plan(*[[t] for t in p])
    y, gu, h = mlaq.gated_ffn_fwd(x, wgu, wd, save=True)
    cos, pos = torch.ones((4, 8), device=cuda_device), torch.zeros((1, 4), dtype=torch.int32, device=cuda_device)
    calls = [lambda: mlaq.gated_ffn_fwd(x, wgu, wd), lambda: mlaq.gated_ffn_bwd(y, x, wgu, wd, gu, h),
             lambda: mlaq.rope_axes(b(4, 2, 8), cos, cos, pos, [0] * 4, 8),
             lambda: mlaq.rope_axes_table(cos, cos, pos, [0] * 4, 8), lambda: mlaq.adamw_step(plan, 1, lr=0.1),
             lambda: mlaq.mxfp8_quantize_rows(x)]
    for call in calls:
        call()
    torch.cuda.synchronize()
    before = [t.clone() for t in p]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for call in calls:
        with pytest.raises(ValueError, match="current device"):
            call()
    assert all(torch.equal(a, c) for a, c in zip(p, before))
