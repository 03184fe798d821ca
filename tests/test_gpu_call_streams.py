"""Calls on a stream that is not the current one, with memory that the library allocates: what the current stream
allocates and fills right behind them changes nothing."""
import pytest
import torch

import up_proj_gemm_gb300 as mlaq

pytestmark = pytest.mark.gpu
bf16 = torch.bfloat16


def test_feed_forward_scratch(cuda_device):
    T, K, F = 300, 512, 1024
    g = torch.Generator().manual_seed(1)
    x, wgu, wd, dy = (torch.randn(s, generator=g).mul(s[-1] ** -0.5).to(bf16).to(cuda_device)
                      for s in ((T, K), (2 * F, K), (K, F), (T, K)))
    y, gu, h = mlaq.gated_ffn_fwd(x, wgu, wd, save=True)
    grads = mlaq.gated_ffn_bwd(dy, x, wgu, wd, gu, h)
    side = torch.cuda.Stream(cuda_device)
    busy = torch.randn((2048, 2048), device=cuda_device)
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(side):
            for _ in range(8):
                busy = busy @ busy
                busy = busy / busy.norm()
        got = mlaq.gated_ffn_fwd(x, wgu, wd, stream=side)
        back = mlaq.gated_ffn_bwd(dy, x, wgu, wd, gu, h, stream=side)
        # blocks of the scratch's sizes, filled on the current stream while the calls wait on the other
        fill = [torch.full(s, float("nan"), dtype=bf16, device=cuda_device) for s in ((T, F), (T, 2 * F)) for _ in range(3)]
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, y) and all(torch.equal(a, b) for a, b in zip(back, grads))
        del fill
