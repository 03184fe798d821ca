"""The feed-forward block at the widths of a large layer, 7168 channels, against its formulas in 64 bits with the bounds
of one product each (see test_gpu_ffn.py)."""
import pytest
import torch

import up_proj_gemm_gb300 as mlaq
from test_gpu_ffn import U, act64, bf16, check, check_forward, f64, make, product

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,F", [(1, 2048), (40, 2048), (300, 2056), (1030, 2048)])
def test_wide(cuda_device, T, F):
    x, wgu, wd, dy = make(T, 7168, F, pitch=64, seed=T)
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
