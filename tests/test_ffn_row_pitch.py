"""The feed-forward block's x with rows that overlap, first of all one row for all tokens: refused, not read as a dense
matrix. Without a GPU, by tensors that report themselves as CUDA tensors; the compiled call's check on a real one."""
import pytest
import torch

import up_proj_gemm_gb300 as mlaq
from up_proj_gemm_gb300 import _build, ffn

bf16 = torch.bfloat16
T, K, F = 6, 16, 24


def overlapping(device):
    row = torch.zeros(1, K, dtype=bf16, device=device)
    flat = torch.zeros(T * K, dtype=bf16, device=device)
    return [row.expand(T, K), flat.as_strided((T, K), (8, 1)), flat.as_strided((T, K), (K - 8, 1))]


def others(device):
    wgu, wd, dy, gu, h = (torch.zeros(s, dtype=bf16, device=device) for s in ((2 * F, K), (K, F), (T, K), (T, 2 * F), (T, F)))
    return wgu, wd, dy, gu, h


def refuse(device):
    wgu, wd, dy, gu, h = others(device)
    for x in overlapping(device):
        with pytest.raises(ValueError, match="overlap"):
            mlaq.gated_ffn_fwd(x, wgu, wd)
        with pytest.raises(ValueError, match="overlap"):
            mlaq.gated_ffn_bwd(dy, x, wgu, wd, gu, h)


def test_refused_by_the_binding(monkeypatch):
    _build.build()
    mlaq.lib()
    pitches = []
    monkeypatch.setattr(mlaq, "_calls", None)
    monkeypatch.setattr(ffn, "_call", lambda fn, what, shape, *a: pitches.append(shape._obj.ld_x))
    monkeypatch.setattr(ffn, "_stream", lambda device, stream: None)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    refuse("cpu")
    assert not pitches
    wgu, wd, dy, gu, h = others("cpu")
    for x, pitch in ((torch.zeros(T, K, dtype=bf16), K), (torch.zeros(T, K + 8, dtype=bf16)[:, :K], K + 8)):
        mlaq.gated_ffn_fwd(x, wgu, wd)
        mlaq.gated_ffn_bwd(dy, x, wgu, wd, gu, h)
        assert pitches[-2:] == [pitch, pitch]
    # a single row has no pitch
    mlaq.gated_ffn_fwd(torch.zeros(1, K, dtype=bf16).as_strided((1, K), (0, 1)), wgu, wd)
    assert pitches[-1] == K


@pytest.mark.gpu
@pytest.mark.parametrize("compiled", [True, False])
def test_refused_by_the_calls(cuda_device, monkeypatch, compiled):
    mlaq.lib()
    if not compiled:
        monkeypatch.setattr(mlaq, "_calls", None)
    elif mlaq._calls is None:
        pytest.skip("calls.cpp was not built here")
    refuse(cuda_device)
