"""Attention takes every size that its documentation names: channels, and query rows of a sequence."""
import ctypes

import pytest
import torch

import up_proj_gemm_gb300 as mlaq
from test_gpu_cache import Case
from test_gpu_cache_attn import attend, check, reference

pytestmark = pytest.mark.gpu


def workspace(Dk, Dv, rows, shared):
    at = 0x40000000  # sizes alone are looked at
    c = mlaq.KvCacheShape(4, 64, 32, 1, Dk, Dv, 0, at, 2 * at, None if shared else 3 * at, None if shared else 4 * at)
    a = mlaq.AttnShape(1, 1, 0, Dk, 4, rows, 1.0, 0)
    return mlaq.lib().mla_cache_attn_workspace_size(ctypes.byref(a), ctypes.byref(c))


@pytest.mark.parametrize("rows", [1, 8, 9, 16, 17, 32, 33, 64, 65, 128, 1000])
def test_every_size_has_a_plan(cuda_device, rows):
    sizes = [(k, v, False) for k in range(16, 257, 16) for v in range(16, 257, 16)]
    sizes += [(k, v, True) for k in range(16, 641, 16) for v in range(16, min(k, 512) + 1, 16)]
    assert not [s for s in sizes if workspace(*s[:2], rows, s[2]) == 0]
    assert workspace(656, 512, rows, True) == workspace(640, 528, rows, True) == workspace(272, 16, rows, False) == 0


@pytest.mark.parametrize("Dk,Dv", [(576, 256), (512, 128), (400, 16), (640, 256)])
@pytest.mark.parametrize("Hq,n", [(33, 1), (64, 1), (128, 1), (11, 9)])
def test_latents_with_few_values(cuda_device, Dk, Dv, Hq, n):
    """Rows whose queries leave no room for two tiles of keys."""
    s = Case(cuda_device, H=1, Dk=Dk, Dv=Dv, page=64, block=32, start=[300, 1], n=[n, 1], shared=True)
    q, scale, out, lse = attend(cuda_device, s, Hq)
    ref = reference(s, q, scale)
    check(lse, ref[1], ref[3], "lse")
    check(out, ref[0], ref[2], "out")
