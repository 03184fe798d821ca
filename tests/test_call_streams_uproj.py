"""Memory of the projection's calls on another stream than the current one: the workspaces that the binding allocates and
drops, and the outputs that it hands back."""
import contextlib

import pytest
import torch

import up_proj_gemm_gb300 as mlaq
from test_call_streams import Stream, check, log  # noqa: F401

bf16, u8 = torch.bfloat16, torch.uint8
T, K, H, Dn, Dr = 64, 256, 4, 32, 32
N = H * (Dn + Dr)


@pytest.fixture
def sizes(monkeypatch, log):  # noqa: F811
    """A workspace is asked for, as on a GPU."""
    monkeypatch.setattr(mlaq.lib(), "mla_q_uproj_workspace_size", lambda s, which: 4096)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    return log


def tensors():
    z = lambda *s: torch.zeros(s, dtype=bf16)  # noqa: E731
    return z(T, H, Dn + Dr), z(N, K), z(T, K), torch.zeros(T, Dr), torch.zeros(T, Dr)


def test_dgrad(sizes):
    dq, W, x, cos, sin = tensors()
    check(sizes, [mlaq.bwd_dgrad(dq, W, cos, sin, H, Dn, Dr, stream=Stream(7))], 1)


def test_mxfp8_gradient(sizes):
    dq, W, x, cos, sin = tensors()
    check(sizes, mlaq.bwd_mxfp8(dq, W, x, cos, sin, H, Dn, Dr, stream=Stream(7)), 1)


def test_outputs(sizes):
    dq, W, x, cos, sin = tensors()
    side = Stream(7)

    def once(*kept):
        check(sizes, kept, 0)
        sizes.calls.clear(), sizes.recorded.clear(), sizes.made.clear()

    once(*mlaq.bwd_wgrad(dq, x, cos, sin, H, Dn, Dr, stream=side))
    once(mlaq.fwd(x, W, cos, sin, H, Dn, Dr, out_mode="bf16", stream=side))
    once(*mlaq.fwd(x, W, cos, sin, H, Dn, Dr, out_mode="mxfp8", stream=side))
    once(*mlaq.mxfp8_quantize_rows(x, stream=side))
    once(*mlaq.mxfp8_quantize_rows(x, group=128, stream=side))
    once(*mlaq.mxfp8_quantize_cols(x, stream=side))
    once(*mlaq.mxfp8_quantize_cols(x, group=128, stream=side))
    once(mlaq.mxfp8_swizzle_scales(torch.zeros(T, 8, dtype=u8), stream=side))
    once(mlaq.rope_table_pack(cos, sin, Dr, stream=side))
    once(*mlaq.kv_fwd(x, torch.zeros(H * (Dn + 32), K, dtype=bf16), torch.zeros(T, Dr, dtype=bf16), cos, sin, H, Dn, 32, Dr,
                      stream=side))
