"""How the axis of each pair may be given to the rotary calls: whatever holds Dr/2 integers means these integers, and
nothing else is taken. Without a GPU: tensors that report themselves as CUDA tensors, calls that are listed."""
import numpy as np
import pytest
import torch

import up_proj_gemm_gb300 as mlaq
from up_proj_gemm_gb300 import _build, rotary

T, H, Dr = 6, 3, 8
AXES = [1, 0, 1, 0]


class Compiled:
    """The compiled calls, which take what they are given."""

    def __init__(self, log):
        self.log = log

    def rope_axes(self, x, cos, sin, pos, axes, Dr, mode):
        self.log.append(axes)
        return x

    def rope_axes_table(self, cos, sin, pos, axes, Dr):
        self.log.append(axes)
        return cos, sin


@pytest.fixture(params=["compiled", "python"])
def given(request, monkeypatch):
    _build.build()
    mlaq.lib()
    log = []
    monkeypatch.setattr(mlaq, "_calls", Compiled(log) if request.param == "compiled" else None)
    monkeypatch.setattr(rotary, "_call", lambda fn, what, *a: log.extend(v for v in a if type(v) is bytes))
    monkeypatch.setattr(rotary, "_stream", lambda device, stream: None)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    return log


def both(axes, Dr=Dr):
    x, cos, pos = torch.zeros(T, H, 12), torch.zeros(32, 8), torch.zeros(2, T, dtype=torch.int32)
    yield lambda: mlaq.rope_axes(x, cos, cos, pos, axes, Dr)
    yield lambda: mlaq.rope_axes_table(cos, cos, pos, axes, Dr)


@pytest.mark.parametrize("axes", [AXES, tuple(AXES), bytes(AXES), bytearray(AXES), np.array(AXES), np.array(AXES, np.int32),
                                  np.array(AXES, np.uint8), torch.tensor(AXES), torch.tensor(AXES, dtype=torch.uint8),
                                  [np.int64(a) for a in AXES]])
def test_taken(given, axes):
    for call in both(axes):
        call()
    assert given == [bytes(AXES)] * 2


@pytest.mark.parametrize("axes", [4, 8, np.int64(4), None, 1.5, "1010", [1.0, 0.0, 1.0, 0.0], np.array(AXES, np.float32),
                                  [256, 0, 0, 0], [-1, 0, 0, 0], AXES[1:], AXES + [0], [], np.array([AXES]), bytes(5)])
def test_refused(given, axes):
    for call in both(axes):
        with pytest.raises((TypeError, ValueError)):
            call()
    assert not given
