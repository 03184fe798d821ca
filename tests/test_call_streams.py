"""Memory of calls on another stream than the current one, without a GPU: streams that only carry a name, allocations
and launches that are listed."""
import contextlib
import ctypes

import pytest
import torch

import up_proj_gemm_gb300 as mlaq
from up_proj_gemm_gb300 import _build, ffn, rotary

bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Log:
    def __init__(self):
        self.current = Stream(0)
        self.made = {}      # address: the stream that was current when it was allocated
        self.recorded = {}  # address: the stream that it was recorded on
        self.calls = []     # (entry point, addresses among its arguments)


@pytest.fixture
def log(monkeypatch):
    _build.build()
    mlaq.lib()
    log, empty, real = Log(), torch.empty, mlaq._call

    def make(*a, **kw):
        t = empty(*a, **kw)
        log.made[t.data_ptr()] = log.current.cuda_stream
        return t

    @contextlib.contextmanager
    def on(stream):
        before, log.current = log.current, stream
        yield
        log.current = before

    def call(fn, what, *args):
        log.calls.append((what, [v if isinstance(v, int) else v.value for v in args
                                 if isinstance(v, (int, ctypes.c_void_p))]))

    monkeypatch.setattr(mlaq, "_calls", None)
    for m in (mlaq, ffn, rotary):
        monkeypatch.setattr(m, "_call", call)
        monkeypatch.setattr(m, "_stream", lambda device, stream: None)
    monkeypatch.setattr(torch, "empty", make)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: log.recorded.__setitem__(t.data_ptr(), s.cuda_stream))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: log.current)
    monkeypatch.setattr(torch.cuda, "stream", on)
    return log


def check(log, kept, dropped):
    """One call was made on stream 7: what it wrote came from that stream; what the caller keeps may be read on stream 0."""
    (what, addresses), = log.calls
    own = [a for a in addresses if a in log.made]
    assert len(own) == len(kept) + dropped, what
    assert all(log.made[a] == 7 for a in own)
    assert {t.data_ptr(): 0 for t in kept} == log.recorded
    assert log.current.cuda_stream == 0


def feed_forward():
    T, K, F = 6, 16, 24
    return [torch.zeros(s, dtype=bf16) for s in ((T, K), (2 * F, K), (K, F), (T, K), (T, 2 * F), (T, F))]


@pytest.mark.parametrize("save", [False, True])
def test_feed_forward(log, save):
    x, wgu, wd, _, _, _ = feed_forward()
    r = mlaq.gated_ffn_fwd(x, wgu, wd, save=save, stream=Stream(7))
    check(log, r if save else [r], 0 if save else 1)  # without saving, h is scratch


def test_feed_forward_gradient(log):
    x, wgu, wd, dy, gu, h = feed_forward()
    check(log, mlaq.gated_ffn_bwd(dy, x, wgu, wd, gu, h, stream=Stream(7)), 1)  # dgate_up is scratch


def test_rotary(log):
    x, cos = torch.zeros(5, 3, 12), torch.zeros(32, 8)
    pos, axes = torch.zeros(2, 5, dtype=i32), [0, 0, 1, 1]
    check(log, [mlaq.rope_axes(x, cos, cos, pos, axes, 8, stream=Stream(7))], 0)
    log.calls.clear(), log.recorded.clear()
    check(log, mlaq.rope_axes_table(cos, cos, pos, axes, 8, stream=Stream(7)), 0)


def test_the_current_stream_by_name(log):
    """stream= the current one: as without it."""
    x, wgu, wd, _, _, _ = feed_forward()
    mlaq.gated_ffn_fwd(x, wgu, wd, stream=Stream(0))
    assert all(log.made[a] == 0 for a in log.calls[0][1] if a in log.made) and not log.recorded
