"""The optimizer's bookkeeping between steps without a GPU: tensors that report themselves as CUDA tensors, steps that
are listed instead of launched, plans read back from their host copy."""
import contextlib
import ctypes
import struct
import weakref

import pytest
import torch

import up_proj_gemm_gb300 as mlaq
from up_proj_gemm_gb300 import _build, optim

bf16, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
HEADER, ENTRY = 48, 72  # bytes of a plan's header and of a tensor's entry: seven addresses, the size, the first place


class FakeStream:
    cuda_stream = 0

    def record_event(self):
        return None

    def wait_event(self, event):
        return None


@pytest.fixture
def steps(monkeypatch):
    """The plans' entries of every step: (param, grad, exp_avg, exp_avg_sq, their scales, master, n)."""
    _build.build()
    mlaq.lib()
    log, real = [], optim._call

    def call(fn, what, *args):
        if what != "mla_adamw_step":
            return real(fn, what, *args)
        host = args[0]
        count = struct.unpack("q", ctypes.string_at(host + 8, 8))[0]
        log.append([struct.unpack("7Qq", ctypes.string_at(host + HEADER + i * ENTRY, 64)) for i in range(count)])

    monkeypatch.setattr(mlaq, "_calls", None)
    monkeypatch.setattr(optim, "_call", call)
    monkeypatch.setattr(optim, "_stream", lambda device, stream: None)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: FakeStream())
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    return log


def made(n=2, bits=32, masters=False, dtype=f32):
    params = [torch.nn.Parameter(torch.ones(40 + i, dtype=dtype)) for i in range(n)]
    for p in params:
        p.grad = torch.ones_like(p)
    return params, mlaq.AdamW(params, 1e-3, state_bits=bits, masters=masters)


def addresses(opt, grads):
    lists = (opt.params, grads, opt.exp_avg, opt.exp_avg_sq, opt.exp_avg_scales, opt.exp_avg_sq_scales, opt.masters)
    return [tuple(0 if v is None else v[i].data_ptr() for v in lists) + (opt.params[i].numel(),)
            for i in range(len(opt.params))]


@pytest.mark.parametrize("bits,masters", [(32, False), (32, True), (8, False)])
def test_a_step_uses_the_buffers_of_its_time(steps, bits, masters):
    """Whatever moved since the last step: a parameter, a gradient, a moment, a scale, a master."""
    params, opt = made(bits=bits, masters=masters)
    grads = [p.grad for p in params]
    moves = [lambda: setattr(params[1], "data", params[1].data.clone()),
             lambda: grads.__setitem__(0, grads[0].clone())]
    for v in (opt.exp_avg, opt.exp_avg_sq, opt.exp_avg_scales, opt.exp_avg_sq_scales, opt.masters):
        if v is not None:
            moves.append(lambda v=v: v.__setitem__(1, v[1].clone()))
    opt.step(grads)
    for i, move in enumerate(moves):
        move()
        opt.step(grads)
        assert steps[-1] == addresses(opt, grads), i
    assert len(steps) == 1 + len(moves)


def test_buffers_that_change_their_type_or_layout_are_checked_again(steps):
    """The same address as another type, size or order is no plan's any more."""
    params, opt = made(n=1)
    buffer = torch.ones(80)
    opt.step([buffer[:40]])
    with pytest.raises(ValueError):  # 40 elements, two apart
        opt.step([buffer[::2]])
    opt.step([buffer.view(bf16)[:40]])  # the same start, now bf16
    assert struct.unpack("4i", ctypes.string_at(opt._plan.host_ptr + 32, 16))[1] == 1
    with pytest.raises(ValueError):
        opt.step([buffer[:39]])
    opt.step([buffer[:40]])
    assert len(steps) == 3


def test_gradients_are_not_held(steps):
    """A dropped gradient is gone, and one at the same place needs no new plan."""
    params, opt = made()
    opt.step()
    plan, refs = opt._plan, [weakref.ref(p.grad) for p in params]
    for p in params:
        p.grad = None
    assert all(r() is None for r in refs)
    buffers = [torch.ones(p.numel()) for p in params]
    opt.step([b.view(-1) for b in buffers])
    assert opt._plan is not plan
    plan = opt._plan
    opt.step([b.view(-1) for b in buffers])  # other tensors, the same buffers
    assert opt._plan is plan and steps[-1] == addresses(opt, buffers)


def test_a_side_stream_keeps_what_it_reads(steps, monkeypatch):
    """Gradients that another stream still reads are recorded on it; on the current one nothing is."""
    class Side(FakeStream):
        cuda_stream = 7

    kept = []
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: kept.append((t.data_ptr(), s.cuda_stream)))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    params, opt = made()
    opt.step()
    opt.step(stream=FakeStream())
    assert not kept
    opt.step(stream=Side())
    assert {(p.grad.data_ptr(), 7) for p in params} <= set(kept)


def test_compiled_comparison():
    """The compiled list of places differs when the Python one does, and only then."""
    _build.build()
    mlaq.lib()
    if mlaq._calls is None:
        pytest.skip("calls.cpp was not built here")
    f = mlaq._calls.adamw_places
    a, b, c = torch.zeros(40), torch.zeros(40), torch.zeros(6, 6)
    assert f([a, b], None, [c]) == f([a.view(-1), b.detach()], None, [c[:]])
    same = [([a], [b]), ([a, b], []), ([a], None, [b]), ([b], [a]), ([a], [b[:39]]), ([a], [b.view(torch.int32)]),
            ([a], [b.view(bf16)[:40]]), ([c], [b]), ([c.t()], [b]), ([a], [b], None)]
    assert len({f(*v) for v in same}) == len(same)
    assert f([a, None]) is None and f((a,)) is None and f([a.to_sparse()]) is None
    assert f([torch.zeros(0)], []) != f([], [torch.zeros(0)])


def test_default_seed():
    """8-bit moments are rounded at random unless it is asked for otherwise."""
    p = [torch.ones(4)]
    assert mlaq.AdamW(p, 1e-3, state_bits=8).seed is not None
    assert mlaq.AdamW(p, 1e-3, state_bits=8, seed=None).seed is None
    assert mlaq.AdamW(p, 1e-3, state_bits=8, seed=5).seed == 5
    assert mlaq.AdamW(p, 1e-3).seed is None


@pytest.mark.parametrize("seed", [0, 1, 11, 2**31, 2**32 - 1, 2**40 + 7, -3])
def test_seeds_of_neighbouring_steps(steps, monkeypatch, seed):
    """The kernel mixes place * 0x9E3779B1 + seed in 32 bits: two seeds a multiple k of that factor apart give place i the
    bits of place i + k. Between a step and any of the four after it that shift is above 64, and no seed repeats. (Of
    8000 pairs with random shifts one in 4000 draws would hold one below it.)"""
    seeds = []
    monkeypatch.setattr(optim, "adamw_step", lambda plan, step, *a: seeds.append(a[5]))
    opt = mlaq.AdamW([torch.ones(4)], 1e-3, state_bits=8, seed=seed)
    for _ in range(2000):
        opt.step([torch.ones(4)])
    assert len(set(seeds)) == 2000 and all(0 <= s < 2**32 for s in seeds)
    inverse = pow(0x9E3779B1, -1, 2**32)
    for apart in (1, 2, 3, 4):
        shifts = [(b - a) * inverse % 2**32 for a, b in zip(seeds, seeds[apart:])]
        assert min(min(s, 2**32 - s) for s in shifts) > 64


def test_a_refused_step_does_not_count(steps):
    """The bias correction goes by the steps that were taken."""
    params, opt = made()
    opt.step()
    with pytest.raises(ValueError):
        opt.step(grad_scale=torch.zeros(2))
    with pytest.raises(ValueError):
        opt.step([p.grad[1:] for p in params])
    assert opt.steps == 1 and len(steps) == 1
    opt.step()
    assert opt.steps == 2


def test_a_captured_step_keeps_its_plan(steps, monkeypatch):
    """What a graph's replays read stays when later steps use other buffers."""
    params, opt = made()
    opt.step()
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    opt.step()
    refs = [weakref.ref(opt._plan.device_copy)] + [weakref.ref(p.grad) for p in params]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    for _ in range(3):
        for p in params:
            p.grad = p.grad.clone()
        opt.step()
        refs.append(weakref.ref(opt._plan.device_copy))
    assert [r() is not None for r in refs] == [True] * 3 + [False] * 2 + [True]
