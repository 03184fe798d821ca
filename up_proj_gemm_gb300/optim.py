"""AdamW over many tensors in one launch: argument marshalling for the
``mla_adamw_*`` entry points of ``include/mlaq.h``.

``adamw_plan`` lists the tensors once; ``adamw_step`` enqueues a step.
``AdamW`` keeps parameters, moments (float32 or MXFP8), optional float32
masters and the step count for a training loop.
"""
from __future__ import annotations

import ctypes

import torch

import up_proj_gemm_gb300 as _pkg

from . import _call, _need, _ptr, _SIGS, _stream, lib

__all__ = ["AdamwPlan", "adamw_plan", "adamw_step", "AdamW"]


class _Tensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "grad", "exp_avg", "exp_avg_sq", "exp_avg_scales",
                                               "exp_avg_sq_scales", "master")] + [("n", ctypes.c_int64)]


class _Args(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps", "weight_decay")] + [
        ("step", ctypes.c_int64), ("stochastic", ctypes.c_int32), ("seed", ctypes.c_uint32)]


_vp, _int, _i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
_SIGS.update({
    "mla_adamw_plan_bytes": (ctypes.c_size_t, [ctypes.POINTER(_Tensor), _i64]),
    "mla_adamw_plan_build": (_int, [ctypes.POINTER(_Tensor), _i64, _int, _int, _int, _vp, ctypes.c_size_t]),
    "mla_adamw_step": (_int, [_vp, _vp, ctypes.POINTER(_Args), _vp, _vp]),
})
_FLOATS = {torch.float32: 0, torch.bfloat16: 1}


class AdamwPlan:
    """The tensors of a step (held here: parameters, gradients, moments, scales, masters), their plan on the host and
    its device copy."""

    def __init__(self, tensors, host, device_copy, device):
        self.tensors, self.host, self.device_copy, self.device = tensors, host, device_copy, device
        self.host_ptr, self.device_ptr = ctypes.addressof(host), device_copy.data_ptr()
        self.stream = torch.cuda.current_stream(device)  # the one the copy was made on
        self.copied = self.stream.record_event()
        self.where = (self.host_ptr, self.device_ptr, -1 if device.index is None else device.index, self.stream.cuda_stream)

    def release_gradients(self):
        """Hold the gradients no longer: whoever takes a step keeps them until it has run."""
        self.tensors[1] = None

    def ready_on(self, stream):
        """Let `stream` use the device copy: after the copying stream, and held until it is done. (A capture starts
        after the device is idle, so a stream under capture has nothing to wait for.)"""
        if stream.cuda_stream != self.stream.cuda_stream and not torch.cuda.is_current_stream_capturing():
            stream.wait_event(self.copied)
            self.device_copy.record_stream(stream)


def adamw_plan(params, grads, exp_avg, exp_avg_sq, masters=None, exp_avg_scales=None, exp_avg_sq_scales=None):
    """A plan for ``adamw_step``: lists of contiguous CUDA tensors on one device.

    params and grads are float32 or bf16 (one type each); exp_avg and
    exp_avg_sq float32, or uint8 E4M3 codes of m and sqrt(v) with uint8 E8M0
    scales of ceil(n/32) elements (zeros are a fresh state); masters optional
    float32 copies of the parameters. Build another plan when a buffer moves."""
    params = list(params)
    if not params:
        raise ValueError("params is empty")
    n = len(params)
    cols = {"grads": list(grads), "exp_avg": list(exp_avg), "exp_avg_sq": list(exp_avg_sq)}
    bits = 8 if cols["exp_avg"] and getattr(cols["exp_avg"][0], "dtype", None) == torch.uint8 else 32
    if (exp_avg_scales is None) != (bits == 32) or (exp_avg_sq_scales is None) != (bits == 32):
        raise ValueError("scales go with uint8 moments, and only with them")
    for name, v in (("exp_avg_scales", exp_avg_scales), ("exp_avg_sq_scales", exp_avg_sq_scales),
                    ("masters", masters)):
        cols[name] = [None] * n if v is None else list(v)
    for name, v in cols.items():
        if len(v) != n:
            raise ValueError(f"{name} must list {n} tensors, got {len(v)}")
    for name, first in (("params", params[0]), ("grads", cols["grads"][0])):
        if not isinstance(first, torch.Tensor) or first.dtype not in _FLOATS:
            raise TypeError(f"{name} must be float32 or bfloat16 tensors")
    dev, pt, gt = params[0].device, params[0].dtype, cols["grads"][0].dtype
    st = torch.uint8 if bits == 8 else torch.float32
    rows = (_Tensor * n)()
    for i, p in enumerate(params):
        _need(p, f"params[{i}]", pt, dev)
        k = p.numel()
        for name, dtype, size in (("grads", gt, k), ("exp_avg", st, k), ("exp_avg_sq", st, k),
                                  ("exp_avg_scales", torch.uint8, -(-k // 32)),
                                  ("exp_avg_sq_scales", torch.uint8, -(-k // 32)), ("masters", torch.float32, k)):
            if cols[name][i] is not None or name not in ("exp_avg_scales", "exp_avg_sq_scales", "masters"):
                _need(cols[name][i], f"{name}[{i}]", dtype, dev, numel=size)
        at = [t.data_ptr() if t is not None and t.numel() else None for t in
              [p] + [cols[c][i] for c in ("grads", "exp_avg", "exp_avg_sq", "exp_avg_scales", "exp_avg_sq_scales",
                                          "masters")]]
        rows[i] = _Tensor(*at, k)
    size = int(lib().mla_adamw_plan_bytes(rows, n))
    host = ctypes.create_string_buffer(max(size, 1))
    _call(lib().mla_adamw_plan_build, "mla_adamw_plan_build", rows, n, _FLOATS[pt], _FLOATS[gt], bits,
          ctypes.addressof(host), size)
    copy = torch.frombuffer(host, dtype=torch.uint8).to(dev)
    return AdamwPlan([params] + list(cols.values()), host, copy, dev)


def adamw_step(plan, step, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, grad_scale=None, seed=None,
               stream=None):
    """Enqueue one AdamW step (t = ``step``, counted from 1) over the plan's
    tensors, in place.

    grad_scale: a float32 CUDA tensor of one element that multiplies every
    gradient. seed: an int, another one each step, rounds the 8-bit moments
    (and bf16 parameters without masters) up or down at random; None rounds
    to nearest, which holds 8-bit moments still where a step moves them by less
    than half a code.

    step, lr, betas, eps, weight_decay and seed are constants of the launch: a
    CUDA graph replays the step with those of its capture, and needs the plan
    as long as it lives."""
    if not isinstance(plan, AdamwPlan):
        raise TypeError("plan must come from adamw_plan")
    c = _pkg._calls
    if c is not None and stream is None and c.adamw_step(*plan.where, step, lr, betas[0], betas[1], eps, weight_decay,
                                                         grad_scale, seed):
        return
    if grad_scale is not None:
        _need(grad_scale, "grad_scale", torch.float32, plan.device, numel=1)
    if stream is None:
        stream = torch.cuda.current_stream(plan.device)
    plan.ready_on(stream)
    a = _Args(lr, betas[0], betas[1], eps, weight_decay, step, 0 if seed is None else 1,
              0 if seed is None else seed & 0xFFFFFFFF)
    _call(lib().mla_adamw_step, "mla_adamw_step", plan.host_ptr, plan.device_ptr, ctypes.byref(a), _ptr(grad_scale),
          _stream(plan.device, stream))


def _places(*lists):
    """Address, size, type and layout of every tensor, to be compared with those of another step, in compiled code
    where it is built (290 tensors: 10 us of a step's host time, 300 without)."""
    lib()
    places = None if _pkg._calls is None else _pkg._calls.adamw_places(*lists)
    if places is None:
        places = [None if v is None else [(t.data_ptr(), t.numel(), t.dtype, t.is_contiguous()) for t in v]
                  for v in lists]
    return places


def _keep(grads, stream):
    """Let nobody have the gradients' memory, once they are dropped, before the step on `stream` (None: the current one)
    has read it: they may be another stream's (290 gradients: 30 us of host time)."""
    if stream is not None and stream.cuda_stream != torch.cuda.current_stream(grads[0].device).cuda_stream:
        for g in grads:
            g.record_stream(stream)
    elif _pkg._calls is None or not _pkg._calls.adamw_keep(grads):
        for g in grads:
            if g.device.type == "cuda":
                g.record_stream(torch.cuda.current_stream(g.device))


def _step_seed(seed, step):
    """The kernel's seed of a step. It adds the seed to a multiple of the element's place, so seeds a small multiple of
    that factor apart give the same bits a few places on: seed and step are mixed beyond sums of multiples (each
    operation is a bijection of 32 bits: no two steps share a seed)."""
    x = (seed + step * 0x3C6EF373) & 0xFFFFFFFF
    x = ((x ^ (x >> 16)) * 0x6A09E667) & 0xFFFFFFFF
    x = ((x ^ (x >> 13)) * 0xBB67AE85) & 0xFFFFFFFF
    return x ^ (x >> 16)


_BY_STATE = object()  # the default seed: at random where the moments need it


class AdamW:
    """AdamW for a list of parameters, one launch per step.

    ``state_bits`` 32 keeps float32 moments, 8 MXFP8 ones. ``masters`` keeps
    float32 copies of bf16 parameters. ``seed`` (an int) rounds at random as
    in ``adamw_step``, from a seed that changes with the step; None rounds to
    nearest. Left out, it is 0 with MXFP8 moments and None with float32 ones:
    a step moves a moment by less than half a step of its 8-bit code, and
    rounded to nearest it would stay where it is (gradients of unit variance,
    beta2 = 0.999: the root of v 0.86 of its value after 50 steps, 0.54 after
    300). ``step()``
    takes the gradients from ``grads`` or the parameters' ``.grad``; the plan
    is rebuilt when a gradient's buffer is another one than at the last step."""

    def __init__(self, params, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, state_bits=32, masters=False,
                 seed=_BY_STATE):
        if state_bits not in (32, 8):
            raise ValueError(f"state_bits must be 32 or 8, got {state_bits}")
        self.params = [p for p in params]
        self.lr, self.betas, self.eps, self.weight_decay = lr, betas, eps, weight_decay
        self.seed = (0 if state_bits == 8 else None) if seed is _BY_STATE else seed
        self.steps = 0
        dtype = torch.uint8 if state_bits == 8 else torch.float32

        def zeros():
            return [torch.zeros(p.shape, dtype=dtype, device=p.device) for p in self.params]

        def scales():
            return [torch.zeros((-(-p.numel() // 32),), dtype=torch.uint8, device=p.device) for p in self.params]

        self.exp_avg, self.exp_avg_sq = zeros(), zeros()
        self.exp_avg_scales = scales() if state_bits == 8 else None
        self.exp_avg_sq_scales = scales() if state_bits == 8 else None
        self.masters = [p.detach().float().clone() for p in self.params] if masters else None
        self._plan, self._places = None, None
        self._captured = []  # what the steps inside captured graphs read

    def step(self, grads=None, grad_scale=None, stream=None):
        """One step; every parameter needs a gradient."""
        grads = [p.grad for p in self.params] if grads is None else list(grads)
        if any(g is None for g in grads):
            raise ValueError("a parameter has no gradient")
        places = _places(self.params, grads, self.exp_avg, self.exp_avg_sq, self.exp_avg_scales,
                         self.exp_avg_sq_scales, self.masters)
        if self._plan is None or places != self._places:
            self._plan = None  # also when the new one is refused
            self._plan = adamw_plan([p.detach() for p in self.params], grads, self.exp_avg, self.exp_avg_sq,
                                    masters=self.masters, exp_avg_scales=self.exp_avg_scales,
                                    exp_avg_sq_scales=self.exp_avg_sq_scales)
            self._plan.release_gradients()
            self._places = places
        step = self.steps + 1
        seed = None if self.seed is None else _step_seed(self.seed, step)
        adamw_step(self._plan, step, self.lr, self.betas, self.eps, self.weight_decay, grad_scale, seed, stream)
        self.steps = step
        if torch.cuda.is_initialized() and torch.cuda.is_current_stream_capturing():
            self._captured.append((self._plan, grads))
        else:
            _keep(grads, stream)
        for p in self.params:  # autograd sees that they were written
            torch.autograd.graph.increment_version(p)
