"""pytest configuration: the ``gpu`` marker and shared fixtures.

Tests marked ``gpu`` need a CUDA device and the in-tree ``libmlaq.so``; the
rest run on the CPU (oracle pins, host-side argument checks, symbol exports).
"""
import ctypes
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built libmlaq.so")


@pytest.fixture(scope="session")
def cuda_device():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


@pytest.fixture(autouse=True)
def fresh_small_blocks(request):
    """Blocks that the C library kept from earlier tests and imports stay away from the optimizer loop's tests, which tell
    a dropped buffer from a new one by its address: with a full list of kept blocks of one size, a new buffer could
    get the dropped one's place."""
    if request.module.__name__ != "test_adamw_loop":
        yield
        return
    libc = ctypes.CDLL(None)
    libc.malloc.restype, libc.malloc.argtypes, libc.free.argtypes = ctypes.c_void_p, [ctypes.c_size_t], [ctypes.c_void_p]
    held = [libc.malloc(size) for size in range(24, 1025, 16) for _ in range(64)]
    yield
    for block in held:
        libc.free(block)
