"""A C entry point that runs out of host memory returns a status; no exception leaves it."""
import os
import subprocess
import sys

import up_proj_gemm_gb300 as mlaq
from up_proj_gemm_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import ctypes, resource, sys
import numpy as np
from up_proj_gemm_gb300 import lib
from up_proj_gemm_gb300.optim import _Tensor
L, count = lib(), 1 << 20
rows = (_Tensor * count)()
flat = np.frombuffer(rows, dtype=np.uint64).reshape(count, 8)
flat[:, :4] = (1 << 40) + np.arange(4 * count, dtype=np.uint64).reshape(count, 4) * 64
flat[:, 7] = 4
plan = ctypes.create_string_buffer(L.mla_adamw_plan_bytes(rows, count))
build = lambda: L.mla_adamw_plan_build(rows, count, 0, 0, 32, ctypes.addressof(plan), len(plan))
print(build(), flush=True)
used = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (used + (16 << 20), resource.RLIM_INFINITY))
print(build(), flush=True)
"""


def test_a_plan_of_very_many_tensors():
    """A million tensors, 176 MB of spans to compare, with 16 MB left."""
    _build.build()
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, MALLOC_TRIM_THRESHOLD_="0"))
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split() == [str(mlaq.STATUS["MLA_OK"]), str(mlaq.STATUS["MLA_ERR_MEMORY"])]


def test_its_name():
    assert mlaq.status_string(mlaq.STATUS["MLA_ERR_MEMORY"]) == "MLA_ERR_MEMORY"
