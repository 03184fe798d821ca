"""Kernels that are launched under the grid before them (csrc/launch.cuh) run while that grid still writes. The
non-coherent load path is for memory that nobody writes while the kernel runs, so their sources must not use it."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "up_proj_gemm_gb300", "csrc")
NON_COHERENT = re.compile(r"__ldg\b|\.nc\b|__restrict__")


def overlapped():
    return [f for f in sorted(glob.glob(os.path.join(CSRC, "*.cu")))
            if '#include "launch.cuh"' in open(f, encoding="utf-8").read()]


def code(path):
    """A source without its comments."""
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path, encoding="utf-8").read(), flags=re.S)


def test_there_are_some():
    assert {os.path.basename(f) for f in overlapped()} >= {"adamw.cu", "ffn.cu", "rope_axes.cu"}


@pytest.mark.parametrize("path", overlapped() + [os.path.join(CSRC, h) for h in ("launch.cuh", "mx.cuh", "ptx.cuh")],
                         ids=os.path.basename)
def test_no_non_coherent_loads(path):
    assert not NON_COHERENT.findall(code(path))
