"""A wait of a kernel that gives up is told to the caller: a source whose kernels wait on barriers or flags writes
MLA_ERR_TIMEOUT where one ran out. (A kernel without a status to write waits for its own copies by groups, which need no
limit.)"""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "up_proj_gemm_gb300", "csrc")
WAIT = re.compile(r"\b(mbar_wait|mbar_try_wait|mbar_test|wait_flag_gpu)\w*\(")


def code(path):
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path, encoding="utf-8").read(), flags=re.S)


def waiting():
    return [f for f in sorted(glob.glob(os.path.join(CSRC, "*.cu"))) if WAIT.search(code(f))]


def test_there_are_some():
    assert {os.path.basename(f) for f in waiting()} >= {"attn.cu", "bwd.cu", "ffn.cu", "fwd.cu", "selftest.cu"}


@pytest.mark.parametrize("path", waiting(), ids=os.path.basename)
def test_a_wait_that_ran_out_is_reported(path):
    assert re.search(r"record_status\([^;]*MLA_ERR_TIMEOUT|=\s*MLA_ERR_TIMEOUT|MLA_ERR_TIMEOUT\s*[:;)]", code(path))
