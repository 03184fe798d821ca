"""Strides whose spans leave 64 bits are refused by the C entry points, before any span is compared or launched. Without a
GPU, with fake device addresses."""
import ctypes

import pytest

import up_proj_gemm_gb300 as mlaq
from up_proj_gemm_gb300 import _build

INV, ALIAS = mlaq.STATUS["MLA_ERR_INVALID_ARG"], mlaq.STATUS["MLA_ERR_ALIAS"]
FAKE = 0x40000000


def p(i):
    return ctypes.c_void_p(FAKE * (i + 1))


@pytest.fixture(scope="module")
def L():
    _build.build()
    return mlaq.lib()


def rope(L, T, H, strides, out=8, x=9):
    """x and out lie above the other buffers."""
    s = mlaq.RopeAxesShape(T, H, 0, 8, 1, 64, 8, *strides, 0)
    return L.mla_rope_axes(ctypes.byref(s), 1, 0, p(x), p(1), p(2), p(3), bytes(4), p(out), None, None)


@pytest.mark.parametrize("at", range(4))
def test_rotary_strides(L, at):
    """2^31 rows 2^40 elements apart: 2^72 bytes."""
    T, H = (2**31 - 1, 1) if at % 2 == 0 else (1, 2**31 - 1)
    strides = [8 * H, 8, 8 * H, 8] if at % 2 == 0 else [0, 8, 0, 8]
    strides[at] = 2**40
    assert rope(L, T, H, strides) == INV
    assert rope(L, T, H, strides, out=9) == INV
    strides[at] = 2**62
    assert rope(L, T, H, strides) == INV


def test_rotary_large_spans(L):
    """What stays in 64 bits is compared: rows 2^57 elements apart overlap nothing below the first, and all above it."""
    assert rope(L, 2, 1, (2**57, 0, 8, 0)) not in (INV, ALIAS)
    assert rope(L, 2, 1, (2**57, 0, 8, 0), out=10) == ALIAS
    assert rope(L, 1, 2, (0, 8, 0, 2**57), out=10) not in (INV, ALIAS)
    assert rope(L, 1, 2, (0, 8, 0, 2**57)) == ALIAS
    assert rope(L, 1, 4, (2**62, 8, 2**62, 8)) not in (INV, ALIAS)  # one token has no stride


def test_feed_forward_pitch(L):
    def fwd(T, ld, y=5):
        s = mlaq.FfnShape(T, 64, 128, ld, 0, 0)
        return L.mla_gated_ffn_fwd(ctypes.byref(s), p(0), p(1), p(2), None, ctypes.c_void_p(2**50), p(y), None, None)

    assert fwd(2**31 - 1024, 2**36) == INV
    assert fwd(2**20, 2**36, y=0) == ALIAS
