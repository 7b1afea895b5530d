"""Refusals of the 4-bit serving calls beside tests/test_q4_host.py's, without a GPU."""
import ctypes

import pytest

from verify_gated_gqa_gb300 import binding as B
from verify_gated_gqa_gb300 import build as build_mod

A = 0x10000        # an aligned fake device address (never dereferenced)


@pytest.fixture(scope="module")
def L():
    build_mod.build()
    return B.lib()


@pytest.mark.parametrize("n,ld,want", [(8, -1, -4), (8, -8, -4), (8, 1, -4), (0, 0, 0), (0, -1, -4)])
def test_axes_stride_between_axes(L, n, ld, want):
    """0 (one row of positions for all axes) or at least n_tok."""
    before = L.ga_debug_cuda_calls()
    assert L.ga_qk_prologue_axes(A, A, A, A, A, A, n, A, ld, 3, (ctypes.c_uint8 * 32)(), A, A, 64,
                                 None) == want
    assert L.ga_debug_cuda_calls() == before
