"""Refusals of the calls over pages beside tests/test_q8_host.py's, without a GPU."""
import pytest

from verify_gated_gqa_gb300 import binding as B
from verify_gated_gqa_gb300 import build as build_mod

A = 0x10000        # an aligned fake device address (never dereferenced)


@pytest.fixture(scope="module")
def L():
    build_mod.build()
    return B.lib()


@pytest.mark.parametrize("moves,want", [(-1, -2), (1 << 30, -4), ((1 << 31) - 9000, -4), ((1 << 31) - 1, -4),
                                        ((1 << 30) - 1, -6), (0, -6)])
def test_compact_limits_its_move_lists(L, moves, want):
    """Below 2^30 entries, as the copies' lists; the workspace is looked at after them (so no case here
    gets as far as a launch)."""
    before = L.ga_debug_cuda_calls()
    assert L.ga_page_compact(4, A, A, 8, A, A, A, 100, A, A, A, moves, A, A, A, None, 0, None) == want
    assert L.ga_debug_cuda_calls() == before
