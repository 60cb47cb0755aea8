"""The plan's work grows with the square of its requests, so their number has a limit."""
import ctypes

import pytest

from draft_sampling_verification_gb300 import _lib, build

P = ctypes.c_void_p(16)        # a non-null, aligned placeholder; never dereferenced


@pytest.mark.parametrize("B", [(1 << 20) + 1, 1 << 24, 1 << 30, 2 ** 31 - 1])
def test_more_requests_are_refused(B):
    build.build()
    assert _lib.load().dspark_cache_plan(P, P, B, 1, 16, P, 4, 4, P, 9, None, None, P, None, None, P,
                                         P, None) == -2
