"""Scales whose product with log2(e) is no fp32 number are refused."""
import ctypes

import pytest

from draft_sampling_verification_gb300 import _lib, build

P = ctypes.c_void_p(16)        # a non-null, aligned placeholder; never dereferenced


@pytest.mark.parametrize("scale", [2.4e38, 2.9e38, -2.4e38, -2.9e38])
def test_scale_too_large(scale):
    build.build()
    # an empty batch: nothing would be launched
    assert _lib.load().dspark_tree_attention(P, 1, 6144, 1024, 128, 0, 6, 8, 2, 128, P, P, 4096, 256,
                                             128, 5, 16, P, 4, 4, P, P, None, scale, P, None, P, P,
                                             None) == -7
