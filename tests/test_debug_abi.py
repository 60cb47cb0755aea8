"""The normal build has no switch that makes attention's waits expire."""
from draft_sampling_verification_gb300 import _lib, build


def test_stall_switch_is_of_the_checked_build_alone():
    build.build()
    lib = _lib.load()
    assert lib.dspark_debug_stall_attention(-1) == 0
    assert lib.dspark_debug_stall_attention(0) == -7
    assert lib.dspark_debug_stall_attention(-2) == -7
