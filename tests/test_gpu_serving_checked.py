"""The bounds-checked build through the cache plan and the logit processing:
their outputs against the plain implementations, and every checked index in
its bounds."""
import ctypes
import os

import numpy as np
import pytest
import torch

from draft_sampling_verification_gb300 import _lib, build
from test_gpu_cache import plan_case, trees
from test_gpu_logits import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def checked_lib():
    if not os.path.exists(build.LIB_CHECKED):
        build.build(checked=True)
    saved = _lib._lib
    _lib._lib = None
    lib = _lib.load(build.LIB_CHECKED)
    yield lib
    _lib._lib = saved


def failures(lib):
    out = (ctypes.c_uint32 * 3)()
    assert lib.dspark_checked_status(out) == 0
    assert out[2] == 1, "not the checked build"
    return out[0]


@pytest.mark.parametrize("B,T", [(1, 1), (300, 6), (40, 64)])
def test_plan_under_checks(checked_lib, B, T):
    rng = np.random.default_rng(B)
    ctx, new = rng.integers(0, 70, B).tolist(), rng.integers(0, T + 1, B).tolist()
    for n_free in (0, 7, B * 9):
        plan_case(ctx, new, T, 16, 9, n_free, trees(rng, B, T))
    assert failures(checked_lib) == 0


@pytest.mark.parametrize("V", [1, 31, 4099, 20011])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_logits_under_checks(checked_lib, V, dtype):
    c = Case(3, 6, V, dtype, history=3 * V if V < 100 else 500, biases=min(V, 60), masks=3, seed=V)
    c.check(c.run()[0])
    torch.cuda.synchronize()
    assert failures(checked_lib) == 0
