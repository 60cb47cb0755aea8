"""A wait inside the tensor kernel that expires: the checked build leaves one
CTA without its copies of keys and values, so its waits for them run into
their limit of 2 s and it ends.  Its requests get DSPARK_ST_TIMEOUT, whatever
the other CTAs that share them report; each of their rows is either the
result or NaN, never what the workspace or the output held before; all other
requests and later calls are as ever.  No fault and no hang is involved."""
import os
import time

import pytest
import torch

import draft_sampling_verification_gb300 as ds
from draft_sampling_verification_gb300 import _lib, build
from test_gpu_tree_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def checked_lib():
    if not os.path.exists(build.LIB_CHECKED):
        build.build(checked=True)
    saved = _lib._lib
    _lib._lib = None
    lib = _lib.load(build.LIB_CHECKED)
    yield lib
    lib.dspark_debug_stall_attention(-1)
    _lib._lib = saved


# two row tiles' CTAs to a team at 64 nodes and 16 heads: CTA 1 and 61 are the second of theirs
@pytest.mark.parametrize("dim,T,heads", [(128, 6, 8), (64, 6, 16), (128, 64, 16), (64, 40, 16),
                                         (256, 6, 8)])
@pytest.mark.parametrize("cta", [0, 1, 61])
def test_its_requests_are_refused(checked_lib, dim, T, heads, cta):
    c = Case([20] * 40 + [3000] * 20, [T] * 60, T, heads=heads, dim=dim, seed=cta)
    a = c.device()
    n = ds.dspark_tree_attention_workspace_bytes(60, T, heads, 2, dim)
    ws = torch.full((n,), 63, dtype=torch.uint8, device="cuda")

    def run():
        ws.fill_(63)                             # 0.747: finite garbage, were it read
        o = [torch.empty_like(a[0]).fill_(7),
             torch.full((60, T, heads), 7.0, device="cuda"),
             torch.full((60,), -1, dtype=torch.int32, device="cuda")]
        t0 = time.perf_counter()
        ds.dspark_tree_attention(*a, c.scale, *o, ws)
        torch.cuda.synchronize()
        return (*o, time.perf_counter() - t0)

    want, wlse, status, _ = run()
    assert (status == 0).all()
    assert checked_lib.dspark_debug_stall_attention(cta) == 0
    out, lse, status, secs = run()
    assert checked_lib.dspark_debug_stall_attention(-1) == 0
    assert 1.5 < secs < 30
    late = status == ds.ST_TIMEOUT
    assert late.any() and ((status == 0) | late).all() and (status == 0).any()
    nan = torch.isnan(out)
    assert torch.equal(nan.all(-1), nan.any(-1)) and torch.equal(nan.all(-1), torch.isnan(lse))
    gone = nan.all(-1)
    assert torch.equal(out[~gone], want[~gone]) and torch.equal(lse[~gone], wlse[~gone])
    assert torch.equal(gone.flatten(1).any(1), late)
    again = run()
    assert torch.equal(again[0], want) and torch.equal(again[1], wlse) and (again[2] == 0).all()
