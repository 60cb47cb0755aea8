"""Latent attention in the bounds-checked build: results within their bounds
as in the other tests, and every checked index (table entries, copies' boxes
and places in shared memory, queries, partial rows, seams, output rows)
inside its own; and a wait that expires."""
import ctypes
import os
import time

import pytest
import torch

import draft_sampling_verification_gb300 as ds
from draft_sampling_verification_gb300 import _lib, build
from test_gpu_latent_attention import Case

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


def failures(lib):
    out = (ctypes.c_uint32 * 3)()
    assert lib.dspark_checked_status(out) == 0
    assert out[2] == 1, "not the checked build"
    return out[0], out[1]


@pytest.mark.parametrize("latent,rope", [(512, 64), (320, 8), (256, 64), (64, 0)])
@pytest.mark.parametrize("T,heads", [(1, 2), (2, 64), (6, 16), (7, 40), (64, 16)])
@pytest.mark.parametrize("page", [8, 16, 24, 32, 64, 128])
def test_under_checks(checked_lib, latent, rope, T, heads, page):
    failures(checked_lib)
    long = 9000 if T * heads <= 128 else 1500                     # cut items
    for ctx, nodes in (([long, long // 3], [T, T - T // 3]),
                       ([0, 1, 63, 128, 37], [T, 1, 0, T // 2 + 1, max(1, T - 1)])):
        c = Case(ctx, nodes, T, heads=heads, latent=latent, rope=rope, page=page, mask="tree",
                 dtype=torch.float16 if T == 7 else torch.bfloat16, seed=T + latent)
        c.run()
        c.table[0, :min(3, c.table.shape[1])] = -1                # released pages
        c.table[1, 0] = c.cache.shape[0] + 5
        c.check(c.run())
    a = c.device()                                                # queries without a map
    a[0] = torch.zeros(c.q.shape[0], c.q.shape[1] + 1, *c.q.shape[2:], dtype=c.q.dtype,
                       device="cuda")[:, 1:].copy_(c.q).transpose(1, 2).contiguous().transpose(1, 2)
    c.check(c.call(*a))
    fails, site = failures(checked_lib)
    assert fails == 0, "site %d failed %d times" % (site, fails)


def test_many_short_items_under_checks(checked_lib):
    failures(checked_lib)
    c = Case([i % 7 for i in range(500)], [1 + i % 3 for i in range(500)], 3, heads=50)
    c.check(c.run())
    fails, site = failures(checked_lib)
    assert fails == 0, "site %d failed %d times" % (site, fails)


@pytest.mark.parametrize("latent,T,heads", [(512, 6, 16), (256, 6, 16), (512, 40, 16)])
@pytest.mark.parametrize("cta", [0, 1, 61])
def test_a_wait_that_expires(checked_lib, latent, T, heads, cta):
    """One CTA is left without its copies, so that its pair's waits run into their limit of 2 s: its
    requests get DSPARK_ST_TIMEOUT, each of their rows is the result or NaN, never what the
    workspace or the output held before; all other requests and later calls are as ever."""
    c = Case([20] * 40 + [3000] * 20, [T] * 60, T, heads=heads, latent=latent, seed=cta)
    ws = torch.empty(c.workspace(), dtype=torch.uint8, device="cuda")

    def run():
        ws.fill_(63)                             # 0.747: finite garbage, were it read
        o = [torch.full((60, T, heads, latent), 7.0, dtype=c.q.dtype, device="cuda"),
             torch.full((60, T, heads), 7.0, device="cuda"),
             torch.full((60,), -1, dtype=torch.int32, device="cuda")]
        t0 = time.perf_counter()
        c.into(o, ws)
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
