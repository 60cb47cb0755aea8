"""The bounds-checked build through attention and the cache write: outputs
within their bounds as in the other tests, and every checked index (table
entries, copies' boxes and places in shared memory, partial rows, seams,
output rows, the write's sources and places) inside its own."""
import ctypes
import os

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
    _lib._lib = saved


def failures(lib):
    out = (ctypes.c_uint32 * 3)()
    assert lib.dspark_checked_status(out) == 0
    assert out[2] == 1, "not the checked build"
    return out[0], out[1]


# every kernel: streaming with 8, 16, 24, 32 and 64 rows a CTA, the tensor kernel's three modes,
# with one and more row tiles
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("T,heads", [(1, 2), (2, 16), (6, 8), (8, 8), (33, 14), (64, 16)])
@pytest.mark.parametrize("page,layout", [(16, "nhd"), (8, "hnd"), (24, "nhd"), (128, "hnd"),
                                         (7, "nhd")])
def test_attention_under_checks(checked_lib, dim, T, heads, page, layout):
    failures(checked_lib)
    long = 9000 if T * heads <= 64 else 1500                      # cut items
    for ctx, nodes in (([long, long // 3], [T, T - T // 3]),
                       ([0, 1, 63, 64, 37], [T, 1, 0, T // 2 + 1, max(1, T - 1)])):
        c = Case(ctx, nodes, T, heads=heads, dim=dim, page=page, layout=layout, mask="tree",
                 dtype=torch.float16 if T == 8 else torch.bfloat16, seed=T + dim)
        c.run()
        c.table[0, :min(3, c.table.shape[1])] = -1                # released pages
        c.table[1, 0] = c.k.shape[0] + 5
        c.check(c.run())
    fails, site = failures(checked_lib)
    assert fails == 0, "site %d failed %d times" % (site, fails)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("T,heads", [(1, 8), (6, 8), (64, 16)])
def test_many_short_items_under_checks(checked_lib, dim, T, heads):
    failures(checked_lib)
    c = Case([i % 90 for i in range(300)], [i * 5 % (T + 1) if i % 9 else 1 for i in range(300)],
             T, heads=heads, dim=dim, seed=1)
    c.run()
    c.ctx[7], c.nodes[8], c.ctx[9] = -1, T + 1, c.table.shape[1] * 16
    status = c.run()[2].tolist()
    assert [b for b in range(300) if status[b]] == [7, 8, 9]
    fails, site = failures(checked_lib)
    assert fails == 0, "site %d failed %d times" % (site, fails)


@pytest.mark.parametrize("source", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("heads,dim,page", [(1, 8, 1), (3, 64, 16), (8, 128, 24), (5, 1024, 7)])
def test_write_under_checks(checked_lib, heads, dim, page, source):
    failures(checked_lib)
    blocks, n = 9, 50
    k, v = (torch.randn(n, heads, dim, device="cuda").to(source) for _ in range(2))
    kc, vc = (torch.zeros(blocks, page, heads, dim, dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    g = torch.Generator().manual_seed(dim)
    slots = torch.randperm(blocks * page + 9, generator=g)[:n] - 5  # some outside the cache
    rows = torch.randint(-2, n + 2, slots.shape, generator=g)
    want = torch.zeros(2, blocks * page, heads, dim, dtype=torch.bfloat16, device="cuda")
    for s, r in zip(slots.tolist(), rows.tolist()):
        if 0 <= s < blocks * page and 0 <= r < n:
            want[0, s], want[1, s] = k[r].to(torch.bfloat16), v[r].to(torch.bfloat16)
    ds.kv_write(k, v, kc, vc, slots.to(torch.int32).cuda(), rows.to(torch.int32).cuda())
    torch.cuda.synchronize()
    assert torch.equal(kc.view(want[0].shape), want[0])
    assert torch.equal(vc.view(want[1].shape), want[1])
    fails, site = failures(checked_lib)
    assert fails == 0, "site %d failed %d times" % (site, fails)
