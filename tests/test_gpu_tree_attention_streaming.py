"""The hard cases of attention on the streaming kernel: few rows of an item,
and blocks that are no multiple of eight token rows, whatever the rows.  The
same claims as in test_gpu_tree_attention, whose shapes take the tensor
kernel: nothing seen, released pages, poison in unseen places, refused
lengths, stale workspaces, other streams and graphs; with that file's bounds."""
import math

import pytest
import torch

import draft_sampling_verification_gb300 as ds
from test_gpu_tree_attention import Case

pytestmark = pytest.mark.gpu

# (head_dim, nodes, query heads on two cached ones, block size): 8 and 16 rows where blocks have
# tensor copies, 8 to 320 where they have none
SHAPES = [(64, 2, 8, 16), (64, 1, 32, 16), (128, 2, 8, 16), (128, 1, 2, 64), (64, 6, 8, 12),
          (64, 40, 16, 12), (128, 4, 8, 12), (128, 6, 8, 3), (128, 8, 8, 12), (128, 40, 16, 12),
          (256, 2, 8, 12), (256, 4, 8, 1), (256, 6, 8, 12), (256, 40, 16, 100)]
DTYPES = [torch.bfloat16, torch.float16]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim,T,heads,page", SHAPES)
def test_rows_that_see_nothing(dim, T, heads, page, dtype):
    c = Case([0, 0, 40], [T, T, T], T, mask="none", dim=dim, heads=heads, page=page, dtype=dtype)
    out, lse, _ = got = c.run()
    c.check(got)
    assert (out[:2] == 0).all() and torch.isneginf(lse[:2]).all()
    c = Case([0, 20], [0, 0], T, dim=dim, heads=heads, page=page, dtype=dtype)
    out, lse, status = c.run()
    assert (out == 0).all() and torch.isneginf(lse).all() and (status == 0).all()


@pytest.mark.parametrize("dim,T,heads,page", SHAPES)
def test_released_pages_are_not_seen(dim, T, heads, page):
    c = Case([500, 333, 64], [T] * 3, T, heads=heads, dim=dim, page=page, mask="tree")
    c.table[0, :3] = -1
    c.table[0, 500 // page] = c.k.shape[0]     # beyond the cache, nodes' places among them
    c.table[1, :] = 2 ** 31 - 1                # nothing left at all
    c.table[2, 64 // page // 2] = -7
    got = c.run()
    c.check(got)
    assert (got[0][1] == 0).all()


@pytest.mark.parametrize("poison", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim,T,heads,page", SHAPES)
def test_unseen_values_do_not_leak(dim, T, heads, page, dtype, poison):
    """Past a request's end, in blocks of nobody, and at the last node, which its tree hides from
    all rows but its own."""
    c = Case([100, 37, 256], [T, max(1, T - 2), max(1, T - 1)], T, mask="tree", heads=heads,
             dim=dim, page=page, dtype=dtype, seed=5)
    live = torch.zeros(c.k.shape[:2], dtype=torch.bool)
    own = []
    for b in range(3):
        n = int(c.nodes[b])
        for i in range(int(c.ctx[b]) + n - 1):
            live[c.table[b, i // page], i % page] = True
        for t in range(n - 1):
            assert not (int(c.mask[b, t]) >> (n - 1)) & 1
        own.append((b, n - 1))
    live = live.cuda()[..., None, None]
    want = c.run()
    c.k, c.v = torch.where(live, c.k, poison), torch.where(live, c.v, poison)
    out, lse, _ = c.run()
    keep = torch.ones(out.shape[:2], dtype=torch.bool, device="cuda")
    for b, t in own:
        keep[b, t] = False
        assert not torch.isfinite(out[b, t]).any()
    assert torch.equal(out[keep], want[0][keep]) and torch.equal(lse[keep], want[1][keep])


@pytest.mark.parametrize("dim,T,heads,page", [s for s in SHAPES if s[1] > 2])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_values_alone_do_not_leak(dim, T, heads, page, value):
    """A value that is not finite, under a finite key, reaches the rows that see its node."""
    c = Case([50, 7], [T, T], T, mask="tree", heads=heads, dim=dim, page=page, seed=9)
    i = 50 + 1
    c.v[int(c.table[0, i // page]), i % page, :, 5] = value
    want = c.run()
    out, _, _ = want
    sees = torch.tensor([(int(c.mask[0, t]) >> 1) & 1 == 1 for t in range(T)])
    got = out[0, :, :, 5].cpu()
    assert torch.isfinite(got[~sees]).all()
    assert (torch.isnan(got[sees]) if math.isnan(value) else got[sees] == value).all()
    rest = torch.cat([out[0, ..., :5], out[0, ..., 6:]], -1)
    assert torch.isfinite(rest).all() and torch.isfinite(out[1]).all()


@pytest.mark.parametrize("dim,T,heads,page", SHAPES)
def test_bad_lengths_are_refused(dim, T, heads, page):
    c = Case([64] * 4, [T] * 4, T, heads=heads, dim=dim, page=page)
    c.ctx[1], c.nodes[2], c.ctx[3] = -1, T + 1, c.table.shape[1] * page
    out, lse, status = c.run()
    assert status.tolist() == [0, ds.ST_BAD_LENGTH, ds.ST_BAD_LENGTH, ds.ST_BAD_LENGTH]
    assert (out[1:] == 0).all() and torch.isneginf(lse[1:]).all()
    c.check((out, lse, torch.zeros_like(status)))


@pytest.mark.parametrize("dim,T,heads,page", SHAPES)
def test_other_stream_stale_workspace_graph_and_repeats(dim, T, heads, page):
    c = Case([3000, 17, 900], [T, T, 1], T, heads=heads, dim=dim, page=page, mask="tree")
    want = c.run()
    c.check(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = c.run(stream=s)
    n = ds.dspark_tree_attention_workspace_bytes(3, T, heads, 2, dim)
    a = c.device()
    outs = [got]
    for fill in (0, 255):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        o = [torch.full_like(t, 7) for t in want]
        ds.dspark_tree_attention(*a, c.scale, *o, ws)
        outs.append(o)
    o = [torch.full_like(t, 7) for t in want]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ds.dspark_tree_attention(*a, c.scale, *o, ws)
    g.replay()
    outs.append(o)
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(x, y) for x, y in zip(want, o))


@pytest.mark.parametrize("dim,T,heads,page", SHAPES)
@pytest.mark.parametrize("scale", [0.0, -0.2])
def test_zero_and_negative_scales(dim, T, heads, page, scale):
    c = Case([100, 3, 300], [T, T, 1], T, heads=heads, dim=dim, page=page, mask="tree", seed=2)
    c.scale = scale
    c.check(c.run(scale=scale))
