"""dspark_tree_attention against attention in 64 bits: head layouts, lengths
from none to long ones, pages of any size, trees, masks that leave a row
nothing, released pages, and what the kernel must not let through (values in
unseen places, other requests, a stale workspace).

The bound on an element comes from the header's rounding rules, with u the
unit roundoff of the type (2^-8 bf16, 2^-11 f16): the softmax weights and
the result are each rounded once, u (sum p|v| + |out|), f16 weights below
its normal range by at most 2^-25 each; the fp32 scores are off by at most
D 2^-23 sum|q k| scale each, which moves a weight by that much again, twice
over (its own and the sum's), and exponentials and sums by a few 2^-22."""
import math

import numpy as np
import pytest
import torch

import draft_sampling_verification_gb300 as ds
import serving_ref as ref

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def f64(t):
    return t.double().cpu().numpy()


class Case:
    """Random inputs: ctx and nodes are the requests' lengths, blocks are scattered."""

    def __init__(self, ctx, nodes, T, heads=8, kv_heads=2, dim=128, page=16,
                 dtype=torch.bfloat16, layout="nhd", mask=None, seed=0, spread=2.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        B = len(ctx)
        self.page, self.scale = page, dim ** -0.5
        pages = [max(0, -(-(c + n) // page)) for c, n in zip(ctx, nodes)]
        wide, blocks = max(pages) + 1, sum(pages) + 5
        store = (blocks, page, kv_heads, dim) if layout == "nhd" else (blocks, kv_heads, page, dim)
        k = torch.randn(store, generator=g, device="cuda").to(dtype)
        v = torch.randn(store, generator=g, device="cuda").to(dtype)
        self.k, self.v = (k, v) if layout == "nhd" else (k.transpose(1, 2), v.transpose(1, 2))
        self.q = (spread * torch.randn(B, T, heads, dim, generator=g, device="cuda")).to(dtype)
        order = torch.randperm(blocks, generator=g, device="cuda").cpu().numpy()
        self.table = np.full((B, wide), -1, np.int32)
        at = 0
        for b in range(B):
            self.table[b, :pages[b]] = order[at:at + pages[b]]
            at += pages[b]
        self.ctx, self.nodes = np.array(ctx, np.int32), np.array(nodes, np.int32)
        rng = np.random.default_rng(seed)
        if mask == "tree":
            self.mask = np.zeros((B, T), np.uint64)
            for b in range(B):
                for t in range(T):
                    parent = int(rng.integers(max(-1, t - 5), t)) if t else -1
                    self.mask[b, t] = np.uint64(1 << t) | (self.mask[b, parent] if parent >= 0
                                                           else np.uint64(0))
        elif mask == "random":
            self.mask = rng.integers(0, 1 << 63, (B, T), dtype=np.uint64) * np.uint64(2) + \
                rng.integers(0, 2, (B, T), dtype=np.uint64)
        elif mask == "none":
            self.mask = np.zeros((B, T), np.uint64)
        else:
            self.mask = None

    def device(self):
        m = None if self.mask is None else torch.from_numpy(self.mask.view(np.int64)).cuda()
        return (self.q, self.k, self.v, torch.from_numpy(self.table).cuda(),
                torch.from_numpy(self.ctx).cuda(), torch.from_numpy(self.nodes).cuda(), m)

    def run(self, **kw):
        r = ds.tree_attention(*self.device(), **kw)
        torch.cuda.synchronize()
        return r

    def check(self, got, k=None, v=None):
        out, lse, status = got
        want, wlse, weight, reach = ref.attention(
            f64(self.q), f64(self.k if k is None else k), f64(self.v if v is None else v),
            self.table, self.ctx, self.nodes, self.mask, self.scale)
        u, D = U[self.q.dtype], self.q.shape[-1]
        score = D * 2.0 ** -23 * reach + 2.0 ** -20
        most = float(np.abs(f64(self.v if v is None else v))[
            np.isfinite(f64(self.v if v is None else v))].max(initial=0))
        small = (self.ctx + self.nodes).max() * most * 2.0 ** -25 if u == 2.0 ** -11 else 0.0
        tol = u * (weight * (1 + u) + np.abs(want)) + 2 * score[..., None] * weight + small
        err = np.abs(f64(out) - want)
        assert np.isfinite(f64(out)).all()
        assert (err <= tol + 1e-30).all(), float((err / (tol + 1e-30)).max())
        lse = f64(lse)
        assert np.array_equal(np.isinf(lse), np.isinf(wlse))
        fine = np.isfinite(wlse)
        assert (np.abs(lse[fine] - wlse[fine]) <= score[fine] + 2.0 ** -22 * np.abs(wlse[fine])
                + 2.0 ** -18).all()
        assert (status.cpu().numpy() == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("T,mask", [(1, None), (6, None), (6, "tree"), (17, "tree"), (64, "tree"),
                                    (64, None), (64, "random")])
def test_types_dims_and_trees(dtype, dim, T, mask):
    c = Case([0, 1, 63, 64, 200, 1000], [T, 1, T, max(1, T - 1), T, 0 if T == 1 else T // 2], T,
             dim=dim, dtype=dtype, mask=mask, seed=dim + T)
    c.check(c.run())


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 3), (8, 1), (7, 1), (14, 2), (32, 8),
                                            (64, 1), (40, 5)])
@pytest.mark.parametrize("T", [1, 6, 33])
def test_head_layouts(heads, kv_heads, T):
    c = Case([130, 77, 512], [T, T, 1], T, heads=heads, kv_heads=kv_heads, mask="tree", seed=heads)
    c.check(c.run())


@pytest.mark.parametrize("page", [1, 3, 8, 16, 24, 100, 128, 1000])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
def test_pages_end_inside_a_tile(page, layout):
    c = Case([0, 5, page - 1, page, page + 1, 333], [6, 4, 6, 6, 1, 6], 6, page=page, layout=layout,
             seed=page)
    c.check(c.run())


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("T,heads", [(2, 4), (13, 8), (20, 16), (64, 16)])
@pytest.mark.parametrize("page", [8, 24, 32, 12])
def test_pages_dims_and_row_counts(page, T, heads, dim):
    """Rows of an item from 4 to 512, on every kernel, with boxes of eight rows, of more, and none."""
    c = Case([37, 0, 260, 129], [T, max(1, T - 3), T, 1], T, heads=heads, kv_heads=2, dim=dim,
             page=page, mask="tree", seed=page + T, dtype=torch.float16)
    c.check(c.run())


@pytest.mark.parametrize("ctx", [[0], [1], [0, 0, 0], [8191], [5000, 1, 300, 20000], [40000, 2]])
@pytest.mark.parametrize("T", [1, 5])
def test_lengths(ctx, T):
    c = Case(ctx, [T] * len(ctx), T, heads=4, kv_heads=1, seed=len(ctx))
    c.check(c.run())


def test_many_requests():
    rng = np.random.default_rng(3)
    c = Case([int(x) for x in rng.integers(0, 300, 700)], [int(x) for x in rng.integers(0, 4, 700)],
             3, heads=2, kv_heads=1, dim=64, seed=1)
    c.check(c.run())


@pytest.mark.parametrize("T", [6, 64])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_rows_that_see_nothing(T, dim):
    c = Case([0, 0, 40], [T, T, T], T, mask="none", dim=dim)
    out, lse, status = got = c.run()
    c.check(got)
    assert (out[:2] == 0).all() and torch.isneginf(lse[:2]).all()
    c = Case([0, 20], [0, 0], T, dim=dim)
    out, lse, status = c.run()
    assert (out == 0).all() and torch.isneginf(lse).all() and (status == 0).all()


@pytest.mark.parametrize("T", [5, 64])
def test_released_pages_are_not_seen(T):
    c = Case([500, 333, 64], [T] * 3, T, heads=16, kv_heads=2)
    c.table[0, :11] = -1
    c.table[0, 17] = c.k.shape[0]              # beyond the cache
    c.table[1, :] = 2 ** 31 - 1                # nothing left at all
    c.table[2, 1] = -7
    got = c.run()
    c.check(got)
    assert (got[0][1] == 0).all()


@pytest.mark.parametrize("poison", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("T,heads", [(6, 8), (40, 16)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_unseen_values_do_not_leak(poison, T, heads, dim):
    """Whatever lies past a request's end, in blocks of nobody or at nodes that a row's tree
    hides stays out of the row."""
    c = Case([100, 37, 256], [T, T - 2, T - 1], T, mask="tree", heads=heads, dim=dim, seed=5)
    k, v = c.k.clone(), c.v.clone()
    live = torch.zeros(c.k.shape[:2], dtype=torch.bool)
    for b in range(3):
        for i in range(int(c.ctx[b] + c.nodes[b])):
            live[c.table[b, i // c.page], i % c.page] = True
    # the last node of each request: hidden from every row but its own
    own = []
    for b in range(3):
        n = int(c.nodes[b])
        for t in range(n - 1):
            assert not (int(c.mask[b, t]) >> (n - 1)) & 1
        i = int(c.ctx[b]) + n - 1
        live[c.table[b, i // c.page], i % c.page] = False
        own.append((b, n - 1))
    live = live.cuda()[..., None, None]
    want = c.run()
    c.k, c.v = torch.where(live, k, poison), torch.where(live, v, poison)
    out, lse, _ = c.run()
    hidden = torch.zeros(out.shape[:2], dtype=torch.bool)
    for b, t in own:
        hidden[b, t] = True
    keep = ~hidden.cuda()
    assert torch.equal(out[keep], want[0][keep]) and torch.equal(lse[keep], want[1][keep])
    for b, t in own:                            # the row that sees the poison shows it
        assert not torch.isfinite(out[b, t]).any()


def test_values_alone_do_not_leak():
    """Infinite values under finite keys, at a node that some rows see and others do not."""
    T = 6
    c = Case([50], [T], T, mask="tree", seed=9)
    i = 50 + 2
    c.v[int(c.table[0, i // 16]), i % 16, :, 5] = math.inf
    out, _, _ = c.run()
    sees = torch.tensor([(int(c.mask[0, t]) >> 2) & 1 == 1 for t in range(T)])
    bad = ~torch.isfinite(out[0, :, :, 5]).all(-1).cpu()
    assert torch.equal(bad, sees)
    rest = torch.cat([out[..., :5], out[..., 6:]], -1)
    assert torch.isfinite(rest).all()


def test_strided_queries_and_tables():
    c = Case([70, 300], [6, 5], 6, heads=8, kv_heads=2)
    want = c.run()
    big = torch.zeros(2, 6, 24, 128, dtype=c.q.dtype, device="cuda")   # q inside a fused qkv
    big[:, :, 8:16] = c.q
    table = torch.full((2, c.table.shape[1] + 9), 99, dtype=torch.int32, device="cuda")
    table[:, :c.table.shape[1]] = torch.from_numpy(c.table)
    a = list(c.device())
    a[0], a[3] = big[:, :, 8:16], table[:, :c.table.shape[1]]
    got = ds.tree_attention(*a)
    by_head = c.q.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    a[0] = by_head
    again = ds.tree_attention(*a)
    torch.cuda.synchronize()
    for x, y, z in zip(want, got, again):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_scale_and_one_tensor_for_both_caches():
    c = Case([90, 11], [3, 3], 3)
    both = torch.stack([c.k, c.v])
    c.k, c.v = both[0], both[1]
    c.scale = 0.31
    c.check(c.run(scale=0.31))
    c.scale = -0.05
    c.check(c.run(scale=-0.05))


def test_offsets_past_32_bits():
    """Blocks whose first element lies beyond 2^32 in the cache."""
    page, kv_heads, dim = 16, 8, 128
    blocks = 2 ** 32 // (page * kv_heads * dim) + 300
    k = torch.empty(blocks, page, kv_heads, dim, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    c = Case([400, 60], [6, 6], 6, kv_heads=kv_heads, heads=16, seed=4)
    n = c.k.shape[0]
    k[blocks - n:], v[blocks - n:] = c.k, c.v
    want = c.run()
    a = list(c.device())
    a[1], a[2] = k, v
    a[3] = torch.where(a[3] >= 0, a[3] + (blocks - n), a[3])
    got = ds.tree_attention(*a)
    torch.cuda.synchronize()
    for x, y in zip(want, got):
        assert torch.equal(x, y)


@pytest.mark.parametrize("T,heads", [(6, 8), (64, 16)])
def test_other_stream_stale_workspace_and_repeats(T, heads):
    c = Case([3000, 17, 900], [T, T, 1], T, heads=heads, mask="tree")
    want = c.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = c.run(stream=s)
    B, T, H, D = c.q.shape
    n = ds.dspark_tree_attention_workspace_bytes(B, T, H, c.k.shape[2], D)
    for fill in (0, 255):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        o, l = torch.full_like(want[0], 7), torch.full_like(want[1], 7)
        st = torch.full_like(want[2], 7)
        a = c.device()
        ds.dspark_tree_attention(*a, c.scale, o, l, st, ws)
        torch.cuda.synchronize()
        for x, y, z in zip(want, got, (o, l, st)):
            assert torch.equal(x, y) and torch.equal(x, z)


@pytest.mark.parametrize("page", [16, 12])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("T,heads", [(1, 2), (1, 16), (6, 8), (5, 10), (7, 40), (64, 2), (33, 14),
                                     (64, 16)])
def test_workspace_bounds(T, heads, dim, page):
    # few items of many tiles, so that nearly every range leaves partial rows
    c = Case([9000, 2500], [T, T - T // 3], T, heads=heads, dim=dim, page=page, mask="tree")
    want = c.run()
    n = ds.dspark_tree_attention_workspace_bytes(2, T, heads, c.k.shape[2], dim)
    for at in (256, 272):
        ws = torch.full((n + 4096,), 90, dtype=torch.uint8, device="cuda")
        out = [torch.empty_like(t) for t in want]
        ds.dspark_tree_attention(*c.device(), c.scale, *out, ws[at:at + n])
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, out))
        assert (ws[:at] == 90).all() and (ws[at + n:] == 90).all()


def test_in_a_graph():
    c = Case([700, 80], [6, 6], 6)
    a = c.device()
    want = c.run()
    out, lse, st = (torch.empty_like(t) for t in want)
    ws = torch.empty(ds.dspark_tree_attention_workspace_bytes(2, 6, 8, 2, 128), dtype=torch.uint8,
                     device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ds.dspark_tree_attention(*a, c.scale, out, lse, st, ws)
    for _ in range(3):
        out.fill_(9)
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_bad_lengths_are_refused():
    c = Case([64, 64, 64, 64], [6, 6, 6, 6], 6)
    c.ctx[1], c.nodes[2], c.ctx[3] = -1, 7, c.table.shape[1] * 16
    out, lse, status = c.run()
    assert status.tolist() == [0, ds.ST_BAD_LENGTH, ds.ST_BAD_LENGTH, ds.ST_BAD_LENGTH]
    assert (out[1:] == 0).all() and torch.isneginf(lse[1:]).all()
    one = Case([64, 64, 64, 64], [6, 6, 6, 6], 6)
    assert torch.equal(one.run()[0][0], out[0])


@pytest.mark.parametrize("dim,T,heads", [(64, 8, 8), (128, 8, 8), (256, 8, 8), (128, 2, 8),
                                         (128, 40, 16)])
@pytest.mark.parametrize("scale", [0.0, -0.2])
def test_zero_and_negative_scales(dim, T, heads, scale):
    c = Case([100, 3, 300], [T, T, 1], T, heads=heads, dim=dim, mask="tree", seed=2)
    c.scale = scale
    c.check(c.run(scale=scale))


def test_lse_is_optional():
    c = Case([64], [6], 6)
    want = c.run()
    out, st = torch.empty_like(want[0]), torch.empty_like(want[2])
    ws = torch.empty(ds.dspark_tree_attention_workspace_bytes(1, 6, 8, 2, 128), dtype=torch.uint8,
                     device="cuda")
    ds.dspark_tree_attention(*c.device(), c.scale, out, None, st, ws)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0])


def test_binding_refuses():
    c = Case([64], [6], 6)
    a = list(c.device())

    def bad(exc, **kw):
        b = list(a)
        for i, x in kw.items():
            b[int(i[1:])] = x
        with pytest.raises(exc):
            ds.tree_attention(*b)

    bad(ValueError, a0=a[0].half())                        # another type than the caches'
    bad(ValueError, a0=a[0][0])                            # three dimensions
    bad(TypeError, a1=a[1].float(), a2=a[2].float())       # a single-precision cache
    bad(ValueError, a2=a[2][:1])                           # caches of different shapes
    bad(ValueError, a3=a[3].long())
    bad(TypeError, a4=a[4].long())
    bad(ValueError, a5=torch.cat([a[5], a[5]]))
    bad(TypeError, a6=torch.zeros(1, 6, dtype=torch.int32, device="cuda"))
    with pytest.raises(RuntimeError):                      # head_dim 96
        ds.tree_attention(a[0][..., :96], a[1][..., :96], a[2][..., :96], *a[3:])
