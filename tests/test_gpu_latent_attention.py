"""dspark_latent_attention against attention in 64 bits: sizes of the latent
vector and of the rotated part, head counts, lengths from none to long ones,
pages, trees, masks that leave a row nothing, released pages, and what the
kernel must not let through.

The bound on an element is that of dspark_tree_attention's tests: with u the
unit roundoff of the type (2^-8 bf16, 2^-11 f16) the softmax weights and the
result are each rounded once, u (sum p|v| + |out|), f16 weights below its
normal range by at most 2^-25 each; the fp32 scores are off by at most W 2^-23
sum|q k| scale each (W elements a row), which moves a weight by that much
again, twice over (its own and the sum's), and exponentials and sums by a few
2^-22."""
import math

import numpy as np
import pytest
import torch

import draft_sampling_verification_gb300 as ds
import latent_ref as ref

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def f64(t):
    return t.double().cpu().numpy()


class Case:
    """Random inputs: ctx and nodes are the requests' lengths, blocks are scattered."""

    def __init__(self, ctx, nodes, T, heads=16, latent=512, rope=64, page=16,
                 dtype=torch.bfloat16, mask=None, seed=0, spread=2.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        B, W = len(ctx), latent + rope
        self.page, self.latent, self.scale = page, latent, W ** -0.5
        pages = [max(0, -(-(c + n) // page)) for c, n in zip(ctx, nodes)]
        wide, blocks = max(pages) + 1, sum(pages) + 5
        self.cache = torch.randn(blocks, page, W, generator=g, device="cuda").to(dtype)
        self.q = (spread * torch.randn(B, T, heads, W, generator=g, device="cuda")).to(dtype)
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
        return [self.q, self.cache, torch.from_numpy(self.table).cuda(),
                torch.from_numpy(self.ctx).cuda(), torch.from_numpy(self.nodes).cuda(), m]

    def call(self, *a, **kw):
        q, cache, table, ctx, nodes, m = a or self.device()
        return ds.latent_attention(q, cache, table, ctx, nodes, self.latent, self.scale,
                                   tree_mask=m, **kw)

    def run(self, **kw):
        r = self.call(**kw)
        torch.cuda.synchronize()
        return r

    def into(self, out, ws):
        q, cache, table, ctx, nodes, m = self.device()
        ds.dspark_latent_attention(q, cache, table, ctx, nodes, self.latent, m, self.scale, *out, ws)

    def workspace(self):
        return ds.dspark_latent_attention_workspace_bytes(*self.q.shape[:3], self.latent)

    def check(self, got):
        out, lse, status = got
        want, wlse, weight, reach = ref.latent_attention(
            f64(self.q), f64(self.cache), self.table, self.ctx, self.nodes, self.mask, self.scale,
            self.latent)
        u, W = U[self.q.dtype], self.q.shape[-1]
        score = W * 2.0 ** -23 * reach + 2.0 ** -20
        most = float(self.cache.abs().max())
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
@pytest.mark.parametrize("latent,rope", [(512, 64), (256, 32)])
@pytest.mark.parametrize("T,mask", [(1, None), (6, None), (6, "tree"), (17, "tree"), (64, "tree"),
                                    (64, None), (64, "random")])
def test_types_sizes_and_trees(dtype, latent, rope, T, mask):
    c = Case([0, 1, 63, 64, 127, 128, 200, 1000], [T, 1, T, max(1, T - 1), T, T, T,
                                                  0 if T == 1 else T // 2], T,
             latent=latent, rope=rope, dtype=dtype, mask=mask, seed=latent + T)
    c.check(c.run())


@pytest.mark.parametrize("latent,rope", [(64, 0), (64, 64), (128, 8), (192, 64), (256, 0), (256, 64),
                                         (320, 24), (384, 64), (448, 40), (512, 0), (512, 8),
                                         (512, 56)])
def test_widths(latent, rope):
    c = Case([5, 300, 131], [3, 2, 3], 3, latent=latent, rope=rope, seed=latent + rope, mask="tree")
    c.check(c.run())


@pytest.mark.parametrize("heads", [1, 2, 7, 16, 21, 64, 65, 127, 128])
@pytest.mark.parametrize("T", [1, 6, 33])
def test_head_counts(heads, T):
    c = Case([130, 77, 512], [T, T, 1], T, heads=heads, mask="tree", seed=heads)
    c.check(c.run())


@pytest.mark.parametrize("page", [8, 16, 24, 32, 40, 64, 96, 128, 1000])
@pytest.mark.parametrize("latent", [256, 512])
def test_pages_end_inside_a_tile(page, latent):
    c = Case([0, 5, page - 1, page, page + 1, 333], [6, 4, 6, 6, 1, 6], 6, page=page, latent=latent,
             seed=page)
    c.check(c.run())


@pytest.mark.parametrize("ctx", [[0], [1], [0, 0, 0], [8191], [5000, 1, 300, 20000], [60000, 2]])
@pytest.mark.parametrize("T,heads", [(1, 16), (5, 4), (4, 128)])
def test_lengths(ctx, T, heads):
    c = Case(ctx, [T] * len(ctx), T, heads=heads, seed=len(ctx))
    c.check(c.run())


def test_many_requests():
    rng = np.random.default_rng(3)
    c = Case([int(x) for x in rng.integers(0, 300, 700)], [int(x) for x in rng.integers(0, 4, 700)],
             3, heads=2, latent=128, rope=16, seed=1)
    c.check(c.run())
    c = Case([int(x) for x in rng.integers(0, 300, 90)], [int(x) for x in rng.integers(0, 4, 90)],
             3, heads=60, latent=512, rope=64, seed=1)
    c.check(c.run())


@pytest.mark.parametrize("T", [6, 64])
@pytest.mark.parametrize("latent", [256, 512])
def test_rows_that_see_nothing(T, latent):
    c = Case([0, 0, 40], [T, T, T], T, mask="none", latent=latent)
    out, lse, status = got = c.run()
    c.check(got)
    assert (out[:2] == 0).all() and torch.isneginf(lse[:2]).all()
    c = Case([0, 20], [0, 0], T, latent=latent)
    out, lse, status = c.run()
    assert (out == 0).all() and torch.isneginf(lse).all() and (status == 0).all()


@pytest.mark.parametrize("T", [5, 64])
def test_released_pages_are_not_seen(T):
    c = Case([500, 333, 64], [T] * 3, T)
    c.table[0, :11] = -1
    c.table[0, 17] = c.cache.shape[0]          # beyond the cache
    c.table[1, :] = 2 ** 31 - 1                # nothing left at all
    c.table[2, 1] = -7
    got = c.run()
    c.check(got)
    assert (got[0][1] == 0).all()


@pytest.mark.parametrize("poison", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("T,heads", [(6, 8), (40, 16)])
@pytest.mark.parametrize("latent", [256, 512])
@pytest.mark.parametrize("page", [16, 64])
def test_unseen_rows_do_not_leak(poison, T, heads, latent, page):
    """Whatever lies past a request's end, in blocks of nobody or at nodes that a row's tree
    hides stays out of the row."""
    c = Case([100, 37, 256], [T, T - 2, T - 1], T, mask="tree", heads=heads, latent=latent, seed=5,
             page=page)
    live = torch.zeros(c.cache.shape[:2], dtype=torch.bool)
    for b in range(3):
        for i in range(int(c.ctx[b] + c.nodes[b])):
            live[c.table[b, i // page], i % page] = True
    # the last node of each request: hidden from every row but its own
    own = []
    for b in range(3):
        n = int(c.nodes[b])
        for t in range(n - 1):
            assert not (int(c.mask[b, t]) >> (n - 1)) & 1
        i = int(c.ctx[b]) + n - 1
        live[c.table[b, i // page], i % page] = False
        own.append((b, n - 1))
    want = c.run()
    c.cache = torch.where(live.cuda()[..., None], c.cache, poison)
    out, lse, _ = c.run()
    hidden = torch.zeros(out.shape[:2], dtype=torch.bool)
    for b, t in own:
        hidden[b, t] = True
    keep = ~hidden.cuda()
    assert torch.equal(out[keep], want[0][keep]) and torch.equal(lse[keep], want[1][keep])
    for b, t in own:                            # the row that sees the poison shows it
        assert not torch.isfinite(out[b, t]).any()


def test_one_element_of_a_node():
    """An infinite element of one node: rows that see it are lost, the others keep their bits."""
    T = 6
    c = Case([50], [T], T, mask="tree", seed=9)
    want = c.run()[0]
    i = 50 + 2
    c.cache[int(c.table[0, i // 16]), i % 16, 5] = math.inf
    out, _, _ = c.run()
    sees = torch.tensor([(int(c.mask[0, t]) >> 2) & 1 == 1 for t in range(T)])
    assert sees.any() and not sees.all()
    assert torch.equal(~torch.isfinite(out[0, :, :, 5]).all(-1).cpu(), sees)
    assert torch.equal(out[0, ~sees], want[0, ~sees])


def test_strided_queries_caches_and_tables():
    c = Case([70, 300], [6, 5], 6, heads=8)
    want = c.run()
    a = c.device()
    big = torch.zeros(2, 6, 24, 640, dtype=c.q.dtype, device="cuda")
    big[:, :, 8:16, 32:608] = c.q
    a[0] = big[:, :, 8:16, 32:608]
    table = torch.full((2, c.table.shape[1] + 9), 99, dtype=torch.int32, device="cuda")
    table[:, :c.table.shape[1]] = torch.from_numpy(c.table)
    a[2] = table[:, :c.table.shape[1]]
    # rows further apart than they are long, every second block of a larger cache, NaN between
    rows = torch.full((2 * c.cache.shape[0], 20, 600), math.nan, dtype=c.q.dtype, device="cuda")
    a[1] = rows[::2, 2:18, 16:592]
    a[1].copy_(c.cache)
    got = c.call(*a)
    a[0] = c.q.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    again = c.call(*a)
    torch.cuda.synchronize()
    for x, y, z in zip(want, got, again):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_single_blocks_requests_and_broadcast_queries():
    """One block, one request, queries that all heads share: dimensions of any stride."""
    c = Case([9], [1], 1, heads=4)
    c.table[0, :] = 0
    c.check(c.run())
    a = c.device()
    a[1] = a[1][:1].as_strided((1, 16, 576), (8, 576, 1))
    c.cache = a[1]
    c.check(c.call(*a))
    c.q = c.q[:, :, :1].expand(1, 1, 4, 576)
    c.check(c.run())


@pytest.mark.parametrize("poison", [math.nan, math.inf, 3e38])
def test_queries_of_no_node(poison):
    """What stands in the queries behind a request's nodes reaches nothing."""
    c = Case([300, 4000, 0], [3, 1, 0], 5, heads=40, seed=8)
    want = c.run()
    for b in range(3):
        c.q[b, int(c.nodes[b]):] = poison
    got = c.run()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    assert (got[0][2] == 0).all() and torch.isneginf(got[1][1, 1:]).all()


def test_sizes_of_one_and_none():
    c = Case([33, 80], [1, 1], 1, heads=1)
    want = c.run()
    a = c.device()
    odd = torch.zeros(2, 577 * 8, dtype=c.q.dtype, device="cuda")
    odd[:, :576] = c.q[:, 0, 0]
    # one node and one head: their strides are no multiples of anything
    a[0] = odd.as_strided((2, 1, 1, 576), (577 * 8, 3, 5, 1))
    got = c.call(*a)
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    a = [c.q[:0], c.cache, a[2][:0], a[3][:0], a[4][:0], None]
    out, lse, status = c.call(*a)
    assert out.shape == (0, 1, 1, 512) and lse.shape == (0, 1, 1) and status.shape == (0,)


@pytest.mark.parametrize("scale", [0.31, -0.05, 0.0, 1e-39])
def test_scales(scale):
    c = Case([90, 11], [3, 3], 3, spread=0.3)
    c.scale = scale
    c.check(c.run())


def test_scores_far_apart():
    """Rising scores, so that the reference moves at every tile; and scores beyond fp16's range."""
    c = Case([2000, 700], [4, 4], 4, heads=32)
    c.cache[:] = 0.01 * c.cache
    for b in range(2):
        for i in range(int(c.ctx[b] + c.nodes[b])):
            c.cache[int(c.table[b, i // 16]), i % 16, 0] = i / 8
    c.q[..., 0] = 8.0
    c.scale = 1.0
    c.check(c.run())
    c.q[..., 0] = -8.0
    c.check(c.run())


def test_offsets_past_32_bits():
    """Blocks whose first element lies beyond 2^32 in the cache."""
    c = Case([400, 60], [6, 6], 6, seed=4)
    blocks = 2 ** 32 // (16 * 576) + 300
    cache = torch.empty(blocks, 16, 576, dtype=torch.bfloat16, device="cuda")
    n = c.cache.shape[0]
    cache[blocks - n:] = c.cache
    want = c.run()
    a = c.device()
    a[1] = cache
    a[2] = torch.where(a[2] >= 0, a[2] + (blocks - n), a[2])
    got = c.call(*a)
    torch.cuda.synchronize()
    for x, y in zip(want, got):
        assert torch.equal(x, y)


@pytest.mark.parametrize("T,heads", [(6, 8), (40, 16)])
def test_other_stream_stale_workspace_and_repeats(T, heads):
    c = Case([3000, 17, 900], [T, T, 1], T, heads=heads, mask="tree")
    want = c.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = c.run(stream=s)
    for fill in (0, 255):
        ws = torch.full((c.workspace(),), fill, dtype=torch.uint8, device="cuda")
        out = [torch.full_like(t, 7) for t in want]
        c.into(out, ws)
        torch.cuda.synchronize()
        for x, y, z in zip(want, got, out):
            assert torch.equal(x, y) and torch.equal(x, z)
    c.into([want[0].clone(), None, want[2].clone()], ws)        # without lse
    torch.cuda.synchronize()


@pytest.mark.parametrize("latent", [256, 512])
@pytest.mark.parametrize("T,heads", [(1, 2), (1, 128), (6, 8), (5, 25), (7, 40), (64, 2), (33, 14),
                                     (64, 16)])
def test_workspace_bounds(T, heads, latent):
    # few items of many tiles, so that nearly every range leaves partial rows
    c = Case([9000, 2500], [T, T - T // 3], T, heads=heads, latent=latent, mask="tree")
    want = c.run()
    n = c.workspace()
    for at in (256, 272):
        ws = torch.full((n + 4096,), 90, dtype=torch.uint8, device="cuda")
        out = [torch.empty_like(t) for t in want]
        c.into(out, ws[at:at + n])
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, out))
        assert (ws[:at] == 90).all() and (ws[at + n:] == 90).all()


def test_in_a_graph():
    c = Case([700, 80], [6, 6], 6)
    a = c.device()
    want = c.run()
    out = [torch.empty_like(t) for t in want]
    ws = torch.empty(c.workspace(), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ds.dspark_latent_attention(*a[:5], c.latent, a[5], c.scale, *out, ws)
    for _ in range(3):
        out[0].fill_(9)
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    a[3].fill_(33)                              # other lengths in the same graph
    c.ctx[:] = 33
    g.replay()
    torch.cuda.synchronize()
    c.check(out)


def test_bad_lengths_are_refused():
    c = Case([64, 64, 64, 64], [6, 6, 6, 6], 6)
    c.ctx[1], c.nodes[2], c.ctx[3] = -1, 7, c.table.shape[1] * 16
    out, lse, status = c.run()
    assert status.tolist() == [0, ds.ST_BAD_LENGTH, ds.ST_BAD_LENGTH, ds.ST_BAD_LENGTH]
    assert (out[1:] == 0).all() and torch.isneginf(lse[1:]).all()
    one = Case([64, 64, 64, 64], [6, 6, 6, 6], 6)
    assert torch.equal(out[0], one.run()[0][0])


def test_against_tree_attention():
    """A latent cache without a rotated part is a cache of one head whose keys are its values."""
    c = Case([300, 40, 7], [6, 5, 6], 6, heads=8, latent=64, rope=0, mask="tree")
    q, cache, table, ctx, nodes, m = c.device()
    one = cache[:, :, None]
    a = ds.tree_attention(q, one, one, table, ctx, nodes, tree_mask=m, scale=c.scale)
    b = c.run()
    # each within its own rounding of the other: two results and two sets of weights
    weight = float(cache.abs().max())
    assert ((a[0].float() - b[0].float()).abs() <= 4 * 2.0 ** -8 * weight).all()
    assert ((a[1] - b[1]).abs() <= 2.0 ** -12).masked_fill(torch.isinf(a[1]), True).all()


def test_the_binding_refuses():
    c = Case([64], [6], 6)
    q, cache, table, ctx, nodes, _ = c.device()
    ok = dict(q=q, cache=cache, block_table=table, ctx_len=ctx, n_nodes=nodes, latent_dim=512,
              scale=0.1)
    ds.latent_attention(**ok)
    for error, kw in ((ValueError, dict(q=q.half())), (ValueError, dict(q=q[..., :512])),
                      (ValueError, dict(q=q[0])), (TypeError, dict(cache=cache.float())),
                      (ValueError, dict(cache=cache[0])), (RuntimeError, dict(latent_dim=500)),
                      (RuntimeError, dict(latent_dim=448)), (RuntimeError, dict(latent_dim=576)),
                      (RuntimeError, dict(scale=float("nan"))),
                      (RuntimeError, dict(cache=cache[:, :12])),
                      (ValueError, dict(block_table=table.long())),
                      (TypeError, dict(ctx_len=ctx.long())),
                      (ValueError, dict(n_nodes=nodes.cpu())),
                      (ValueError, dict(cache=cache.transpose(1, 2)))):
        with pytest.raises(error):
            ds.latent_attention(**{**ok, **kw})
    with pytest.raises(ValueError):
        c.into([torch.empty(1, 6, 16, 512, dtype=q.dtype, device="cuda"), None,
                torch.empty(1, dtype=torch.int32, device="cuda")],
               torch.empty(c.workspace() - 1, dtype=torch.uint8, device="cuda"))
