"""The new operators together, as a serving loop uses them: plan, rotation and
write, attention over the cache, a commit that writes the kept nodes again;
over a latent cache and over keys and values.  And their helpers on streams
of the caller's."""
import math

import numpy as np
import pytest
import torch

import draft_sampling_verification_gb300 as ds
from test_gpu_helper_streams import check_dropped_outputs

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def rand(g, *s):
    return torch.randn(*s, generator=g, device="cuda")


def turned(x, positions, freq, interleaved):
    """[n, heads, rot] float64, every pair turned."""
    angle = positions.double()[:, None, None] * freq
    c, s = angle.cos(), angle.sin()
    half = x.shape[-1] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :half], x[..., half:])
    y = (a * c - b * s, b * c + a * s)
    return torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)


def freqs(rot, base):
    return base ** (-2 * torch.arange(rot // 2, device="cuda").double() / rot)


class Text:
    """What the requests' tokens are, by position: rows that the plain side attends over."""

    def __init__(self, B):
        self.rows = [[] for _ in range(B)]


def plan_of(lens, new, T, table, free, page, parents):
    p = ds.cache_plan(i32(lens), i32(new), T, page, table, free, parents=parents)
    assert (p["status"] == 0).all()
    return p


@pytest.mark.parametrize("interleaved", [False, True])
def test_latent_steps(interleaved):
    g = torch.Generator(device="cuda").manual_seed(3)
    B, T, H, L, R, page = 3, 5, 4, 128, 32, 8
    table = torch.full((B, 12), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(40, generator=g, device="cuda").to(torch.int32)
    cache = torch.full((40, page, L + R), math.nan, dtype=torch.bfloat16, device="cuda")
    rope, freq = ds.rope_table(R, base=1e4), freqs(R, 1e4)
    w = 1 + 0.1 * rand(g, L)
    parents = i32([[-1, 0, 0, 1, 2]] * B)
    parent = [-1, 0, 0, 1, 2]
    lens, kept = [0] * B, [torch.zeros(0, L + R, device="cuda").double() for _ in range(B)]
    scale = (64 + R) ** -0.5

    def plain_rows(x, positions):
        c, r = x[:, :L].double(), x[:, L:].double()
        c = c / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-6) * w.double()
        return torch.cat([c, turned(r[:, None], positions, freq, interleaved)[:, 0]], -1)

    # prompts of different lengths
    prompt = [11, 1, 20]
    p = plan_of(lens, prompt, 20, table, free, page, None)
    x = rand(g, B * 20, L + R)
    ds.latent_write(x[:, :L], x[:, L:], p["positions"].view(-1), rope, cache, p["slots"].view(-1),
                    weight=w, interleaved=interleaved)
    free = free[int(p["taken"]):].contiguous()
    for b in range(B):
        at = torch.arange(prompt[b], device="cuda")
        kept[b] = plain_rows(x[b * 20:b * 20 + prompt[b]], at)
    lens = prompt
    for step in range(3):
        p = plan_of(lens, [T] * B, T, table, free, page, parents)
        x, q = rand(g, B * T, L + R), 1.5 * rand(g, B, T, H, L + R).bfloat16()
        at = p["positions"].view(-1)
        ds.latent_write(x[:, :L], x[:, L:], at, rope, cache, p["slots"].view(-1), weight=w,
                        interleaved=interleaved)
        want_q = torch.cat([q[..., :L].double(), turned(
            q[..., L:].double().view(B * T, H, R), at, freq, interleaved).view(B, T, H, R)], -1)
        part = q[..., L:]
        ds.qk_rotate(part, None, at, rope, interleaved=interleaved, out=(part, None))
        out, lse, status = ds.latent_attention(q, cache, table, i32(lens), i32([T] * B), L, scale,
                                               tree_mask=p["tree_mask"])
        assert (status == 0).all()
        nodes = [plain_rows(x[b * T:(b + 1) * T], at[b * T:(b + 1) * T]) for b in range(B)]
        for b in range(B):
            for t in range(T):
                see = [t]
                while parent[see[-1]] >= 0:
                    see.append(parent[see[-1]])
                assert int(at[b * T + t]) == lens[b] + len(see) - 1
                rows = torch.cat([kept[b], nodes[b][sorted(see)]])
                s = want_q[b, t] @ rows.T * scale
                want = s.softmax(-1) @ rows[:, :L]
                # rows, rotated queries, weights and the result each rounded to bf16: the scores
                # are off by 2^-7 of sum |q k| scale, which moves a weight by as much
                reach = (want_q[b, t].abs() @ rows.abs().T * scale).amax(-1, keepdim=True)
                mean = s.softmax(-1) @ rows[:, :L].abs()
                tol = 2.0 ** -8 * (2 * mean + want.abs()) + 2 * 2.0 ** -7 * reach * mean
                assert ((out[b, t].double() - want).abs() <= tol).all()
                assert ((lse[b, t].double() - s.logsumexp(-1)).abs() <= 2.0 ** -7 * reach[:, 0]).all()
        # the path 0, 2, 4 is kept in one request, 0 in the others: written again behind the text
        path = [[0, 2, 4], [0], [0]]
        n = [len(r) for r in path]
        p = plan_of(lens, n, 3, table, free, page, None)
        rows = i32([[b * T + r[i] if i < len(r) else -1 for i in range(3)]
                    for b, r in enumerate(path)])
        ds.latent_write(x[:, :L], x[:, L:], p["positions"].view(-1), rope, cache,
                        p["slots"].view(-1), rows=rows.view(-1), weight=w, interleaved=interleaved)
        free = free[int(p["taken"]):].contiguous()
        for b in range(B):
            kept[b] = torch.cat([kept[b], nodes[b][path[b]]])
        lens = [a + b for a, b in zip(lens, n)]


def test_keys_and_values_steps():
    """rotate_write and tree_attention against the same with qk_rotate and kv_write, and against
    attention on turned keys: what a token's place is changes nothing but its angle."""
    g = torch.Generator(device="cuda").manual_seed(4)
    B, T, Hq, Hk, D, page = 2, 6, 8, 2, 64, 16
    rope, freq = ds.rope_table(D, base=1e4), freqs(D, 1e4)
    w = 1 + 0.1 * rand(g, D)
    table = torch.full((B, 8), -1, dtype=torch.int32, device="cuda")
    free = i32(range(16))
    kc, vc = (torch.zeros(16, page, Hk, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lens, new = [0, 0], [40, 23]
    p = plan_of(lens, new, 40, table, free, page, None)
    x = rand(g, B * 40, Hq + 2 * Hk, D)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
    at, slots = p["positions"].view(-1), p["slots"].view(-1)
    out, _, _ = ds.rotate_write(q, k, v, at, rope, kc, vc, slots, q_weight=w, k_weight=w)
    k2, v2 = torch.zeros_like(kc), torch.zeros_like(vc)
    qr, kr = (torch.empty(t.shape, dtype=torch.bfloat16, device="cuda") for t in (q, k))
    ds.qk_rotate(q, k, at, rope, w, w, out=(qr, kr))
    ds.kv_write(kr, v.bfloat16(), k2, v2, slots)
    assert torch.equal(out, qr) and torch.equal(kc, k2) and torch.equal(vc, v2)
    # the prompts' last six tokens as nodes of a chain
    nodes = torch.stack([out[b * 40 + new[b] - T:b * 40 + new[b]] for b in range(B)])
    got, _, status = ds.tree_attention(nodes, kc, vc, table, i32([34, 17]), i32([T, T]))
    assert (status == 0).all()

    def norm(t):
        t = t.double()
        return t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) * w.double()

    for b in range(B):
        rows = slice(b * 40, b * 40 + new[b])
        places = torch.arange(new[b], device="cuda")
        kk = turned(norm(k[rows]), places, freq, False).repeat_interleave(Hq // Hk, 1)
        qq = turned(norm(q[rows]), places, freq, False)[-T:]
        vv = v[rows].double().repeat_interleave(Hq // Hk, 1)
        s = torch.einsum("thd,lhd->htl", qq, kk) * D ** -0.5
        s += torch.full((T, new[b]), -math.inf, device="cuda").double().triu(new[b] - T + 1)
        want = torch.einsum("htl,lhd->thd", s.softmax(-1), vv)
        mean = torch.einsum("htl,lhd->thd", s.softmax(-1), vv.abs())
        reach = torch.einsum("thd,lhd->htl", qq.abs(), kk.abs()).amax(-1).T[..., None] * D ** -0.5
        # as above: keys, queries, values, weights and the result rounded to bf16
        tol = 2.0 ** -8 * (2 * mean + want.abs()) + 2 * 2.0 ** -7 * reach * mean
        assert ((got[b].double() - want).abs() <= tol).all()


def test_graphs_of_one_workspace():
    """Two captured calls that share a workspace, replayed in turn and interleaved on one stream."""
    from test_gpu_latent_attention import Case
    a = Case([3000, 100], [4, 4], 4, heads=32, seed=1)
    b = Case([70, 2500], [4, 2], 4, heads=32, seed=2)
    want = [a.run(), b.run()]
    ws = torch.empty(a.workspace(), dtype=torch.uint8, device="cuda")
    outs, graphs, keep = [], [], []
    for c in (a, b):
        out = [torch.empty_like(t) for t in want[0]]
        d = c.device()
        keep.append(d)                                       # a graph reads the addresses it saw
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ds.dspark_latent_attention(*d[:5], c.latent, d[5], c.scale, *out, ws)
        outs.append(out)
        graphs.append(graph)
    for _ in range(5):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for out, w in zip(outs, want):
        assert all(torch.equal(x, y) for x, y in zip(out, w))


def test_two_calls_at_once():
    """Calls on two streams, each with its own workspace, whose CTAs share the device."""
    from test_gpu_latent_attention import Case
    a = Case([4000, 100, 900], [4, 4, 1], 4, heads=32, seed=1)
    b = Case([70, 5000], [6, 2], 6, heads=20, latent=256, seed=2)
    want = [a.run(), b.run()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    args = [a.device(), b.device()]
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        for c, s, d in zip((a, b), streams, args):
            got.append(c.call(*d, stream=s))
    torch.cuda.synchronize()
    for i, r in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(r, want[i % 2]))


def test_dropped_outputs():
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, table = rand(g, 300, 8, 64), rand(g, 300, 2, 64), ds.rope_table(64)
    at = i32(range(300))
    check_dropped_outputs(lambda s: ds.qk_rotate(q, k, at, table, stream=s))
    kc = torch.zeros(40, 8, 2, 64, device="cuda", dtype=torch.bfloat16)
    vc = torch.zeros_like(kc)
    check_dropped_outputs(lambda s: ds.rotate_write(q, k, k, at, table, kc, vc, at, stream=s),
                          {kc.data_ptr(), vc.data_ptr()})
    x = rand(g, 4, 2, 8, 320).bfloat16()
    cache, blocks = rand(g, 20, 16, 320).bfloat16(), i32(range(20)).view(4, 5)
    check_dropped_outputs(lambda s: ds.latent_attention(x, cache, blocks, i32([60, 3, 0, 20]),
                                                        i32([2, 2, 1, 2]), 256, 0.1, stream=s))
