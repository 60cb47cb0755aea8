"""dspark_cache_plan and dspark_kv_write: integers against a plain
implementation, cache contents bit for bit against the copied or once
rounded sources."""
import math

import numpy as np
import pytest
import torch

import draft_sampling_verification_gb300 as ds
import serving_ref as ref

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def plan_case(ctx, new, max_new, page, max_blocks, n_free, parents=None, seed=0, spare=0):
    rng = np.random.default_rng(seed)
    B = len(ctx)
    ids = rng.permutation(B * max_blocks + n_free + spare + 1)
    table = ids[:B * max_blocks].reshape(B, max_blocks).copy()
    free = ids[B * max_blocks:B * max_blocks + n_free + spare]
    want = ref.cache_plan(ctx, new, max_new, page, table.tolist(), free.tolist(), n_free, parents)
    dev = i32(table)
    got = ds.cache_plan(i32(ctx), i32(new), max_new, page, dev, i32(free),
                        i32([n_free]) if spare else None,
                        None if parents is None else i32(parents))
    torch.cuda.synchronize()
    assert got["status"].tolist() == want["status"]
    assert got["taken"].tolist() == [want["taken"]]
    assert got["block_table"] is dev and dev.tolist() == want["table"]
    assert got["slots"].tolist() == want["slots"]
    assert got["positions"].tolist() == want["positions"]
    if max_new <= 64:
        m = got["tree_mask"].cpu().numpy().view(np.uint64)
        assert m.tolist() == want["tree_mask"]
    return want


def trees(rng, B, T):
    return [[int(rng.integers(-1, t)) if t else -1 for t in range(T)] for _ in range(B)]


@pytest.mark.parametrize("B", [1, 2, 170, 171, 600])
@pytest.mark.parametrize("T", [1, 6, 64])
@pytest.mark.parametrize("page", [1, 16, 24])
def test_plan_of_chains_and_trees(B, T, page):
    rng = np.random.default_rng(B + T)
    ctx = rng.integers(0, 90, B).tolist()
    new = rng.integers(0, T + 1, B).tolist()
    blocks = -(-(90 + T) // page)
    for parents in (None, trees(rng, B, T)):
        w = plan_case(ctx, new, T, page, blocks, B * blocks, parents, seed=B)
        assert set(w["status"]) <= {0}


@pytest.mark.parametrize("B,T", [(1, 65), (3, 1023), (2, 1024), (5, 1025), (4, 5000)])
def test_plan_of_prompts(B, T):
    rng = np.random.default_rng(T)
    new = [T] + rng.integers(0, T + 1, B - 1).tolist()
    plan_case([0, 7, 16, 3, 0][:B], new, T, 16, T // 16 + 3, B * (T // 16 + 3))


@pytest.mark.parametrize("n_free", [0, 1, 5, 17, 18, 40])
@pytest.mark.parametrize("spare", [0, 9])
def test_plan_with_too_few_blocks(n_free, spare):
    """A refused request and every later one that needs blocks get none; those that need none go on."""
    ctx = [16, 3, 32, 0, 15, 31, 8, 40]
    new = [6, 6, 1, 40, 1, 2, 0, 30]
    plan_case(ctx, new, 40, 16, 6, n_free, spare=spare)


def test_plan_refuses_lengths_and_trees():
    ctx = [5, -1, 10, 10, 60, 2 ** 31 - 1, 0, 33]
    new = [6, 2, -3, 7, 6, 6, 0, 6]
    rng = np.random.default_rng(0)
    t = trees(rng, 8, 6)
    t[0][3], t[7][2] = 3, -2                     # not before its node; below -1
    t[6][1] = 5                                  # no live node: nothing to refuse
    w = plan_case(ctx, new, 6, 16, 4, 20, t)
    assert w["status"] == [12, 11, 11, 11, 11, 11, 0, 12]


def test_plan_many_groups_run_out():
    """The list ends in the middle of the batch, groups of requests after it."""
    B = 3000
    rng = np.random.default_rng(7)
    ctx, new = rng.integers(0, 64, B).tolist(), rng.integers(0, 7, B).tolist()
    for n_free in (0, 100, 337, 5000):
        plan_case(ctx, new, 6, 16, 5, n_free, spare=3)


def test_plan_negative_entries_and_repeat():
    """A released page gives no slot; a second call changes nothing."""
    table = i32([[4, -1, -1], [-1, 9, -1]])
    args = (i32([5, 20]), i32([3, 3]), 3, 16, table, i32([7, 8]))
    a = ds.cache_plan(*args)
    first = {k: v.clone() for k, v in a.items()}
    b = ds.cache_plan(*args)
    torch.cuda.synchronize()
    assert a["slots"].tolist() == [[69, 70, 71], [148, 149, 150]]
    for k in first:
        assert torch.equal(first[k], b[k])
    gone = ds.cache_plan(i32([5, 5]), i32([2, 2]), 2, 16, i32([[-3], [2 ** 31 - 1]]), i32([]))
    torch.cuda.synchronize()
    assert gone["slots"].tolist() == [[-1, -1], [-1, -1]]


def test_plan_binding_refuses():
    ok = [i32([5]), i32([3]), 3, 16, i32([[4, -1]]), i32([7])]

    def bad(exc, **kw):
        a = list(ok)
        for k, x in kw.items():
            a[int(k[1:])] = x
        with pytest.raises(exc):
            ds.cache_plan(*a)

    bad(TypeError, a0=ok[0].long())
    bad(ValueError, a1=i32([1, 2]))
    bad(ValueError, a4=ok[4].long())
    bad(RuntimeError, a3=0)
    bad(RuntimeError, a3=2048)
    bad(RuntimeError, a2=0)
    with pytest.raises(RuntimeError):            # masks and trees end at 64 nodes
        ds.cache_plan(ok[0], ok[1], 65, 16, ok[4], ok[5],
                      parents=torch.zeros(1, 65, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("source", ["same", "f32"])
@pytest.mark.parametrize("n,heads,dim,page,layout", [(1, 1, 8, 1, "nhd"), (7, 3, 64, 16, "nhd"),
                                                     (300, 8, 128, 16, "hnd"),
                                                     (33, 2, 256, 24, "hnd"),
                                                     (5000, 4, 128, 64, "nhd")])
def test_write(dtype, source, n, heads, dim, page, layout):
    g = torch.Generator(device="cuda").manual_seed(n)
    blocks = -(-n // page) + 3
    store = (blocks, page, heads, dim) if layout == "nhd" else (blocks, heads, page, dim)
    kc, vc = (torch.randn(store, generator=g, device="cuda").to(dtype) for _ in range(2))
    if layout == "hnd":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    src = torch.float32 if source == "f32" else dtype
    qkv = torch.randn(n, 3 * heads, dim, generator=g, device="cuda").to(src)   # a fused projection
    k, v = qkv[:, heads:2 * heads], qkv[:, 2 * heads:]
    if n > 5:
        k[3, 0, :4] = torch.tensor([math.nan, math.inf, -0.0, 1e30])
    slots = torch.randperm(blocks * page, generator=g, device="cuda")[:n].to(torch.int32)
    if n > 5:
        slots[1], slots[2], slots[4] = -1, blocks * page, -2 ** 31
    wk, wv = kc.clone(), vc.clone()
    for i, s in enumerate(slots.tolist()):
        if 0 <= s < blocks * page:
            wk[s // page, s % page], wv[s // page, s % page] = k[i].to(dtype), v[i].to(dtype)
    got = ds.kv_write(k, v, kc, vc, slots)
    torch.cuda.synchronize()
    for a, b in zip(got, (wk, wv)):
        nan = torch.isnan(b)
        assert torch.equal(torch.isnan(a), nan)
        assert torch.equal(torch.where(nan, 0, a), torch.where(nan, 0, b))


def test_write_picks_source_rows():
    """A committed path written again to the positions that follow the text."""
    k = torch.randn(2, 6, 4, 64, device="cuda").to(torch.bfloat16)
    v = torch.randn(2, 6, 4, 64, device="cuda").to(torch.bfloat16)
    kc = torch.zeros(5, 16, 4, 64, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    ds.kv_write(k, v, kc, vc, i32([17, 18, 40, 3, 4, -1]), rows=i32([0, 3, 6, -1, 12, 7]))
    torch.cuda.synchronize()
    flat, rows = kc.view(80, 4, 64), {17: 0, 18: 3, 40: 6}
    for s in range(80):
        w = k.view(12, 4, 64)[rows[s]] if s in rows else torch.zeros_like(flat[s])
        assert torch.equal(flat[s], w)
        w = v.view(12, 4, 64)[rows[s]] if s in rows else torch.zeros_like(flat[s])
        assert torch.equal(vc.view(80, 4, 64)[s], w)


def test_write_far_slots_and_empty():
    """A slot whose row begins past 2^32 elements; no tokens at all."""
    blocks = 2 ** 32 // (16 * 8 * 128) + 2
    kc = torch.empty(blocks, 16, 8, 128, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    k = torch.randn(2, 8, 128, device="cuda")
    v = torch.randn(2, 8, 128, device="cuda")
    kc[0], vc[0] = 1, 2
    ds.kv_write(k, v, kc, vc, i32([blocks * 16 - 1, blocks * 16 - 9]))
    ds.kv_write(k[:0], v[:0], kc, vc, i32([]))
    torch.cuda.synchronize()
    assert torch.equal(kc[-1, 15], k[0].bfloat16()) and torch.equal(vc[-1, 7], v[1].bfloat16())
    assert (kc[0] == 1).all() and (vc[0] == 2).all()


def test_write_binding_refuses():
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    kc = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    s = i32([0, 1, 2])
    for a in ((k.half(), k.half(), kc, kc, s), (k, k.float(), kc, kc, s),
              (k, k, kc.float(), kc.float(), s), (k, k, kc, kc, s.long())):
        with pytest.raises(TypeError):
            ds.kv_write(*a)
    for a in ((k, k, kc, kc, s[:2]), (k[:, :1], k[:, :1], kc, kc, s),
              (k.transpose(1, 2), k.transpose(1, 2), kc, kc, s), (k, k, kc, kc[:3], s)):
        with pytest.raises(ValueError):
            ds.kv_write(*a)
    odd = torch.zeros(3 * 2 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(3, 2, 64)
    with pytest.raises(RuntimeError):            # not 16-byte aligned
        ds.kv_write(odd, odd, kc, kc, s)
