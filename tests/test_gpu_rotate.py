"""dspark_qk_rotate, dspark_rotate_write and dspark_latent_write against
norms and rotations in 64 bits.

The bound on an element, with u the unit roundoff of its type (2^-24, bf16
2^-8, f16 2^-11) and e = 2^-24.  Norm: a sum of squares is off by at most 16 e
(each square 1, at most 2 x 7 additions in a lane and over lanes, its mean 1),
of which the root takes half, rsqrtf 4 e (2 units in the last place), the two
products 2 e: 14 e.  Turn: the angle, at most half a turn, is rounded to fp32
once (pi e), sincospif is off by 2 units in the last place of values below 1
(4 e), the magnitude 1 e; the pair's products and sum 2 e: 11 e.  So 32 e of
the terms' magnitudes is more than all of it, and then one rounding, u |y|
(f16 below its normal range: 2^-25)."""
import ctypes
import os

import numpy as np
import pytest
import torch

import draft_sampling_verification_gb300 as ds
import latent_ref as ref
from draft_sampling_verification_gb300 import _lib, build

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def rand(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


def near(got, want, size):
    u = U[got.dtype]
    tol = u * np.abs(want) + 32 * 2.0 ** -24 * size + (2.0 ** -25 if got.dtype is F16 else 0)
    err = np.abs(f64(got) - want)
    assert (err <= tol * (1 + u) + 1e-37).all(), float((err - tol).max())


def check_heads(got, x, w, positions, freq, start, interleaved, magnitude, eps=1e-6):
    n = positions.numel()
    want, size = ref.head(f64(x).reshape(n, *x.shape[-2:]), f64(w), eps,
                          positions.cpu().numpy().reshape(n), freq, start, interleaved, magnitude)
    near(got, want.reshape(got.shape), size.reshape(got.shape))


TYPES = [(F32, F32), (F32, BF16), (F32, F16), (BF16, BF16), (F16, F16)]


@pytest.mark.parametrize("src,dst", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot,start", [(64, 64, 0), (128, 128, 0), (256, 256, 0), (128, 32, 0),
                                           (128, 64, 64), (80, 16, 8), (96, 48, 48), (8, 8, 0),
                                           (24, 8, 16), (256, 8, 248), (200, 128, 40)])
def test_types_layouts_and_parts(src, dst, interleaved, dim, rot, start):
    n, Hq, Hk = 9, 6, 2
    q, k = rand(dim, n, Hq, dim).to(src), rand(rot, n, Hk, dim).to(src)
    qw, kw = 1 + 0.1 * rand(1, dim), 1 + 0.1 * rand(2, dim)
    positions = i32([0, 1, 2, 77, -1, 4095, 131071, 1000003, 5])
    how = dict(base=5e5, scaling="parts", factor=8.0, original_len=8192, low=1.0, high=4.0)
    table, freq = ds.rope_table(rot, **how), ref.frequencies(rot, **how)
    out = (torch.full((n, Hq, dim), 7.0, device="cuda", dtype=dst),
           torch.full((n, Hk, dim), 7.0, device="cuda", dtype=dst))
    got = ds.qk_rotate(q, k, positions, table, qw, kw, rot_start=start, interleaved=interleaved,
                       magnitude=1.25, out=out)
    assert got[0] is out[0] and got[1] is out[1]
    for o, x, w in ((out[0], q, qw), (out[1], k, kw)):
        check_heads(o, x, w, positions, freq, start, interleaved, 1.25)
        assert (o[4] == 0).all()


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (28, 4), (64, 1), (5, 5), (128, 128)])
@pytest.mark.parametrize("n", [1, 3, 4, 6, 131, 1000])
def test_head_counts_and_tokens(n, heads, kv_heads):
    q, k = rand(n, n, heads, 64).to(BF16), rand(heads, n, kv_heads, 64).to(BF16)
    positions = i32(np.arange(n) * 37 % 5000)
    table, freq = ds.rope_table(64), ref.frequencies(64)
    a, b = ds.qk_rotate(q, k, positions, table)
    check_heads(a, q, None, positions, freq, 0, False, 1.0)
    check_heads(b, k, None, positions, freq, 0, False, 1.0)


def test_one_side_norms_alone_and_one_norm():
    q, k, positions = rand(0, 5, 3, 128).to(F16), rand(1, 5, 2, 128).to(F16), i32([3, 1, -1, 0, 9])
    table, freq, w = ds.rope_table(128), ref.frequencies(128), 1 + 0.1 * rand(3, 128)
    a, none = ds.qk_rotate(q, None, positions, table)
    assert none is None
    check_heads(a, q, None, positions, freq, 0, False, 1.0)
    none, b = ds.qk_rotate(None, k, positions, table, k_weight=w, eps=0.5)
    assert none is None
    check_heads(b, k, w, positions, freq, 0, False, 1.0, 0.5)
    a, b = ds.qk_rotate(q, k, positions, None, q_weight=w, k_weight=w)   # no rotation
    check_heads(a, q, w, positions, np.zeros(0), 0, False, 1.0)
    check_heads(b, k, w, positions, np.zeros(0), 0, False, 1.0)
    a, b = ds.qk_rotate(q, k, positions, table, k_weight=w)
    check_heads(a, q, None, positions, freq, 0, False, 1.0)
    check_heads(b, k, w, positions, freq, 0, False, 1.0)
    empty = ds.qk_rotate(q[:0], k[:0], positions[:0], table)
    assert empty[0].shape == (0, 3, 128) and empty[1].shape == (0, 2, 128)


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_views_of_one_projection(interleaved):
    x = rand(5, 2, 7, 12, 96).to(BF16)
    kept = x.clone()
    positions, table = i32(np.arange(14).reshape(2, 7) * 1000), ds.rope_table(48)
    w = 1 + 0.1 * rand(6, 96)
    q, k = x[:, :, :8], x[:, :, 8:10]
    ds.qk_rotate(q, k, positions, table, w, w, rot_start=48, interleaved=interleaved, out=(q, k))
    freq = ref.frequencies(48)
    check_heads(x[:, :, :8], kept[:, :, :8], w, positions, freq, 48, interleaved, 1.0)
    check_heads(x[:, :, 8:10], kept[:, :, 8:10], w, positions, freq, 48, interleaved, 1.0)
    assert torch.equal(x[:, :, 10:], kept[:, :, 10:])          # the values' part
    # heads outermost, and a part of wider rows as the output
    y = rand(7, 6, 14, 64).to(BF16)
    wide = torch.full((14, 6, 160), 3.0, device="cuda", dtype=BF16)
    table = ds.rope_table(64)
    ds.qk_rotate(y.transpose(0, 1), None, positions, table, interleaved=interleaved,
                 out=(wide[:, :, 96:], None))
    check_heads(wide[:, :, 96:], y.transpose(0, 1), None, positions, ref.frequencies(64), 0,
                interleaved, 1.0)
    assert (wide[:, :, :96] == 3).all()


def test_far_positions():
    """The angle is the table's entry times the position modulo a turn, exactly: at 2^31 - 1 too."""
    far = [2 ** 31 - 1, 2 ** 30 + 7, 123456789, 2 ** 24 + 1]
    table = ds.rope_table(64, base=1e6)
    q = rand(8, 4, 2, 64)
    got = f64(ds.qk_rotate(q, None, i32(far), table)[0])
    x = f64(q)
    for t, p in enumerate(far):
        for i, turn in enumerate(table.tolist()):
            angle = (turn * p % 2 ** 64) / 2 ** 64 * 2 * np.pi
            a, b = x[t, :, i], x[t, :, i + 32]
            for at, want in ((i, a * np.cos(angle) - b * np.sin(angle)),
                             (i + 32, b * np.cos(angle) + a * np.sin(angle))):
                assert (np.abs(got[t, :, at] - want) <= 32 * 2.0 ** -24 *
                        (np.abs(a) + np.abs(b))).all()


def test_relative_positions():
    """Products of rotated queries and keys depend on the distance alone."""
    q, k, table = rand(1, 1, 1, 128), rand(2, 1, 1, 128), ds.rope_table(128, base=1e4)
    a, b = (ds.qk_rotate(x.expand(3, 1, 128).contiguous(), None, i32(p), table)[0].double()
            for x, p in ((q, [5, 1005, 100005]), (k, [0, 1000, 100000])))
    s = (a * b).sum(-1).flatten()
    # both rows of 128 elements off by 32 e of their terms
    bound = 4 * 32 * 2.0 ** -24 * 2 * float(a.abs().max() * b.abs().max()) * 128
    assert (s - s[0]).abs().max() <= bound


def test_padding_is_not_read():
    q = rand(3, 4, 2, 64).to(BF16)
    q[1] = float("nan")
    q[2] = float("inf")
    out = ds.qk_rotate(q, None, i32([4, -1, -2 ** 31, 7]), ds.rope_table(64),
                       q_weight=torch.ones(64, device="cuda"))[0]
    assert (out[1:3] == 0).all() and torch.isfinite(out).all()
    q = rand(3, 4, 2, 64).to(BF16)
    q[0, 1, 3] = float("inf")                                   # one head's own, and no other's
    out = ds.qk_rotate(q, None, i32([4, 5, 6, 7]), ds.rope_table(64, base=1e4))[0]
    bad = ~torch.isfinite(out)
    assert bad[0, 1, 3] and bad[0, 1, 35] and bad.sum() == 2
    zero = ds.qk_rotate(torch.zeros(1, 1, 64, device="cuda"), None, i32([9]), ds.rope_table(64),
                        q_weight=torch.ones(64, device="cuda"))[0]
    assert (zero == 0).all()


def caches(blocks, page, heads, dim, dtype, layout):
    store = (blocks, page, heads, dim) if layout == "nhd" else (blocks, heads, page, dim)
    k, v = (torch.full(store, f, device="cuda", dtype=dtype) for f in (5.0, 6.0))
    return (k, v) if layout == "nhd" else (k.transpose(1, 2), v.transpose(1, 2))


@pytest.mark.parametrize("src,dst", TYPES[1:])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("dim,rot,start,page", [(128, 128, 0, 16), (64, 32, 0, 24), (256, 64, 192, 8),
                                                (96, 96, 0, 7)])
def test_write(src, dst, layout, dim, rot, start, page):
    n, Hq, Hk, blocks = 29, 6, 2, 9
    x = rand(dim, n, Hq + 2 * Hk, dim).to(src)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
    kc, vc = caches(blocks, page, Hk, dim, dst, layout)
    positions = np.arange(n) * 3 + 100
    positions[[4, 11]] = -1
    slots = np.random.default_rng(0).permutation(blocks * page)[:n]
    slots[[7, 8, 9]] = [-1, blocks * page, 2 ** 31 - 1]
    w, table, freq = 1 + 0.1 * rand(1, dim), ds.rope_table(rot, base=5e5), \
        ref.frequencies(rot, base=5e5)
    out, kr, vr = ds.rotate_write(q, k, v, i32(positions), table, kc, vc, i32(slots), q_weight=w,
                                  k_weight=w, rot_start=start)
    assert kr is kc and vr is vc and out.dtype is dst
    check_heads(out, q, w, i32(positions), freq, start, False, 1.0)
    kept = (positions >= 0) & (slots >= 0) & (slots < blocks * page)
    want, size = ref.head(f64(k), f64(w), 1e-6, positions, freq, start, False, 1.0)
    at = torch.tensor(slots[kept], device="cuda")
    near(kc[at // page, at % page], want[kept], size[kept])
    assert torch.equal(vc[at // page, at % page], v[torch.tensor(kept, device="cuda")].to(dst))
    rest = torch.ones(blocks * page, dtype=torch.bool, device="cuda")
    rest[at] = False
    rest = torch.nonzero(rest)[:, 0]
    assert (kc[rest // page, rest % page] == 5).all() and (vc[rest // page, rest % page] == 6).all()


def test_write_by_rows():
    """A committed path: chosen source tokens to other positions and slots, without queries."""
    k, v = rand(0, 12, 2, 64).to(BF16), rand(1, 12, 2, 64).to(BF16)
    kc, vc = caches(4, 16, 2, 64, BF16, "nhd")
    rows, slots, positions = [7, 0, 12, -1, 7, 3], [0, 20, 21, 22, 63, 5], [9, 8, 7, 6, 100000, -1]
    table, freq = ds.rope_table(64), ref.frequencies(64)
    out, _, _ = ds.rotate_write(None, k, v, i32(positions), table, kc, vc, i32(slots),
                                rows=i32(rows))
    assert out is None
    x = f64(k)[[7, 0, 7]]
    want, size = ref.head(x, None, 0, np.array([9, 8, 100000]), freq, 0, False, 1.0)
    flat_k, flat_v = kc.view(64, 2, 64), vc.view(64, 2, 64)
    near(flat_k[[0, 20, 63]], want, size)
    assert torch.equal(flat_v[[0, 20, 63]], v[[7, 0, 7]])
    left = [i for i in range(64) if i not in (0, 20, 63)]
    assert (flat_k[left] == 5).all() and (flat_v[left] == 6).all()


def test_write_is_kv_write_without_a_turn():
    """At position 0, without norms: the plain write, for every type it shares."""
    for src, dst in TYPES[1:]:
        k, v = rand(0, 33, 3, 128).to(src), rand(1, 33, 3, 128).to(src)
        slots = i32(np.random.default_rng(1).permutation(48)[:33])
        a, b = caches(3, 16, 3, 128, dst, "hnd"), caches(3, 16, 3, 128, dst, "hnd")
        ds.kv_write(k, v, *a, slots)
        ds.rotate_write(None, k, v, torch.zeros_like(slots), ds.rope_table(128), *b, slots)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("src,dst", TYPES[1:])
@pytest.mark.parametrize("latent,rope", [(512, 64), (256, 32), (64, 0), (320, 8), (448, 56)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_latent_write(src, dst, latent, rope, interleaved):
    n, blocks, page, W = 37, 4, 12, latent + rope
    x = rand(latent, n, W + 8).to(src)[:, :W]                  # tokens further apart than a row
    c, r = x[:, :latent], x[:, latent:] if rope else None
    cache = torch.full((blocks, page, W + 16), 5.0, device="cuda", dtype=dst)[:, :, 8:8 + W]
    positions = np.arange(n) * 911
    positions[3] = -1
    slots = np.random.default_rng(2).permutation(blocks * page)[:n]
    slots[[5, 6]] = [-7, blocks * page]
    w = 1 + 0.1 * rand(1, latent)
    table, freq = (ds.rope_table(rope), ref.frequencies(rope)) if rope else (None, np.zeros(0))
    got = ds.latent_write(c, r, i32(positions), table, cache, i32(slots), weight=w,
                          interleaved=interleaved, magnitude=0.75)
    assert got is cache
    kept = (positions >= 0) & (slots >= 0) & (slots < blocks * page)
    a = ref.head(f64(c)[:, None], f64(w), 1e-6, positions, np.zeros(0), 0, False, 1.0)
    b = ref.head(f64(x[:, latent:])[:, None], None, 0, positions, freq, 0, interleaved, 0.75)
    want, size = (np.concatenate([i, j], -1)[:, 0] for i, j in zip(a, b))
    at = torch.tensor(slots[kept], device="cuda")
    near(cache[at // page, at % page], want[kept], size[kept])
    rest = torch.ones(blocks * page, dtype=torch.bool, device="cuda")
    rest[at] = False
    rest = torch.nonzero(rest)[:, 0]
    assert (cache[rest // page, rest % page] == 5).all()
    whole = cache.as_strided((blocks, page, W + 16), cache.stride(), cache.storage_offset() - 8)
    assert (whole[:, :, :8] == 5).all() and (whole[:, :, 8 + W:] == 5).all()


def test_latent_write_by_rows_and_without_norm():
    c, r = rand(0, 5, 128).to(F16), rand(1, 5, 64).to(F16)
    cache = torch.zeros(2, 8, 192, device="cuda", dtype=F16)
    rows, slots, positions = [4, 4, 5, -1, 0], [3, 15, 1, 2, 0], [10, 20, 1, 1, 0]
    ds.latent_write(c, r, i32(positions), ds.rope_table(64), cache, i32(slots), rows=i32(rows))
    flat = cache.view(16, 192)
    assert torch.equal(flat[[3, 15, 0], :128], c[[4, 4, 0]]) and torch.equal(flat[0, 128:], r[0])
    want, size = ref.head(f64(r)[[4, 4], None], None, 0, np.array([10, 20]), ref.frequencies(64), 0,
                          False, 1.0)
    near(flat[[3, 15], 128:], want[:, 0], size[:, 0])
    assert (flat[[1, 2] + list(range(4, 15))] == 0).all()


def test_replay_streams_and_repeats():
    """The same bits from an eager call, another stream and a replayed graph with new inputs."""
    table, w = ds.rope_table(128), 1 + 0.1 * rand(0, 128)
    q, k, v = (rand(i, 6, h, 128).to(BF16) for i, h in ((1, 8), (2, 2), (3, 2)))
    kc, vc = caches(4, 16, 2, 128, BF16, "nhd")
    positions, slots = i32([3, 4, 5, 6, 7, 8]), i32([0, 9, 17, 33, 40, 63])
    call = lambda s=None: ds.rotate_write(q, k, v, positions, table, kc, vc, slots,  # noqa: E731
                                          q_weight=w, k_weight=w, stream=s)
    first = call()[0].clone()
    keys = kc.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = call(side)[0]
    side.synchronize()
    assert torch.equal(out, first) and torch.equal(kc, keys)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()[0]
    q.copy_(rand(9, 6, 8, 128))
    positions.add_(100)
    graph.replay()
    torch.cuda.synchronize()
    want = call()[0]
    assert torch.equal(out, want) and not torch.equal(out, first) and not torch.equal(kc, keys)


def test_the_binding_refuses():
    q, k, table = rand(0, 4, 2, 64), rand(1, 4, 2, 64), ds.rope_table(64)
    at = i32([0, 1, 2, 3])
    kc, vc = caches(2, 8, 2, 64, BF16, "nhd")
    for error, call in (
            (ValueError, lambda: ds.qk_rotate(None, None, at, table)),
            (ValueError, lambda: ds.qk_rotate(q, k, at[:3], table)),
            (ValueError, lambda: ds.qk_rotate(q, k[:3], at, table)),
            (ValueError, lambda: ds.qk_rotate(q, k.bfloat16(), at, table)),
            (ValueError, lambda: ds.qk_rotate(q.cpu(), k.cpu(), at, table)),
            (TypeError, lambda: ds.qk_rotate(q.double(), None, at, table)),
            (TypeError, lambda: ds.qk_rotate(q, k, at.long(), table)),
            (TypeError, lambda: ds.qk_rotate(q, k, at, table.int())),
            (ValueError, lambda: ds.qk_rotate(q, k, at, table.cpu())),
            (ValueError, lambda: ds.qk_rotate(q, k, at, table, q_weight=table[:8].float())),
            (RuntimeError, lambda: ds.qk_rotate(q, k, at, table, rot_start=8)),
            (RuntimeError, lambda: ds.qk_rotate(q, k, at, table, eps=-1.0)),
            (RuntimeError, lambda: ds.qk_rotate(q.bfloat16(), None, at, table, out=(q, None))),
            (ValueError, lambda: ds.qk_rotate(q, None, at, table,
                                              out=(q[:, :1].expand(4, 2, 64), None))),
            (ValueError, lambda: ds.qk_rotate(q.transpose(1, 2), None, at, table)),
            (TypeError, lambda: ds.rotate_write(q.half(), k.half(), k.half(), at, table, kc, vc, at)),
            (RuntimeError, lambda: ds.rotate_write(q, k, k, at, table, kc, vc, at, rows=at)),
            (ValueError, lambda: ds.rotate_write(q, k, k[:, :1], at, table, kc, vc, at)),
            (ValueError, lambda: ds.rotate_write(q, k, k, at, table, kc, vc, at[:3])),
            (ValueError, lambda: ds.rotate_write(q[:3], k, k, at, table, kc, vc, at))):
        with pytest.raises(error):
            call()
    cache, c, r = torch.zeros(2, 8, 192, device="cuda", dtype=BF16), rand(0, 4, 128), rand(1, 4, 64)
    for error, call in (
            (ValueError, lambda: ds.latent_write(c, r, at, None, cache, at)),
            (ValueError, lambda: ds.latent_write(c, r, at, table[:8], cache, at)),
            (ValueError, lambda: ds.latent_write(c, None, at, None, cache, at)),
            (ValueError, lambda: ds.latent_write(c, r[:3], at, table, cache, at)),
            (ValueError, lambda: ds.latent_write(c, r, at, table, cache, at[:2])),
            (TypeError, lambda: ds.latent_write(c.half(), r.half(), at, table, cache, at)),
            (TypeError, lambda: ds.latent_write(c, r, at, table, cache.float(), at)),
            (RuntimeError, lambda: ds.latent_write(c[:, :96], r, at, table, cache[..., :160], at))):
        with pytest.raises(error):
            call()


def test_under_checks():
    """The bounds-checked build: every checked index inside its bound."""
    if not os.path.exists(build.LIB_CHECKED):
        build.build(checked=True)
    saved, _lib._lib = _lib._lib, None
    try:
        lib = _lib.load(build.LIB_CHECKED)
        count = (ctypes.c_uint32 * 3)()
        assert lib.dspark_checked_status(count) == 0 and count[2] == 1
        for dim, rot, start in ((64, 64, 0), (256, 256, 0), (80, 16, 8), (8, 8, 0)):
            test_types_layouts_and_parts(F32, BF16, False, dim, rot, start)
            test_types_layouts_and_parts(F16, F16, True, dim, rot, start)
        test_write(BF16, BF16, "hnd", 96, 96, 0, 7)
        test_write_by_rows()
        test_latent_write(F32, F16, 512, 64, False)
        test_latent_write(BF16, BF16, 64, 0, True)
        torch.cuda.synchronize()
        assert lib.dspark_checked_status(count) == 0
        assert count[0] == 0, "site %d failed %d times" % (count[1], count[0])
    finally:
        _lib._lib = saved
