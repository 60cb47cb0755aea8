"""Rotation, latent write and latent attention at the ends of their ranges:
offsets past 32 bits in sources and caches, the largest batch and the most
rows, broadcast sources, in place for every type."""
import numpy as np
import pytest
import torch

import draft_sampling_verification_gb300 as ds
import latent_ref as ref
from test_gpu_latent_attention import Case
from test_gpu_rotate import BF16, F16, F32, check_heads, f64, i32, near, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place(dtype, interleaved):
    x = rand(1, 33, 10, 128).to(dtype)
    kept, w, table = x.clone(), 1 + 0.1 * rand(2, 128), ds.rope_table(64)
    positions = i32(np.arange(33) * 17 - 17)                    # the first is padding
    ds.qk_rotate(x[:, :8], x[:, 8:], positions, table, w, w, rot_start=32, interleaved=interleaved,
                 out=(x[:, :8], x[:, 8:]))
    check_heads(x, kept, w, positions, ref.frequencies(64), 32, interleaved, 1.0)
    assert (x[0] == 0).all()


def test_write_with_queries_in_place():
    x = rand(3, 21, 8, 64).to(BF16)
    kept, table = x.clone(), ds.rope_table(64)
    kc, vc = (torch.zeros(3, 8, 2, 64, device="cuda", dtype=BF16) for _ in range(2))
    at = i32(np.arange(21))
    out, _, _ = ds.rotate_write(x[:, :4], x[:, 4:6], x[:, 6:], at, table, kc, vc, at, out=x[:, :4])
    check_heads(out, kept[:, :4], None, at, ref.frequencies(64), 0, False, 1.0)
    check_heads(kc.view(24, 2, 64)[:21], kept[:, 4:6], None, at, ref.frequencies(64), 0, False, 1.0)
    assert torch.equal(vc.view(24, 2, 64)[:21], kept[:, 6:]) and torch.equal(x[:, 4:], kept[:, 4:])


def test_broadcast_sources():
    table, freq = ds.rope_table(64), ref.frequencies(64)
    one = rand(4, 7, 1, 64).to(BF16)
    q = one.expand(7, 5, 64)                                    # one head for all
    k = rand(5, 1, 2, 64).to(BF16).expand(7, 2, 64)             # one token for all
    positions = i32([5, 0, 3, 1000, -1, 7, 2])
    a, b = ds.qk_rotate(q, k, positions, table)
    check_heads(a, q, None, positions, freq, 0, False, 1.0)
    check_heads(b, k, None, positions, freq, 0, False, 1.0)


def test_far_sources():
    """Tokens 2^30 elements apart: the last begins past 2^32 elements and 2^33 bytes."""
    big = torch.empty(4 * 2 ** 30 + 4096, dtype=BF16, device="cuda")
    x = big.as_strided((5, 6, 64), (2 ** 30, 64, 1))
    x.copy_(rand(6, 5, 6, 64))
    table, freq, at = ds.rope_table(64), ref.frequencies(64), i32([1, 2, 3, 4, 50000])
    kc, vc = (torch.zeros(1, 8, 2, 64, device="cuda", dtype=BF16) for _ in range(2))
    out, _, _ = ds.rotate_write(x[:, :2], x[:, 2:4], x[:, 4:], at, table, kc, vc, i32(range(5)))
    check_heads(out, x[:, :2], None, at, freq, 0, False, 1.0)
    check_heads(kc[0, :5], x[:, 2:4], None, at, freq, 0, False, 1.0)
    assert torch.equal(vc[0, :5], x[:, 4:])
    ds.qk_rotate(x[:, :2], None, at, table, out=(x[:, :2], None))          # far outputs
    assert torch.equal(x[:, :2], out)
    cache = torch.zeros(1, 8, 128, device="cuda", dtype=BF16)
    c = big.as_strided((5, 64), (2 ** 30, 1), 128)
    ds.latent_write(c, x[:, 5], at, table, cache, i32([4, 3, 2, 1, 0]))
    assert torch.equal(cache[0, [4, 3, 2, 1, 0], :64], c)
    y, size = ref.head(f64(x[:, 5:]), None, 0, at.cpu().numpy(), freq, 0, False, 1.0)
    near(cache[0, [4, 3, 2, 1, 0], 64:], y[:, 0], size[:, 0])


def test_far_slots():
    """Blocks whose first element lies beyond 2^32 in the cache."""
    blocks = 2 ** 32 // (16 * 2 * 64) + 40
    kc = torch.empty(blocks, 16, 2, 64, device="cuda", dtype=BF16)
    vc = torch.empty_like(kc)
    kc[-40:], vc[-40:] = 5, 6
    k, v = rand(0, 30, 2, 64).to(BF16), rand(1, 30, 2, 64).to(BF16)
    at = blocks * 16 - 1 - 7 * np.arange(30)
    ds.rotate_write(None, k, v, torch.zeros(30, dtype=torch.int32, device="cuda"),
                    ds.rope_table(64), kc, vc, i32(at))
    rows = torch.tensor(at, device="cuda")
    assert torch.equal(kc[rows // 16, rows % 16], k) and torch.equal(vc[rows // 16, rows % 16], v)
    assert int((kc[-40:] != 5).any(-1).sum()) <= 60
    cache = kc.view(-1, 16, 128)
    ds.latent_write(k.view(30, 128), None, torch.zeros(30, dtype=torch.int32, device="cuda"), None,
                    cache, i32(at - 1))
    rows = rows - 1
    assert torch.equal(cache[rows // 16, rows % 16], k.view(30, 128))


def test_the_largest_batch():
    """65,535 requests of seven kinds: items of one tile, which no range cuts."""
    c = Case([0, 1, 50, 100, 3, 0, 127], [1, 1, 1, 0, 1, 0, 1], 1, heads=3, latent=64, rope=8)
    want = c.run()
    c.check(want)
    q, cache, table, ctx, nodes, _ = c.device()
    of = torch.arange(65535, device="cuda") % 7
    got = c.call(q[of], cache, table[of].contiguous(), ctx[of].contiguous(), nodes[of].contiguous(),
                 None)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y[of]) for x, y in zip(got, want))
    with pytest.raises(RuntimeError):
        c.call(q[[0] * 65536], cache, table[[0] * 65536], ctx[[0] * 65536], nodes[[0] * 65536], None)


@pytest.mark.parametrize("latent", [512, 128])
def test_the_most_rows(latent):
    c = Case([700, 3], [64, 61], 64, heads=128, latent=latent, mask="tree", seed=latent)
    c.check(c.run())


def test_queries_far_apart():
    """Requests of the queries 2^31 elements apart, through their map and without one."""
    c = Case([300, 40], [2, 2], 2, heads=4)
    want = c.run()
    a = c.device()
    big = torch.empty(2 ** 31 + 2 * 4 * 576 * 2, dtype=BF16, device="cuda")
    for node in (4 * 576, 4 * 576 + 8):
        a[0] = big.as_strided((2, 2, 4, 576), (2 ** 31, node, 576, 1))
        a[0].copy_(c.q)
        got = c.call(*a)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_tensors_of_another_device_are_refused(monkeypatch):
    """The calls launch on the current device; stood in for by another device's number."""
    q, k, table, at = rand(0, 4, 2, 64).to(BF16), rand(1, 4, 1, 64).to(BF16), ds.rope_table(64), \
        i32([0, 1, 2, 3])
    kc, vc = (torch.zeros(1, 8, 1, 64, device="cuda", dtype=BF16) for _ in range(2))
    cache, c = torch.zeros(1, 8, 64, device="cuda", dtype=BF16), rand(2, 4, 64).to(BF16)
    one = i32([1])
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    for call in (lambda: ds.qk_rotate(q, k, at, table),
                 lambda: ds.qk_rotate(q, k, at, table, out=(q, k)),
                 lambda: ds.rotate_write(q, k, k, at, table, kc, vc, at),
                 lambda: ds.latent_write(c, None, at, None, cache, at),
                 lambda: ds.latent_attention(q[:1, None, :, :], cache, one[None], one, one, 64, 0.1)):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()
