"""Single-token forms as views: a dimension of one element may have any
stride, which the calls must neither refuse nor take for the distance between
tokens or rows."""
import pytest
import torch

import draft_sampling_verification_gb300 as ds

pytestmark = pytest.mark.gpu


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def odd_strides(t, dims, stride=24):
    """t with another stride in its dimensions of one element."""
    st = list(t.stride())
    for d in dims:
        assert t.shape[d] == 1
        st[d] = stride
    return t.as_strided(t.shape, st, t.storage_offset())


@pytest.mark.parametrize("source", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("heads", [1, 2])
def test_write_of_one_token_a_request(source, heads):
    """k and v [B, 1, heads, dim] cut from a fused projection."""
    B, dim = 5, 64
    qkv = torch.randn(B, 3 * heads, dim, device="cuda").to(source)
    k, v = qkv[:, heads:2 * heads], qkv[:, 2 * heads:]
    slots = i32(3, 40, -1, 17, 0)
    caches = [torch.zeros(4, 16, heads, dim, dtype=torch.bfloat16, device="cuda") for _ in range(6)]
    ds.kv_write(k, v, *caches[:2], slots)
    ds.kv_write(k.unsqueeze(1), v.unsqueeze(1), *caches[2:4], slots)
    dims = [1] + ([2] if heads == 1 else [])
    ds.kv_write(odd_strides(k.unsqueeze(1), dims), v.unsqueeze(1), *caches[4:], slots)
    torch.cuda.synchronize()
    want = torch.zeros(64, heads, dim, dtype=torch.bfloat16, device="cuda")
    want[[3, 40, 17, 0]] = k[[0, 1, 3, 4]].to(torch.bfloat16)
    for c in caches[::2]:
        assert torch.equal(c.view(64, heads, dim), want)
    want[[3, 40, 17, 0]] = v[[0, 1, 3, 4]].to(torch.bfloat16)
    for c in caches[1::2]:
        assert torch.equal(c.view(64, heads, dim), want)


def test_write_of_one_token_in_all():
    k = torch.randn(1, 1, 2, 64, device="cuda").bfloat16()
    kc = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    ds.kv_write(odd_strides(k, [0, 1], 3), k, kc, vc, i32(5))
    torch.cuda.synchronize()
    assert torch.equal(kc[0, 5], k[0, 0]) and torch.equal(vc[0, 5], k[0, 0])


def test_tokens_not_uniformly_strided_are_refused():
    k = torch.zeros(4, 3, 2, 64, dtype=torch.bfloat16, device="cuda")[:, :2]
    kc = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        ds.kv_write(k, k, kc, kc, torch.zeros(8, dtype=torch.int32, device="cuda"))
    x = torch.zeros(4, 3, 50, device="cuda")
    with pytest.raises(ValueError):
        ds.logits_process(x[:, :2])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_logits_of_one_row_a_request(dtype):
    """The last row of each request's six, without a copy: in place, and out of place."""
    x = torch.randn(4, 6, 333, device="cuda").to(dtype)
    ids, values = i32(3, 9, 3, 9).view(4, 1), torch.full((4, 1), 2.5, device="cuda")
    kw = dict(bias_ids=ids, bias_values=values)
    want, _ = ds.logits_process(x[:, 5:].contiguous(), **kw)
    got, _ = ds.logits_process(x[:, 5:], **kw)
    assert torch.equal(got, want)
    odd, _ = ds.logits_process(odd_strides(x[:, 5:], [1], 7), **kw)
    assert torch.equal(odd, want)
    y = x.clone()
    part = y[:, 5:]
    ds.logits_process(part, out=part, **kw)
    torch.cuda.synchronize()
    assert torch.equal(part, want) and torch.equal(y[:, :5], x[:, :5])


def test_verification_and_q_of_views():
    """The same rows for the calls that take a whole batch's logits.  Probabilities at another
    alignment are sums in another order: each of the two sums within 333 2^-24 of its value."""
    x = torch.randn(4, 6, 333, device="cuda")
    a, b = ds.q_build(x[:, 5:].contiguous()), ds.q_build(x[:, 5:])
    p, q = ds.target_probs(x[:, 2:3].contiguous()), ds.target_probs(x[:, 2:3])
    torch.cuda.synchronize()
    assert torch.equal(a["counts"], b["counts"]) and torch.equal(p[1], q[1])
    assert ((p[0] - q[0]).abs() <= 2 * 333 * 2.0 ** -24 * p[0]).all()
