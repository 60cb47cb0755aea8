"""dspark_logits_process with ids that a request's bias list holds more than
once: each entry is an addition of its own, in list order and rounded to
fp32, so the result equals that of the same additions in numpy bit for bit."""
import numpy as np
import pytest
import torch

import draft_sampling_verification_gb300 as ds

pytestmark = pytest.mark.gpu


def by_steps(x, ids, values, n):
    y = x.copy()
    for b in range(x.shape[0]):
        for i in range(n[b]):
            if 0 <= ids[b, i] < x.shape[2]:
                y[b, :, ids[b, i]] = y[b, :, ids[b, i]] + values[b, i]   # fp32
    return y


def run(x, ids, values, n, dtype=torch.float32, **kw):
    out, status = ds.logits_process(
        torch.from_numpy(x).to(dtype).cuda(), bias_ids=torch.from_numpy(ids).cuda(),
        bias_values=torch.from_numpy(values).cuda(),
        n_bias=torch.from_numpy(np.asarray(n, np.int32)).cuda(), **kw)
    torch.cuda.synchronize()
    assert (status == 0).all()
    return out


def test_two_small_biases_on_a_large_logit():
    """2^24 + 1 rounds back to 2^24, twice; the biases' sum first would give 2^24 + 2."""
    x = np.full((1, 2, 40), 2.0 ** 24, np.float32)
    ids, values = np.array([[7, 7]], np.int32), np.ones((1, 2), np.float32)
    got = run(x, ids, values, [2]).cpu().numpy()
    assert np.array_equal(got, by_steps(x, ids, values, [2]))
    assert got[0, 0, 7] == 2.0 ** 24


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,entries", [(5, 64), (300, 900), (20011, 3000)])
def test_repeated_ids_in_list_order(V, entries, dtype):
    rng = np.random.default_rng(V)
    B = 3
    x = (rng.normal(0, 1, (B, 4, V)) * 10.0 ** rng.integers(-3, 4, (B, 4, V))).astype(np.float32)
    x = torch.from_numpy(x).to(dtype).float().numpy()
    ids = rng.integers(-2, min(V, entries // 3) + 2, (B, entries)).astype(np.int32)
    values = (rng.normal(0, 1, (B, entries)) * 10.0 ** rng.integers(-3, 4, (B, entries))).astype(
        np.float32)
    n = [entries, 0, entries - 5]
    want = torch.from_numpy(by_steps(x, ids, values, n)).to(dtype)
    for _ in range(3):
        assert torch.equal(run(x, ids, values, n, dtype).cpu(), want)


def test_repeated_ids_of_tokens_in_the_text():
    """Penalties first, then the biases in order; tokens with one entry and with none beside them."""
    x = np.full((1, 1, 64), 3.0, np.float32)
    ids = np.array([[9, 4, 9, 30, 9, 4]], np.int32)
    values = np.array([[2.0 ** 24, 1.0, 1.0, 0.25, -2.0 ** 24, 2.0 ** -30]], np.float32)
    history = torch.tensor([[9, 9, 5, 4]], dtype=torch.int32, device="cuda")
    one = torch.ones(1, device="cuda")
    got = run(x, ids, values, [6], history=history,
              history_len=torch.tensor([4], dtype=torch.int32, device="cuda"), frequency=one)
    y = x.copy()
    y[0, 0, 9], y[0, 0, 5], y[0, 0, 4] = 1.0, 2.0, 2.0
    assert np.array_equal(got.cpu().numpy(), by_steps(y, ids, values, [6]))
