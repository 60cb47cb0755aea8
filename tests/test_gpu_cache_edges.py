"""The plan of an empty batch."""
import pytest
import torch

import draft_sampling_verification_gb300 as ds

pytestmark = pytest.mark.gpu


def test_plan_of_no_requests_takes_no_blocks():
    """An idle step: taken[0] is 0, not what its memory held before."""
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    table = torch.empty(0, 4, dtype=torch.int32, device="cuda")
    free = torch.arange(9, dtype=torch.int32, device="cuda")
    torch.cuda.empty_cache()
    del_me = [torch.full((1,), 7, dtype=torch.int32, device="cuda") for _ in range(64)]
    torch.cuda.synchronize()
    del del_me
    got = ds.cache_plan(none, none, 6, 16, table, free)
    torch.cuda.synchronize()
    assert got["taken"].tolist() == [0]
    assert got["slots"].shape == (0, 6) and got["status"].shape == (0,)


@pytest.mark.parametrize("other", [False, True])
def test_plan_of_no_requests_writes_taken(other):
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    cells = torch.empty(0, 6, dtype=torch.int32, device="cuda")
    table = torch.empty(0, 4, dtype=torch.int32, device="cuda")
    free = torch.arange(9, dtype=torch.int32, device="cuda")
    taken = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream() if other else torch.cuda.current_stream()
    s.wait_stream(torch.cuda.current_stream())
    ds.dspark_cache_plan(none, none, 6, 16, table, free, None, None, cells, None, None, taken,
                         none, s)
    torch.cuda.synchronize()
    assert taken.tolist() == [0]


def test_plan_of_the_most_requests():
    """2^20 requests of one token, a list that runs out near the end."""
    B, page = 1 << 20, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    ctx = torch.randint(0, 2 * page, (B,), generator=g, device="cuda", dtype=torch.int32)
    new = torch.ones_like(ctx)
    table = torch.arange(3 * B, dtype=torch.int32, device="cuda").view(B, 3)
    need = (ctx % page == 0).long()
    upto = need.cumsum(0)
    n = int(upto[-1]) - 1000
    free = torch.arange(3 * B, 3 * B + n, dtype=torch.int32, device="cuda")
    held = (ctx.long() + page - 1) // page
    entry = torch.gather(table, 1, (ctx.long() // page)[:, None])[:, 0].long()
    got = ds.cache_plan(ctx, new, 1, page, table, free)
    torch.cuda.synchronize()
    given = (need == 0) | (upto <= n)
    block = torch.where(need == 1, free[(upto - 1).clamp(0, n - 1)].long(), entry)
    slot = torch.where(given, block * page + ctx % page, -1)
    assert torch.equal(got["slots"][:, 0].long(), slot)
    assert torch.equal(got["status"], torch.where(given, 0, ds.ST_NO_BLOCKS).to(torch.int32))
    assert got["taken"].tolist() == [n]
    row = torch.arange(B, device="cuda")[(need == 1) & given]
    assert torch.equal(table[row, held[row]].long(), block[row])
