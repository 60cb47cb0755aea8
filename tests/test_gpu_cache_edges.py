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
