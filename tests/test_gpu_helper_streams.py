"""The allocating helpers on a stream of the caller's: their outputs belong
to that stream's memory.  An output that is dropped while the stream still
works must not come back as another tensor of the current stream that the
late kernel then writes over."""
import numpy as np
import pytest
import torch

import draft_sampling_verification_gb300 as ds

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def tensors(x):
    if isinstance(x, torch.Tensor):
        return [x]
    if isinstance(x, dict):
        x = x.values()
    return [t for y in x for t in tensors(y)] if isinstance(x, (tuple, list, type({}.values()))) \
        else []


def check_dropped_outputs(call, keep=()):
    """call(stream) -> outputs; keep: the data pointers of what the caller owns."""
    call(None)                                   # the kernel is loaded: no wait at its launch
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(60_000_000)            # some tens of ms: the call's kernels come late
    outs = [t for t in tensors(call(s)) if t.data_ptr() not in keep]
    assert outs
    sizes = [(t.shape, t.dtype) for t in outs]
    del outs
    mine = [torch.full(shape, 77, dtype=dtype, device="cuda") for shape, dtype in sizes]
    torch.cuda.synchronize()
    for t in mine:
        assert (t == 77).all()


def test_logits_process():
    x = torch.randn(3, 2, 5000, device="cuda")
    check_dropped_outputs(lambda s: ds.logits_process(x, stream=s))


def test_logits_process_status_alone():
    x = torch.randn(3, 2, 5000, device="cuda")
    y = torch.empty_like(x)
    check_dropped_outputs(lambda s: ds.logits_process(x, out=y, stream=s), {y.data_ptr()})


@pytest.mark.parametrize("max_new", [6, 100])
def test_cache_plan(max_new):
    table = torch.full((300, 40), -1, dtype=torch.int32, device="cuda")
    ctx, new, free = i32([0] * 300), i32([max_new] * 300), i32(range(9000))
    check_dropped_outputs(lambda s: ds.cache_plan(ctx, new, max_new, 16, table, free, stream=s),
                          {table.data_ptr()})


def test_tree_attention():
    k = torch.randn(8, 16, 2, 64, device="cuda").bfloat16()
    q = torch.randn(3, 6, 4, 64, device="cuda").bfloat16()
    table = i32([[0, 1], [2, 3], [4, 5]])
    ctx, nodes = i32([7, 20, 0]), i32([6, 6, 6])
    check_dropped_outputs(lambda s: ds.tree_attention(q, k, k, table, ctx, nodes, stream=s))


@pytest.mark.parametrize("top_k", [0, 16])
def test_q_and_verification(top_k):
    B, depth, V = 3, 2, 5000
    x, y = torch.randn(B * depth, V, device="cuda"), torch.randn(B * (depth + 1), V, device="cuda")
    q = ds.q_build(x, top_k=top_k)
    drafts, _ = ds.draft_sample(q, B, depth, V, 5)
    for call in (lambda s: ds.q_build(x, None, top_k, s),
                 lambda s: ds.q_build_sample(x, B, depth, 5, top_k=top_k, stream=s),
                 lambda s: ds.q_build_sample_sharded(x, B, depth, 2, 5, top_k=top_k, stream=s),
                 lambda s: ds.draft_sample(q, B, depth, V, 5, None, s),
                 lambda s: ds.verify_greedy(y, drafts, s),
                 lambda s: ds.verify_ratio(y, drafts, q, 5, stream=s),
                 lambda s: ds.verify_match(y, drafts, 5, stream=s),
                 lambda s: ds.target_probs(y, stream=s),
                 lambda s: ds.q_pack(q, V, s)):
        check_dropped_outputs(call)


def test_whole_step():
    B, depth, V = 3, 2, 5000
    x, y = torch.randn(B * depth, V, device="cuda"), torch.randn(B * (depth + 1), V, device="cuda")
    anchors, flags = i32([1, 2, 3]), i32([1, 2, 4])
    q = ds.q_build(x)
    wire, _ = ds.q_pack(q, V)
    for call in (lambda s: ds.spec_step(x, y, B, depth, 5, stream=s),
                 lambda s: ds.q_chain_sample(x, B, depth, 5, anchors, stream=s),
                 lambda s: ds.q_validate(wire, V, stream=s),
                 lambda s: ds.verify_stats(flags, s)):
        check_dropped_outputs(call)
