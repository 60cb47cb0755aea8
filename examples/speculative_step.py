"""Speculative decoding of a toy model through the library: a paged cache
planned and written on the GPU, tree attention over it, processed logits and
greedy verification.

    python examples/speculative_step.py

The model is one attention layer between an embedding and a vocabulary head,
with random weights; the drafter is a bigram table.  Each step drafts two
chains from the last committed token (a tree of 1 + 2 * depth nodes), runs
the target over all nodes at once, verifies both chains and commits the
longer.  The work between the library's calls (projections, the head, the
choice of a chain) is plain torch.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import draft_sampling_verification_gb300 as ds  # noqa: E402


class ToyModel:
    def __init__(self, V, heads=8, kv_heads=2, dim=64, max_tokens=4096, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        width = heads * dim
        self.V, self.heads, self.kv_heads, self.dim = V, heads, kv_heads, dim
        self.embed, self.place = w(V, width), 0.1 * w(max_tokens, width)
        self.mix = 0.6  # of the attention in what the head sees
        self.wq = w(width, width) * 2 / width ** 0.5
        self.wk = w(width, kv_heads * dim) / width ** 0.5
        self.wv = w(width, kv_heads * dim) / width ** 0.5
        self.head = w(width, V) / width ** 0.5

    def project(self, tokens, positions):
        """(x, q, k, v) of tokens [B, T] at their positions; padding (-1) gives anything."""
        x = self.embed[tokens.clamp(min=0)] + self.place[positions.clamp(min=0)]
        shape = tokens.shape
        q = (x @ self.wq).to(torch.bfloat16).view(*shape, self.heads, self.dim)
        k = (x @ self.wk).to(torch.bfloat16).view(*shape, self.kv_heads, self.dim)
        v = (x @ self.wv).to(torch.bfloat16).view(*shape, self.kv_heads, self.dim)
        return x, q, k, v

    def logits(self, x, attention):
        return (x + self.mix * attention.float().flatten(2)) @ self.head


class Cache:
    """The paged cache of B requests and the list of its free blocks, taken from the front."""

    def __init__(self, model, B, max_tokens, page=16):
        wide = -(-max_tokens // page)
        blocks = B * wide
        self.page = page
        self.k = torch.zeros(blocks, page, model.kv_heads, model.dim, dtype=torch.bfloat16,
                             device="cuda")
        self.v = torch.zeros_like(self.k)
        self.table = torch.full((B, wide), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(blocks, device="cuda").to(torch.int32)
        self.len = torch.zeros(B, dtype=torch.int32, device="cuda")

    def plan(self, new, width, parents=None, keep=True):
        """keep=False: the blocks granted stay on the list, for a pass whose tokens may be dropped."""
        plan = ds.cache_plan(self.len, new, width, self.page, self.table, self.free,
                             parents=parents)
        assert int(plan["status"].abs().sum()) == 0, plan["status"]
        if keep:
            self.free = self.free[int(plan["taken"]):].contiguous()
        return plan


def two_chains(bigram, anchors, depth):
    """Drafts [B, 2 * depth] and the parents [B, 1 + 2 * depth] of their tree: after the anchor
    the likeliest and the second likeliest next token, then the likeliest ones."""
    B = anchors.shape[0]
    first = bigram[anchors.long()].topk(2, dim=-1).indices               # [B, 2]
    chains = [first]
    for _ in range(depth - 1):
        chains.append(bigram[chains[-1]].argmax(-1))
    drafts = torch.stack(chains, -1).reshape(B, 2 * depth).to(torch.int32)
    up = [-1] + list(range(depth)) + [0] + list(range(depth + 1, 2 * depth))
    parents = torch.tensor(up, dtype=torch.int32, device="cuda").expand(B, -1).contiguous()
    return drafts, parents


def step(model, cache, bigram, text, lens, prompt, depth, processors):
    """One speculative step: commits 1 to depth + 1 tokens of each request into text [B, max] and
    lens [B].  The last committed token is not in the cache yet: it is the anchor."""
    B, T = text.shape[0], 1 + 2 * depth
    rows = torch.arange(B, device="cuda")
    anchors = text[rows, lens.long() - 1]
    drafts, parents = two_chains(bigram, anchors, depth)
    nodes = torch.cat([anchors[:, None], drafts], 1)                     # [B, T]
    count = torch.full((B,), T, dtype=torch.int32, device="cuda")

    # the target pass over the tree
    plan = cache.plan(count, T, parents, keep=False)
    x, q, k, v = model.project(nodes, plan["positions"])
    ds.kv_write(k, v, cache.k, cache.v, plan["slots"].view(-1))
    out, _, _ = ds.tree_attention(q, cache.k, cache.v, cache.table, cache.len, count,
                                  tree_mask=plan["tree_mask"])
    raw = model.logits(x, out)
    # node t follows the drafts that its tree shows: bit j of a row is draft j, node j + 1
    target, _ = ds.logits_process(raw, text, prompt, lens, draft_tokens=drafts,
                                  row_mask=plan["tree_mask"] >> 1, **processors)

    # both chains as requests of their own
    chain = torch.arange(depth, device="cuda") + torch.tensor([[1], [1 + depth]], device="cuda")
    path = torch.cat([torch.zeros_like(chain[:, :1]), chain], 1)         # [2, depth + 1] nodes
    accepted, committed, status = ds.verify_greedy(target[:, path].reshape(-1, model.V),
                                                   drafts.view(2 * B, depth))
    assert int(status.abs().sum()) == 0
    accepted, committed = accepted.view(B, 2), committed.view(B, 2, depth + 1)
    best = accepted.argmax(1)
    n = accepted[rows, best].to(torch.int32)                             # drafts kept

    # the kept nodes' keys and values go to the places behind the text; the rest is dropped with
    # the blocks that the tree was granted
    again = cache.plan(n + 1, depth + 1)
    source = (path[best] + rows[:, None] * T).to(torch.int32)
    ds.kv_write(k, v, cache.k, cache.v, again["slots"].view(-1), rows=source.view(-1))
    cache.len += n + 1
    at = lens[:, None] + torch.arange(depth + 1, device="cuda")
    new = committed[rows, best]
    keep = new >= 0
    text[rows[:, None].expand_as(at)[keep], at[keep].long()] = new[keep]
    lens += n + 1
    return raw, target, nodes, plan, n


def run(B=8, V=2003, prompt_tokens=40, steps=12, depth=4, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    model = ToyModel(V, seed=seed)
    most = prompt_tokens + steps * (depth + 1) + 1
    cache = Cache(model, B, most + 2 * depth + 1)
    # a drafter that knows the model a little: the head on the embedding alone, with noise
    bigram = model.embed @ model.head
    bigram += 0.1 * bigram.std() * torch.randn(V, V, generator=g, device="cuda")

    text = torch.full((B, most), -1, dtype=torch.int32, device="cuda")
    lens = torch.randint(2, prompt_tokens + 1, (B,), generator=g, device="cuda",
                         dtype=torch.int32)
    at = torch.arange(most, device="cuda")
    words = torch.randint(0, V, (B, most), generator=g, device="cuda", dtype=torch.int32)
    text = torch.where(at < lens[:, None], words, text)
    prompt = lens.clone()
    # the prompt up to its last token, the first anchor
    plan = cache.plan(lens - 1, prompt_tokens)
    _, _, k, v = model.project(text[:, :prompt_tokens], plan["positions"])
    ds.kv_write(k, v, cache.k, cache.v, plan["slots"].view(-1))
    cache.len += lens - 1

    # mild penalties, one favoured token, and a grammar that forbids every seventh
    allowed = torch.arange(32 * ((V + 31) // 32), device="cuda") % 7 != 3
    bits = (allowed.view(-1, 32).long() << torch.arange(32, device="cuda")).sum(-1)
    processors = dict(
        repetition=torch.full((B,), 1.1, device="cuda"),
        frequency=torch.full((B,), 0.2, device="cuda"),
        bias_ids=torch.full((B, 1), 5, dtype=torch.int32, device="cuda"),
        bias_values=torch.full((B, 1), 0.5, device="cuda"),
        mask_words=torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32)[None],
        mask_rows=torch.zeros(B, 1 + 2 * depth, dtype=torch.int32, device="cuda"))
    kept = []
    for _ in range(steps):
        kept.append(step(model, cache, bigram, text, lens, prompt, depth, processors)[-1])
    torch.cuda.synchronize()
    return model, cache, bigram, text, lens, prompt, processors, torch.stack(kept)


if __name__ == "__main__":
    *_, text, lens, prompt, _, kept = run()
    print("tokens a step: %.2f" % float(kept.float().mean() + 1))
    for b in range(3):
        print("request %d: ... %s" % (b, text[b, int(prompt[b]):int(lens[b])].tolist()))
