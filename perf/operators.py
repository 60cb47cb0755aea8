"""The operators around a speculative step, measured: the plan of a paged
key/value cache, the write of new keys and values into it, attention of the
drafted nodes over it, and the processing of the logits that verification
reads.

A case is a dict of plain values; `prepare` makes its inputs on the GPU from
a seed, `run` is one call, `work` the bytes and operations the call cannot do
without, `exact` the operator's definition in 64 bits on the host.  With
`own` false `run` computes the plain form (elementary torch operations in 32
bits), with `own` true it calls the library.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
VOCAB = 129280  # the repository's vocabulary; its depth is 5 (6 rows a request)


# ------------------------------------------------------------------- cases
def listed():
    att = dict(op="attention", depth=6, heads=32, kv_heads=8, dim=128, page=16, layout="nhd",
               dtype="bf16", tree=False)
    lg = dict(op="logits", rows=6, vocab=VOCAB, drafts=5, tree=False)
    return [
        # one user's chat a few hundred tokens in: the call's latency
        dict(att, name="attention_one", batch=1, lo=717, hi=717),
        # a serving batch at depth 5, short and long requests side by side
        dict(att, name="attention_batch", batch=64, lo=300, hi=8000),
        # two requests over long documents: few rows, a long axis
        dict(att, name="attention_long", batch=2, lo=120001, hi=131063, page=64, layout="hnd"),
        # wide draft trees, many query heads to a cached head: the matrix products count
        dict(att, name="attention_tree", batch=16, lo=2500, hi=8100, depth=64, heads=64, page=32,
             dtype="f16", tree=True),
        # one request's six target rows, short history, no grammar
        dict(lg, name="logits_one", batch=1, dtype="bf16", history=900, biases=0, masks=0,
             masked=0.0),
        # a batch with some structured outputs, single-precision logits
        dict(lg, name="logits_batch", batch=64, dtype="f32", history=4000, biases=40, masks=16,
             masked=0.5),
        # the largest batch, every row under a grammar
        dict(lg, name="logits_large", batch=256, dtype="bf16", history=2000, biases=8, masks=64,
             masked=1.0),
        # the plan of a batch's chains, one page added by some of the requests
        dict(op="plan", name="plan_chain", batch=256, new=6, page=16, lo=30, hi=8000, tree=False,
             prompt=False, short=0.0),
        # wide trees, with a free list that runs out before the last requests
        dict(op="plan", name="plan_tree", batch=1023, new=64, page=32, lo=1, hi=16000, tree=True,
             prompt=False, short=0.1),
        # admitting prompts: nothing cached yet, thousands of slots a request
        dict(op="plan", name="plan_prompts", batch=96, new=8192, page=16, lo=0, hi=0, tree=False,
             prompt=True, short=0.0),
        # the drafted tokens' keys and values of one layer
        dict(op="write", name="write_step", batch=64, new=6, kv_heads=8, dim=128, page=16,
             layout="nhd", dtype="bf16", source="bf16", skip=0.2),
        # a prompt pass of 64 thousand tokens, sources in single precision
        dict(op="write", name="write_prompts", batch=16, new=4096, kv_heads=8, dim=128, page=64,
             layout="hnd", dtype="bf16", source="f32", skip=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "logits", "logits", "plan", "write"])
    if op == "attention":
        c = dict(op=op, depth=_log(rng, 1, 64), kv_heads=rng.choice([1, 2, 4, 8, 16]),
                 dim=rng.choice([64, 128, 128, 256]), page=rng.choice([8, 16, 24, 32, 64, 128]),
                 layout=rng.choice(["nhd", "hnd"]), dtype=rng.choice(["bf16", "bf16", "f16"]))
        c["heads"] = c["kv_heads"] * rng.choice([1, 2, 4, 7, 8])
        c["tree"] = c["depth"] > 2 and rng.random() < 0.5
        c["hi"] = _log(rng, 16, 131072)
        c["lo"] = _log(rng, 1, c["hi"])
        # at most the largest listed case: a gigabyte of keys and values, 2.7e11 operations
        token = 4 * c["kv_heads"] * c["dim"]
        ops = 4 * c["depth"] * c["heads"] * c["dim"]
        most = min(1.0e9 / (token * c["hi"]), 2.0e11 / (ops * c["hi"]),
                   1.0e9 / (c["depth"] * c["heads"] * c["hi"]))
        c["batch"] = _log(rng, 1, max(1, min(128, most)))
        if most < 1:
            c["hi"] = max(16, int(c["hi"] * most))
            c["lo"] = min(c["lo"], c["hi"])
        return c
    if op == "logits":
        c = dict(op=op, vocab=rng.choice([_log(rng, 1000, 131072), 32000, 50257, VOCAB]),
                 dtype=rng.choice(["bf16", "f32"]), history=_log(rng, 1, 8000),
                 biases=rng.choice([0, 1, 30, 300]), masks=_log(rng, 1, 64),
                 masked=rng.choice([0.0, 0.5, 1.0]))
        c["drafts"] = rng.choice([0, 1, 3, 5, 7, 15])
        c["rows"] = c["drafts"] + 1
        c["tree"] = c["drafts"] > 3 and rng.random() < 0.5
        most = 1.9e8 / (c["vocab"] * c["rows"]) / (2 if c["dtype"] == "f32" else 1)
        c["batch"] = _log(rng, 1, max(1, min(512, most)))
        return c
    if op == "plan":
        prompt = rng.random() < 0.3
        hi = 0 if prompt else _log(rng, 10, 30000)
        new = _log(rng, 100, 8000) if prompt else _log(rng, 1, 64)
        return dict(op=op, batch=_log(rng, 1, 90 if prompt else 1000), new=new,
                    page=rng.choice([8, 16, 24, 32, 64, 128]), lo=0 if prompt else _log(rng, 1, hi),
                    hi=hi, tree=not prompt and new > 2 and rng.random() < 0.5, prompt=prompt,
                    short=rng.choice([0.0, 0.0, 0.2]))
    new = _log(rng, 1, 4096)
    c = dict(op=op, new=new, kv_heads=rng.choice([1, 2, 4, 8, 16]), dim=rng.choice([64, 128, 256]),
             page=rng.choice([8, 16, 24, 32, 64, 128]), layout=rng.choice(["nhd", "hnd"]),
             dtype=rng.choice(["bf16", "f16"]), skip=rng.choice([0.0, 0.2]))
    c["source"] = rng.choice([c["dtype"], "f32"])
    c["batch"] = _log(rng, 1, max(1, min(256, 6.0e7 / (new * c["kv_heads"] * c["dim"]))))
    return c


# -------------------------------------------------------- inputs of a case
def _lengths(n, lo, hi):
    """n lengths in [lo, hi], evenly spread over the logarithm, in a mixed order."""
    if n == 1 or lo >= hi:
        return [hi] * n
    at = [(i * 0.6180339887498949) % 1.0 for i in range(n)]
    order = sorted(range(n), key=lambda i: at[i])
    lens = [0] * n
    for rank, i in enumerate(order):
        lens[i] = round(max(lo, 1) * (hi / max(lo, 1)) ** (rank / (n - 1)))
    return lens


def _nodes(n, depth):
    """The requests' node counts: most draft to the full depth, some to less."""
    return [depth if i % 4 else max(1, depth - (i // 4) % depth) for i in range(n)]


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 17)
    return g


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _parents(B, T, g):
    """Random trees: node 0 is the root (the anchor), node i hangs below one of the eight before it."""
    i = torch.arange(T, device=DEV)
    back = 1 + (torch.rand(B, T, generator=g, device=DEV) * torch.clamp(i, 1, 8)).long()
    return (i - back).clamp(min=-1).where(i > 0, torch.full_like(back, -1)).to(torch.int32)


def _closure(parents):
    """[B, T, T] booleans: whether node j is node i or an ancestor of it."""
    T = parents.shape[1]
    step = (parents[:, :, None] == torch.arange(T, device=parents.device)) | torch.eye(
        T, dtype=torch.bool, device=parents.device)
    square = lambda m: (m.float() @ m.float()) > 0  # noqa: E731
    return square(square(square(square(square(square(step))))))


def _bits(seen):
    """[.., T] booleans as the bits of one int64."""
    return (seen.long() << torch.arange(seen.shape[-1], device=seen.device)).sum(-1)


def _cache(blocks, c, g=None):
    """The two caches [blocks, page, kv_heads, dim], stored by token or by head."""
    shape = (blocks, c["page"], c["kv_heads"], c["dim"])
    store = shape if c["layout"] == "nhd" else (shape[0], shape[2], shape[1], shape[3])
    make = lambda: (torch.zeros(store, dtype=TYPES[c["dtype"]], device=DEV) if g is None else  # noqa: E731
                    torch.randn(store, dtype=TYPES[c["dtype"]], generator=g, device=DEV))
    k, v = make(), make()
    return (k, v) if c["layout"] == "nhd" else (k.transpose(1, 2), v.transpose(1, 2))


def prepare(case, seed):
    g = _gen(seed)
    return {"attention": _prepare_attention, "logits": _prepare_logits, "plan": _prepare_plan,
            "write": _prepare_write}[case["op"]](case, g)


def _prepare_attention(c, g):
    B, T, page = c["batch"], c["depth"], c["page"]
    ctx, n = _lengths(B, c["lo"], c["hi"]), _nodes(B, T)
    pages = [-(-(a + b) // page) for a, b in zip(ctx, n)]
    blocks, wide = sum(pages) + 3, max(pages) + 1
    k, v = _cache(blocks, c, g)
    table = torch.full((B, wide), -1, dtype=torch.int32)
    order = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32).cpu()
    at = 0
    for b in range(B):
        table[b, :pages[b]] = order[at:at + pages[b]]
        at += pages[b]
    # queries of a trained model: scores a few units wide, so some keys stand out
    q = (2.5 * torch.randn(B, T, c["heads"], c["dim"], generator=g, device=DEV)).to(
        TYPES[c["dtype"]])
    mask = _bits(_closure(_parents(B, T, g))) if c["tree"] else None
    return {"op": "attention", "q": q, "k": k, "v": v, "table": table.to(DEV), "ctx": _ints(ctx),
            "nodes": _ints(n), "mask": mask}


def _prepare_logits(c, g):
    B, R, V, nd, H = c["batch"], c["rows"], c["vocab"], c["drafts"], c["history"]
    x = 3 * torch.randn(B, R, V, generator=g, device=DEV)
    rand = lambda *s: torch.rand(*s, generator=g, device=DEV)  # noqa: E731
    # texts repeat themselves: ids spread over the logarithm of the vocabulary
    ids = lambda *s: (float(V) ** rand(*s)).long().clamp(max=V) - 1  # noqa: E731
    history = ids(B, H).to(torch.int32)
    lens = _lengths(B, max(1, H // 4), H)
    drafts = ids(B, nd).to(torch.int32) if nd else None
    s = {"op": "logits", "x": x.to(TYPES[c["dtype"]]), "history": history, "lens": _ints(lens),
         "prompt": _ints([n // 2 for n in lens]), "drafts": drafts,
         "rows": _bits(_closure(_parents(B, R, g))[:, :, 1:]) if c["tree"] else None,
         "repetition": 1 + 0.3 * rand(B), "frequency": 0.5 * rand(B), "presence": rand(B),
         "bias_ids": None, "bias_values": None, "biases": None, "words": None, "which": None}
    if c["biases"]:
        n = min(c["biases"], V)
        first = (rand(B, 1) * V).long()
        s["bias_ids"] = ((first + 97 * torch.arange(n, device=DEV)) % V).to(torch.int32)
        s["bias_values"] = 4 * torch.randn(B, n, generator=g, device=DEV)
        s["biases"] = _ints(_lengths(B, max(1, n // 2), n))
    if c["masked"] > 0:
        # grammars let through a few tokens, or nearly all
        W = -(-V // 32)
        share = torch.where(rand(c["masks"], 1, 1) < 0.5, 0.02, 0.9)
        on = (rand(c["masks"], W, 32) < share).long() << torch.arange(32, device=DEV)
        on = on.sum(-1)
        s["words"] = torch.where(on >= 1 << 31, on - (1 << 32), on).to(torch.int32)
        which = (rand(B, R) * c["masks"]).long()
        s["which"] = torch.where(rand(B, 1) < c["masked"], which, -1).to(torch.int32)
    return s


def _prepare_plan(c, g):
    B, T, page = c["batch"], c["new"], c["page"]
    ctx = _lengths(B, c["lo"], c["hi"]) if c["hi"] else [0] * B
    new = _lengths(B, max(1, T // 8), T) if c["prompt"] else _nodes(B, T)
    held = [-(-a // page) for a in ctx]
    need = [-(-(a + b) // page) - h for a, b, h in zip(ctx, new, held)]
    wide = max(h + x for h, x in zip(held, need)) + 1
    free = max(1, int(sum(need) * (1 - c["short"])))
    blocks = sum(held) + max(free, sum(need)) + 64
    order = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
    j = torch.arange(wide, device=DEV)
    h = _ints(held).long()
    start = torch.cumsum(h, 0) - h
    table = torch.where(j < h[:, None], order[(start[:, None] + j).clamp(max=blocks - 1)], -1)
    left = order[sum(held):].contiguous()
    return {"op": "plan", "ctx": _ints(ctx), "new": _ints(new), "width": T, "page": page,
            "table": table.to(torch.int32).contiguous(), "free": left, "count": _ints([free]),
            "parents": _parents(B, T, g) if c["tree"] else None}


def _prepare_write(c, g):
    B, T, page = c["batch"], c["new"], c["page"]
    n = B * T
    blocks = -(-n // page) + 8
    kc, vc = _cache(blocks, c)
    t = lambda: torch.randn(n, c["kv_heads"], c["dim"], generator=g, device=DEV).to(  # noqa: E731
        TYPES[c["source"]])
    k, v = t(), t()
    order = torch.randperm(blocks, generator=g, device=DEV)
    i = torch.arange(n, device=DEV)
    slots = order[i // page] * page + i % page
    slots = torch.where(torch.rand(n, generator=g, device=DEV) < c["skip"], -1, slots)
    return {"op": "write", "k": k, "v": v, "kc": kc, "vc": vc, "slots": slots.to(torch.int32)}


# ------------------------------------------------------------------ a pass
def run(state):
    if own:
        import draft_sampling_verification_gb300 as ds
        s = state
        if s["op"] == "attention":
            return ds.tree_attention(s["q"], s["k"], s["v"], s["table"], s["ctx"], s["nodes"],
                                     tree_mask=s["mask"])
        if s["op"] == "logits":
            return ds.logits_process(s["x"], s["history"], s["prompt"], s["lens"],
                                     draft_tokens=s["drafts"], row_mask=s["rows"],
                                     repetition=s["repetition"], frequency=s["frequency"],
                                     presence=s["presence"], bias_ids=s["bias_ids"],
                                     bias_values=s["bias_values"], n_bias=s["biases"],
                                     mask_words=s["words"], mask_rows=s["which"])
        if s["op"] == "plan":
            return ds.cache_plan(s["ctx"], s["new"], s["width"], s["page"], s["table"], s["free"],
                                 s["count"], parents=s["parents"])
        return ds.kv_write(s["k"], s["v"], s["kc"], s["vc"], s["slots"])
    return {"attention": _plain_attention, "logits": _plain_logits, "plan": _plain_plan,
            "write": _plain_write}[state["op"]](state)


def _plain_attention(s):
    """(out, lse, status): softmax(q k^T / sqrt(dim)) v over the cached tokens and the nodes that the mask shows."""
    q, k, v, table = s["q"].float(), s["k"], s["v"], s["table"].long()
    B, T, Hq, D = q.shape
    blocks, page, Hk, _ = k.shape
    L = table.shape[1] * page
    ctx, n = s["ctx"].long(), s["nodes"].long()
    gather = lambda c: c[table.clamp(min=0)].reshape(B, L, Hk, D).float()  # noqa: E731
    pos = torch.arange(L, device=q.device)
    node = pos - ctx[:, None]                                           # [B, L]
    held = (table >= 0).repeat_interleave(page, 1) & (node < n[:, None])
    t = torch.arange(T, device=q.device)
    bits = s["mask"] if s["mask"] is not None else ((2 << t) - 1).expand(B, T)
    shown = (bits[:, :, None] >> node.clamp(0, 63)[:, None, :]) & 1     # [B, T, L]
    seen = held[:, None] & ((node < 0)[:, None] | (shown == 1)) & (t < n[:, None])[:, :, None]
    seen = seen[:, None, None]                                          # [B, 1, 1, T, L]
    qs = q.reshape(B, T, Hk, Hq // Hk, D).permute(0, 2, 3, 1, 4)        # [B, Hk, G, T, D]
    ks = gather(k).masked_fill(~held[:, :, None, None], 0).permute(0, 2, 3, 1)
    vs = gather(v).masked_fill(~held[:, :, None, None], 0).permute(0, 2, 1, 3)
    a = (qs.reshape(B, Hk, -1, D) @ ks).reshape(B, Hk, -1, T, L) / math.sqrt(D)
    a = a.masked_fill(~seen, -math.inf)
    m = a.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    a = torch.exp(a - m)
    z = a.sum(-1, keepdim=True)
    o = (a.reshape(B, Hk, -1, L) @ vs).reshape(B, Hk, -1, T, D) / torch.where(z == 0, 1.0, z)
    lse = (m + torch.log(z))[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, D)
    lse = lse.permute(0, 3, 1, 2).reshape(B, T, Hq)
    return o.to(s["q"].dtype), lse, torch.zeros_like(s["ctx"])


def _plain_logits(s):
    """(logits, status): repeated tokens' penalties, then biases, then the grammar's mask."""
    x = s["x"].float()
    B, R, V = x.shape
    at = torch.arange(s["history"].shape[1], device=x.device)
    ids = s["history"].long()
    fine = (ids >= 0) & (ids < V) & (at < s["lens"][:, None])
    early = at < s["prompt"][:, None]
    count = lambda on: torch.zeros(B, V + 1, device=x.device).scatter_add_(  # noqa: E731
        1, torch.where(on, ids, V), torch.ones_like(ids, dtype=torch.float32))[:, None, :V]
    prompt, said = count(fine & early), count(fine & ~early)
    if s["drafts"] is not None:
        nd = s["drafts"].shape[1]
        j = torch.arange(nd, device=x.device)
        bits = s["rows"] if s["rows"] is not None else (
            (1 << torch.arange(R, device=x.device)) - 1).expand(B, R)
        before = ((bits[:, :, None] >> j) & 1) == 1                     # [B, R, nd]
        d = s["drafts"].long()[:, None].expand(B, R, nd)
        said = said + torch.zeros(B, R, V + 1, device=x.device).scatter_add_(
            2, torch.where(before & (d >= 0) & (d < V), d, V),
            torch.ones(B, R, nd, device=x.device))[..., :V]
    per = lambda t: t[:, None, None]  # noqa: E731
    r = per(s["repetition"])
    x = torch.where((prompt + said) > 0, torch.where(x > 0, x / r, x * r), x)
    x = x - per(s["frequency"]) * said - per(s["presence"]) * (said > 0)
    if s["bias_ids"] is not None:
        on = torch.arange(s["bias_ids"].shape[1], device=x.device) < s["biases"][:, None]
        x = x + torch.zeros(B, V + 1, device=x.device).scatter_add_(
            1, torch.where(on, s["bias_ids"].long(), V), s["bias_values"])[:, None, :V]
    if s["words"] is not None:
        w = s["words"][s["which"].long().clamp(min=0)]                  # [B, R, W]
        on = ((w[..., None] >> torch.arange(32, device=x.device, dtype=torch.int32)) & 1) == 1
        on = on.reshape(B, R, -1)[..., :V] | (s["which"] < 0)[..., None]
        x = torch.where(on, x, -math.inf)
    return x.to(s["x"].dtype), torch.zeros(B, dtype=torch.int32, device=x.device)


def _plain_plan(s):
    ctx, new, page, T = s["ctx"].long(), s["new"].long(), s["page"], s["width"]
    table, free = s["table"].long(), s["free"].long()
    wide = table.shape[1]
    held, end = (ctx + page - 1) // page, (ctx + new + page - 1) // page
    fine = (ctx >= 0) & (new >= 0) & (new <= T) & (end <= wide)
    need = torch.where(fine, end - held, 0)
    upto = torch.cumsum(need, 0)
    given = fine & ((need == 0) | (upto <= s["count"]))
    j = torch.arange(wide, device=ctx.device) - held[:, None]
    fresh = given[:, None] & (j >= 0) & (j < need[:, None])
    at = ((upto - need)[:, None] + j).clamp(0, free.numel() - 1)
    table = torch.where(fresh, free[at], table)
    t = torch.arange(T, device=ctx.device)
    live = given[:, None] & (t < new[:, None])
    pos = ctx[:, None] + t
    block = torch.gather(table, 1, (pos // page).clamp(0, wide - 1))
    slots = torch.where(live & (block >= 0), block * page + pos % page, -1)
    out = {"block_table": table, "slots": slots,
           "taken": torch.where(given & (need > 0), upto, 0).amax(0, keepdim=True),
           "status": torch.where(fine, torch.where(given, 0, 10), 11)}
    if T <= 64:
        if s["parents"] is not None:
            seen = _closure(s["parents"])
        else:
            seen = (t[:, None] >= t).expand(ctx.shape[0], T, T)
        mask = torch.where(live, _bits(seen), 0)
        pos = ctx[:, None] + seen.sum(-1) - 1
        out["tree_mask"] = mask
    out["positions"] = torch.where(live, pos, -1)
    return {k: (t if k == "tree_mask" else t.to(torch.int32)) for k, t in out.items()}


def _plain_write(s):
    slots = s["slots"].long()
    on = slots >= 0
    page = s["kc"].shape[1]
    block, row = slots[on] // page, slots[on] % page
    s["kc"][block, row] = s["k"][on].to(s["kc"].dtype)
    s["vc"][block, row] = s["v"][on].to(s["vc"].dtype)
    return s["kc"], s["vc"]


# ------------------------------------------------------------ what it takes
def work(case):
    c, B = case, case["batch"]
    if c["op"] == "attention":
        e = SIZE[c["dtype"]]
        ctx, n = _lengths(B, c["lo"], c["hi"]), _nodes(B, c["depth"])
        tokens = sum(a + b for a, b in zip(ctx, n))
        rows = B * c["depth"] * c["heads"]
        pairs = sum(b * a + b * (b + 1) // 2 for a, b in zip(ctx, n))
        return {"bytes": 2 * tokens * c["kv_heads"] * c["dim"] * e + rows * (2 * c["dim"] * e + 4)
                + 4 * sum(-(-(a + b) // c["page"]) for a, b in zip(ctx, n)),
                "flops": 4 * pairs * c["heads"] * c["dim"]}
    if c["op"] == "logits":
        cells = B * c["rows"] * c["vocab"]
        lens = _lengths(B, max(1, c["history"] // 4), c["history"])
        masks = c["masks"] * (-(-c["vocab"] // 32)) * 4 if c["masked"] else 0
        return {"bytes": 2 * cells * SIZE[c["dtype"]] + 4 * sum(lens) + 8 * B * c["biases"]
                + masks, "flops": cells}
    if c["op"] == "plan":
        T, page = c["new"], c["page"]
        ctx = _lengths(B, c["lo"], c["hi"]) if c["hi"] else [0] * B
        new = _lengths(B, max(1, T // 8), T) if c["prompt"] else _nodes(B, T)
        blocks = sum(-(-(a + b) // page) - (-(-a // page)) for a, b in zip(ctx, new))
        cells = B * T
        return {"bytes": 12 * B + 8 * blocks + 8 * cells + (8 * cells if T <= 64 else 0)
                + (4 * cells if c["tree"] else 0), "flops": 4 * cells}
    cells = 2 * B * c["new"] * c["kv_heads"] * c["dim"] * (1 - c["skip"])
    return {"bytes": cells * (SIZE[c["source"]] + SIZE[c["dtype"]]) + 4 * B * c["new"],
            "flops": cells}


# ------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attention":
        return _exact_attention(s)
    if case["op"] == "logits":
        return _exact_logits(s)
    if case["op"] == "write":
        return _exact_write(s)
    return None  # whole numbers only


def _host(t):
    return None if t is None else t.cpu().numpy()


def _exact_attention(s):
    q, table = s["q"].double().cpu().numpy(), _host(s["table"])
    B, T, Hq, D = q.shape
    page, Hk = s["k"].shape[1], s["k"].shape[2]
    G = Hq // Hk
    out = np.zeros((B, T, Hq, D))
    lse = np.full((B, T, Hq), -np.inf)
    for b in range(B):
        ctx, n = int(s["ctx"][b]), int(s["nodes"][b])
        rows = s["table"][b, :-(-(ctx + n) // page)].long()
        keys, vals = (c[rows].transpose(0, 2).transpose(1, 2).reshape(Hk, -1, D)[:, :ctx + n]
                      .double().cpu().numpy() for c in (s["k"], s["v"]))
        seen = np.ones((n, ctx + n), dtype=bool)
        for i in range(n):
            word = (2 << i) - 1 if s["mask"] is None else int(s["mask"][b, i])
            seen[i, ctx:] = [(word >> j) & 1 for j in range(n)]
        for h in range(Hk):
            qh = q[b, :n, h * G:(h + 1) * G].reshape(n * G, D)
            a = qh @ keys[h].T
            a *= D ** -0.5
            a = np.where(np.repeat(seen, G, 0), a, -np.inf)
            m = a.max(1, keepdims=True)
            a -= m
            np.exp(a, out=a)
            z = a.sum(1, keepdims=True)
            out[b, :n, h * G:(h + 1) * G] = (a @ vals[h] / z).reshape(n, G, D)
            lse[b, :n, h * G:(h + 1) * G] = (m + np.log(z)).reshape(n, G)
    return out, lse, None


def _exact_logits(s):
    x = _host(s["x"].float())
    B, R, V = x.shape
    y = np.empty(x.shape)
    history, lens, prompt, drafts = (_host(s[k]) for k in ("history", "lens", "prompt", "drafts"))
    rep, freq, pres = (_host(s[k]).astype(np.float64) for k in
                       ("repetition", "frequency", "presence"))
    rows, words, which = _host(s["rows"]), _host(s["words"]), _host(s["which"])
    ids, values, biases = _host(s["bias_ids"]), _host(s["bias_values"]), _host(s["biases"])
    for b in range(B):
        asked = np.zeros(V, dtype=bool)
        asked[history[b, :prompt[b]]] = True
        told = np.bincount(history[b, prompt[b]:lens[b]], minlength=V)
        for r in range(R):
            z, c = x[b, r].astype(np.float64), told.copy()
            for j in range(0 if drafts is None else drafts.shape[1]):
                if (j < r) if rows is None else (int(rows[b, r]) >> j) & 1:
                    c[drafts[b, j]] += 1
            old = np.flatnonzero(asked | (c > 0))
            t = z[old]
            z[old] = np.where(t > 0, t / rep[b], t * rep[b]) - freq[b] * c[old] \
                - pres[b] * (c[old] > 0)
            if ids is not None:
                np.add.at(z, ids[b, :biases[b]], values[b, :biases[b]].astype(np.float64))
            if which is not None and which[b, r] >= 0:
                on = np.unpackbits(words[which[b, r]].astype("<i4").view(np.uint8),
                                   bitorder="little")[:V]
                z[on == 0] = -np.inf
            y[b, r] = z
    return y, None


def _exact_write(s):
    out = []
    slots = _host(s["slots"])
    for src, cache in ((s["k"], s["kc"]), (s["v"], s["vc"])):
        blocks, page, heads, dim = cache.shape
        x = np.zeros((blocks * page, heads, dim))
        x[slots[slots >= 0]] = src.double().cpu().numpy()[slots >= 0]
        out.append(x.reshape(blocks, page, heads, dim))
    return tuple(out)
