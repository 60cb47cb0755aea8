"""More operators around a speculative step, measured: the rotation of queries
and keys by their positions (with the norm of each head, and with the write
into the paged cache), the write of a latent cache, and attention of the
drafted nodes over a latent cache.

A case is a dict of plain values; `prepare` makes its inputs on the GPU from
a seed, `run` is one call, `work` the bytes and operations the call cannot do
without, `exact` the operator's definition in 64 bits.  With `own` false
`run` computes the plain form (elementary torch operations in 32 bits, angles
in 64), with `own` true it calls the library.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6


# ------------------------------------------------------------------- cases
def listed():
    # depth 5 drafts and the anchor: 6 rows a request, as in the repository's workloads
    ro = dict(op="rotate", new=6, heads=32, kv_heads=8, dim=128, rot=128, last=False,
              interleaved=False, norm=True, base=1e6, scaling="none", source="bf16", dtype="bf16",
              write=True, page=16)
    wr = dict(op="latent_write", new=6, latent=512, rope=64, page=64, norm=True, interleaved=True,
              base=1e4, scaling="parts", source="bf16", dtype="bf16", skip=0.2)
    la = dict(op="latent", depth=6, heads=16, latent=512, rope=64, page=64, dtype="bf16",
              tree=False)
    return [
        # one user's step: six nodes through norm, rotation and the cache write; latency
        dict(ro, name="rotate_one", batch=1, lo=717, hi=717),
        # a serving batch's step, one layer
        dict(ro, name="rotate_batch", batch=64, lo=300, hi=8000),
        # prompts far into long documents: single-precision projections, part of each head
        # rotated, interleaved pairs, frequencies scaled by parts
        dict(ro, name="rotate_prompt", batch=4, new=4096, lo=90000, hi=125000, rot=64,
             interleaved=True, source="f32", scaling="parts", page=64),
        # a cacheless pass of a model without head norms: an odd number of tokens, f16
        dict(ro, name="rotate_plain", batch=1, new=4099, lo=0, hi=0, heads=28, kv_heads=4, dim=64,
             rot=64, norm=False, base=1e4, scaling="linear", source="f16", dtype="f16",
             write=False),
        # the drafted tokens' latent rows of one layer
        dict(wr, name="latent_write_step", batch=64, lo=300, hi=8000),
        # a prompt pass of 64 thousand tokens, sources in single precision
        dict(wr, name="latent_write_prompts", batch=16, new=4096, lo=0, hi=0, source="f32",
             skip=0.0),
        # one user's single token a few hundred tokens in: the call's latency
        dict(la, name="latent_one", batch=1, lo=717, hi=717, depth=1),
        # a serving batch at depth 5 on a part of the heads, as one of several GPUs holds them
        dict(la, name="latent_batch", batch=64, lo=300, hi=8000),
        # plain decoding of a large batch, one token a request and all the heads
        dict(la, name="latent_decode", batch=256, lo=300, hi=8000, depth=1, heads=128),
        # two requests over long documents
        dict(la, name="latent_long", batch=2, lo=120001, hi=131063, heads=32),
        # draft trees: the matrix products count
        dict(la, name="latent_tree", batch=16, lo=2500, hi=8100, depth=24, heads=32, page=32,
             dtype="f16", tree=True),
        # a small model's latent vectors, an odd number of heads, odd blocks
        dict(la, name="latent_small", batch=32, lo=100, hi=2000, depth=4, heads=21, latent=256,
             rope=32, page=24),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "rotate", "latent_write", "latent", "latent", "latent"])
    c = dict(op=op, page=rng.choice([8, 16, 24, 32, 64, 128]))
    if op == "latent":
        c.update(depth=_log(rng, 1, 64) if rng.random() < 0.7 else 1,
                 heads=rng.choice([1, 8, 16, 16, 20, 32, 64, 128, _log(rng, 1, 128)]),
                 latent=rng.choice([512, 512, 512, 256, 384, 64]),
                 rope=rng.choice([64, 64, 32, 16, 0]), dtype=rng.choice(["bf16", "bf16", "f16"]))
        c["tree"] = c["depth"] > 2 and rng.random() < 0.5
        c["hi"] = _log(rng, 16, 131072)
        c["lo"] = _log(rng, 1, c["hi"])
        # at most the largest listed case: 0.7 GB of cache, 1.6e11 operations
        token = 2 * (c["latent"] + c["rope"])
        ops = c["depth"] * c["heads"] * (token + 2 * c["latent"])
        most = min(0.7e9 / (token * c["hi"]), 1.6e11 / (ops * c["hi"]),
                   2.5e8 / (c["depth"] * c["heads"] * c["hi"]))
        c["batch"] = _log(rng, 1, max(1, min(256, most)))
        if most < 1:
            c["hi"] = max(16, int(c["hi"] * most))
            c["lo"] = min(c["lo"], c["hi"])
        return c
    prompt = rng.random() < 0.4
    c["new"] = _log(rng, 64, 8192) if prompt else _log(rng, 1, 64)
    c["hi"] = 0 if rng.random() < 0.3 else _log(rng, 2, 130000)
    c["lo"] = _log(rng, 1, c["hi"]) if c["hi"] else 0
    c["interleaved"] = rng.random() < 0.5
    c["norm"] = rng.random() < 0.7
    c["base"] = rng.choice([1e4, 5e5, 1e6])
    c["scaling"] = rng.choice(["none", "none", "linear", "parts"])
    c["dtype"] = rng.choice(["bf16", "bf16", "f16"])
    c["source"] = rng.choice([c["dtype"], c["dtype"], "f32"])
    if op == "rotate":
        c["dim"] = rng.choice([64, 80, 96, 128, 128, 256])
        c["rot"] = rng.choice([r for r in (c["dim"], c["dim"], c["dim"] // 2, 64, 32, 16)
                               if r % 16 == 0 and r <= c["dim"]])
        c["last"] = rng.random() < 0.3
        c["kv_heads"] = rng.choice([1, 2, 4, 8, 16])
        c["heads"] = c["kv_heads"] * rng.choice([1, 2, 4, 7, 8])
        c["write"] = rng.random() < 0.6
        if not c["write"]:
            c["dtype"] = c["source"]
        row = (c["heads"] + 2 * c["kv_heads"]) * c["dim"]
    else:
        c["latent"] = rng.choice([512, 512, 256, 384, 64])
        c["rope"] = rng.choice([64, 64, 32, 16])
        c["skip"] = rng.choice([0.0, 0.2])
        row = 16 * (c["latent"] + c["rope"])  # at most a sixteenth of a wide model's heads
    most = 1.0e8 / (c["new"] * row)
    c["batch"] = _log(rng, 1, max(1, min(256, most)))
    if most < 1:
        c["new"] = max(1, int(c["new"] * most))
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
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 29)
    return g


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _scaling(c, rot):
    """The arguments of the table of a case, and its magnitude."""
    if c["scaling"] == "linear":
        return dict(scaling="linear", factor=4.0), 1.0
    if c["scaling"] == "parts":
        return dict(scaling="parts", factor=32.0, original_len=4096, low=1.0, high=32.0), \
            0.1 * math.log(32.0) + 1.0
    return {}, 1.0


def _frequencies(c, rot):
    """[rot / 2] radians a position, float64."""
    f = c["base"] ** (-2.0 * np.arange(rot // 2) / rot)
    args = _scaling(c, rot)[0]
    if c["scaling"] == "linear":
        f = f / args["factor"]
    if c["scaling"] == "parts":
        turns = args["original_len"] * f / (2 * math.pi)
        keep = np.clip((turns - args["low"]) / (args["high"] - args["low"]), 0.0, 1.0)
        f = f * (keep + (1 - keep) / args["factor"])
    return f


def _table(s, c, rot):
    """What a program keeps of the frequencies."""
    s["freq"] = torch.tensor(_frequencies(c, rot), device=DEV)
    s["magnitude"] = _scaling(c, rot)[1]
    if own:
        import draft_sampling_verification_gb300 as ds
        s["table"] = ds.rope_table(rot, base=c["base"], device=DEV, **_scaling(c, rot)[0])


def _places(c, g):
    """Positions [batch * new] (-1: padding) and slots, blocks in a random order."""
    B, T, page = c["batch"], c["new"], c["page"]
    n = B * T
    t = torch.arange(T, device=DEV)
    ctx = _ints(_lengths(B, c["lo"], c["hi"])) if c["hi"] else _ints([0] * B)
    live = t < _ints(_nodes(B, T))[:, None] if B > 1 else (t >= 0).expand(B, T)
    positions = torch.where(live, ctx[:, None] + t, -1).to(torch.int32).reshape(n)
    blocks = -(-n // page) + 8
    order = torch.randperm(blocks, generator=g, device=DEV)
    i = torch.arange(n, device=DEV)
    slots = torch.where(positions >= 0, order[i // page] * page + i % page, -1)
    return positions, slots.to(torch.int32), blocks


def prepare(case, seed):
    g = _gen(seed)
    return {"rotate": _prepare_rotate, "latent_write": _prepare_write,
            "latent": _prepare_latent}[case["op"]](case, g)


def _prepare_rotate(c, g):
    n, Hq, Hk, D = c["batch"] * c["new"], c["heads"], c["kv_heads"], c["dim"]
    positions, slots, blocks = _places(c, g)
    # one projection's output, of which queries, keys and values are views
    x = torch.randn(n, Hq + 2 * Hk, D, generator=g, device=DEV).to(TYPES[c["source"]])
    weight = lambda: 1 + 0.2 * torch.randn(D, generator=g, device=DEV)  # noqa: E731
    s = {"op": "rotate", "q": x[:, :Hq], "k": x[:, Hq:Hq + Hk], "v": x[:, Hq + Hk:],
         "positions": positions, "start": D - c["rot"] if c["last"] else 0, "rot": c["rot"],
         "interleaved": c["interleaved"], "qw": weight() if c["norm"] else None,
         "kw": weight() if c["norm"] else None, "kc": None, "dtype": TYPES[c["dtype"]]}
    if c["write"]:
        s["slots"] = slots
        s["kc"], s["vc"] = (torch.zeros(blocks, c["page"], Hk, D, dtype=s["dtype"], device=DEV)
                            for _ in range(2))
    _table(s, c, c["rot"])
    return s


def _prepare_write(c, g):
    n, L, R = c["batch"] * c["new"], c["latent"], c["rope"]
    positions, slots, blocks = _places(c, g)
    x = torch.randn(n, L + R, generator=g, device=DEV).to(TYPES[c["source"]])
    drop = torch.rand(n, generator=g, device=DEV) < c["skip"]
    s = {"op": "latent_write", "c": x[:, :L], "r": x[:, L:], "positions": positions,
         "slots": torch.where(drop, -1, slots), "interleaved": c["interleaved"],
         "w": 1 + 0.2 * torch.randn(L, generator=g, device=DEV) if c["norm"] else None,
         "cache": torch.zeros(blocks, c["page"], L + R, dtype=TYPES[c["dtype"]], device=DEV)}
    _table(s, c, R)
    return s


def _parents(B, T, g):
    """Random trees: node 0 is the root (the anchor), node i hangs below one of the eight before it."""
    i = torch.arange(T, device=DEV)
    back = 1 + (torch.rand(B, T, generator=g, device=DEV) * torch.clamp(i, 1, 8)).long()
    return (i - back).clamp(min=-1).where(i > 0, torch.full_like(back, -1)).to(torch.int32)


def _ancestors(parents):
    """[B, T] int64: bit j set where node j is the node or an ancestor of it."""
    B, T = parents.shape
    bits = torch.zeros(B, T, dtype=torch.int64, device=DEV)
    for t in range(T):
        p = parents[:, t:t + 1].long()
        above = torch.gather(bits, 1, p.clamp(min=0))[:, 0]
        bits[:, t] = (1 << t) | torch.where(p[:, 0] >= 0, above, 0)
    return bits


def _prepare_latent(c, g):
    B, T, page, W = c["batch"], c["depth"], c["page"], c["latent"] + c["rope"]
    ctx, n = _lengths(B, c["lo"], c["hi"]), _nodes(B, T)
    pages = [-(-(a + b) // page) for a, b in zip(ctx, n)]
    blocks, wide = sum(pages) + 3, max(pages) + 1
    cache = torch.randn(blocks, page, W, generator=g, device=DEV).to(TYPES[c["dtype"]])
    table = torch.full((B, wide), -1, dtype=torch.int32)
    order = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32).cpu()
    at = 0
    for b in range(B):
        table[b, :pages[b]] = order[at:at + pages[b]]
        at += pages[b]
    # queries of a trained model: scores a few units wide, so some keys stand out
    scale = (128 + c["rope"]) ** -0.5
    q = torch.randn(B, T, c["heads"], W, generator=g, device=DEV)
    q = (q * (2.5 / (scale * math.sqrt(W)))).to(TYPES[c["dtype"]])
    return {"op": "latent", "q": q, "cache": cache, "table": table.to(DEV), "ctx": _ints(ctx),
            "nodes": _ints(n), "mask": _ancestors(_parents(B, T, g)) if c["tree"] else None,
            "latent": c["latent"], "scale": scale}


# ------------------------------------------------------------------ a pass
def run(state):
    s = state
    if own:
        import draft_sampling_verification_gb300 as ds
        if s["op"] == "latent":
            return ds.latent_attention(s["q"], s["cache"], s["table"], s["ctx"], s["nodes"],
                                       s["latent"], s["scale"], tree_mask=s["mask"])
        if s["op"] == "latent_write":
            return ds.latent_write(s["c"], s["r"], s["positions"], s["table"], s["cache"],
                                   s["slots"], weight=s["w"], eps=EPS,
                                   interleaved=s["interleaved"], magnitude=s["magnitude"])
        how = dict(q_weight=s["qw"], k_weight=s["kw"], eps=EPS, rot_start=s["start"],
                   interleaved=s["interleaved"], magnitude=s["magnitude"])
        if s["kc"] is None:
            return ds.qk_rotate(s["q"], s["k"], s["positions"], s["table"], **how)
        return ds.rotate_write(s["q"], s["k"], s["v"], s["positions"], s["table"], s["kc"],
                               s["vc"], s["slots"], **how)
    return {"rotate": _plain_rotate, "latent_write": _plain_write,
            "latent": _plain_latent}[s["op"]](s)


def _plain_norm(x, w):
    if w is None:
        return x
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _plain_turn(x, s):
    """The pairs of x [n, .., rot] turned by their positions' angles."""
    n, rot = x.shape[0], x.shape[-1]
    angle = s["positions"].double()[:, None] * s["freq"]
    angle = angle.reshape(n, *[1] * (x.dim() - 2), rot // 2)
    cos, sin = ((f(angle) * s["magnitude"]).float() for f in (torch.cos, torch.sin))
    if s["interleaved"]:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    a, b = x[..., :rot // 2], x[..., rot // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_store(cache, slots, rows):
    on = slots >= 0
    at, page = slots[on].long(), cache.shape[1]
    cache[at // page, at % page] = rows[on].to(cache.dtype)


def _plain_rotate(s):
    """(q, k) normed and rotated, padding's rows 0; or (q, k cache, v cache)."""
    def head(x, w):
        x = _plain_norm(x.float(), w)
        lo, hi = s["start"], s["start"] + s["rot"]
        x = torch.cat([x[..., :lo], _plain_turn(x[..., lo:hi], s), x[..., hi:]], -1)
        return x.masked_fill((s["positions"] < 0)[:, None, None], 0).to(s["dtype"])

    q, k = head(s["q"], s["qw"]), head(s["k"], s["kw"])
    if s["kc"] is None:
        return q, k
    _plain_store(s["kc"], s["slots"], k)
    _plain_store(s["vc"], s["slots"], s["v"])
    return q, s["kc"], s["vc"]


def _plain_write(s):
    rows = torch.cat([_plain_norm(s["c"].float(), s["w"]), _plain_turn(s["r"].float(), s)], -1)
    _plain_store(s["cache"], s["slots"], rows)
    return s["cache"]


def _plain_latent(s):
    """(out, lse, status): softmax(scale q row^T) row[:latent] over the cached tokens and the nodes
    that the mask shows."""
    q, table, latent = s["q"].float(), s["table"].long(), s["latent"]
    B, T, H, W = q.shape
    page = s["cache"].shape[1]
    L = table.shape[1] * page
    ctx, n = s["ctx"].long(), s["nodes"].long()
    node = torch.arange(L, device=q.device) - ctx[:, None]              # [B, L]
    held = (table >= 0).repeat_interleave(page, 1) & (node < n[:, None])
    t = torch.arange(T, device=q.device)
    bits = s["mask"] if s["mask"] is not None else ((2 << t) - 1).expand(B, T)
    shown = (bits[:, :, None] >> node.clamp(0, 63)[:, None, :]) & 1     # [B, T, L]
    seen = held[:, None] & ((node < 0)[:, None] | (shown == 1)) & (t < n[:, None])[:, :, None]
    rows = s["cache"][table.clamp(min=0)].reshape(B, L, W).float()
    rows = rows.masked_fill(~held[:, :, None], 0)
    a = (q.reshape(B, T * H, W) @ rows.transpose(1, 2)).reshape(B, T, H, L) * s["scale"]
    a = a.masked_fill(~seen[:, :, None], -math.inf)
    m = a.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    a = torch.exp(a - m)
    z = a.sum(-1, keepdim=True)
    o = (a.reshape(B, T * H, L) @ rows[..., :latent]).reshape(B, T, H, latent)
    o = o / torch.where(z == 0, 1.0, z)
    return o.to(s["q"].dtype), (m + torch.log(z))[..., 0], torch.zeros_like(s["ctx"])


# ------------------------------------------------------------ what it takes
def work(case):
    c, B = case, case["batch"]
    if c["op"] == "latent":
        e, W = SIZE[c["dtype"]], c["latent"] + c["rope"]
        ctx, n = _lengths(B, c["lo"], c["hi"]), _nodes(B, c["depth"])
        tokens = sum(a + b for a, b in zip(ctx, n))
        rows = B * c["depth"] * c["heads"]
        pairs = sum(b * a + b * (b + 1) // 2 for a, b in zip(ctx, n))
        return {"bytes": tokens * W * e + rows * ((W + c["latent"]) * e + 4)
                + 4 * sum(-(-(a + b) // c["page"]) for a, b in zip(ctx, n)),
                "flops": 2 * pairs * c["heads"] * (W + c["latent"])}
    n = B * c["new"]
    live = sum(_nodes(B, c["new"])) if B > 1 else n
    move = SIZE[c["source"]] + SIZE[c["dtype"]]
    if c["op"] == "latent_write":
        cells = live * (1 - c["skip"]) * (c["latent"] + c["rope"])
        return {"bytes": cells * move + 8 * n, "flops": 6 * cells}
    q, k = c["heads"] * c["dim"], c["kv_heads"] * c["dim"]
    cells = live * (q + k * (2 if c["write"] else 1))
    padding = (n - live) * (q if c["write"] else q + k) * SIZE[c["dtype"]]
    return {"bytes": cells * move + padding + n * (8 if c["write"] else 4), "flops": 6 * cells}


# ------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "latent":
        return _exact_latent(s)
    return (_exact_rotate if case["op"] == "rotate" else _exact_write)(case, s)


def _exact_head(x, w, case, positions, start, rot, interleaved):
    """x [n, heads, dim] float64: the norm, then each pair as a complex number times its turn."""
    if w is not None:
        x = x * (np.square(x).mean(-1, keepdims=True) + EPS) ** -0.5 * w.double().cpu().numpy()
    y = x.copy()
    if rot:
        turn = np.exp(1j * np.outer(positions.astype(np.float64), _frequencies(case, rot)))
        turn = turn[:, None, :] * _scaling(case, rot)[1]
        i = np.arange(rot // 2)
        first = start + (2 * i if interleaved else i)
        second = first + (1 if interleaved else rot // 2)
        z = (x[..., first] + 1j * x[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_store(cache, slots, rows):
    blocks, page = cache.shape[:2]
    flat = np.zeros((blocks * page, *rows.shape[1:]))
    flat[slots[slots >= 0]] = rows[slots >= 0]
    return flat.reshape(blocks, page, *rows.shape[1:])


def _exact_rotate(case, s):
    positions = s["positions"].cpu().numpy()
    host = lambda t: t.double().cpu().numpy()  # noqa: E731
    q, k = (_exact_head(host(s[x]), s[w], case, positions, s["start"], s["rot"], s["interleaved"])
            for x, w in (("q", "qw"), ("k", "kw")))
    q[positions < 0] = 0
    k[positions < 0] = 0
    if s["kc"] is None:
        return q, k
    slots = s["slots"].cpu().numpy()
    return q, _exact_store(s["kc"], slots, k), _exact_store(s["vc"], slots, host(s["v"]))


def _exact_write(case, s):
    host = lambda t: t.double().cpu().numpy()[:, None]  # noqa: E731
    positions = s["positions"].cpu().numpy()
    c = _exact_head(host(s["c"]), s["w"], case, positions, 0, 0, False)
    r = _exact_head(host(s["r"]), None, case, positions, 0, s["r"].shape[1], s["interleaved"])
    rows = np.concatenate([c, r], -1)[:, 0]
    return _exact_store(s["cache"], s["slots"].cpu().numpy(), rows)


def _exact_latent(s):
    q, latent = s["q"], s["latent"]
    B, T, H, W = q.shape
    page = s["cache"].shape[1]
    out = torch.zeros(B, T, H, latent, dtype=torch.float64)
    lse = torch.full((B, T, H), -math.inf, dtype=torch.float64)
    for b in range(B):
        ctx, n = int(s["ctx"][b]), int(s["nodes"][b])
        blocks = s["table"][b, :-(-(ctx + n) // page)].long()
        rows = s["cache"][blocks].reshape(-1, W)[:ctx + n].double()
        for i in range(n):
            word = (2 << i) - 1 if s["mask"] is None else int(s["mask"][b, i])
            see = list(range(ctx)) + [ctx + j for j in range(n) if (word >> j) & 1]
            r = rows if len(see) == ctx + n else rows[torch.tensor(see, device=rows.device)]
            a = q[b, i].double() @ r.T * s["scale"]
            lse[b, i] = torch.logsumexp(a, -1).cpu()
            out[b, i] = (torch.softmax(a, -1) @ r[:, :latent]).cpu()
    return out.numpy(), lse.numpy(), None
