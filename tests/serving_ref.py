"""Plain implementations, in Python integers and 64-bit floats, of the
operators around a speculative step: the plan of the paged cache, attention
of the nodes over it and the processing of the logits.  Written from the
formulas in include/dspark.h."""
import numpy as np

OK, NO_BLOCKS, BAD_LENGTH, BAD_TREE, BAD_PENALTY = 0, 10, 11, 12, 13


def cache_plan(ctx, new, max_new, page, table, free, n_free, parents=None):
    """dict(table, slots, positions, tree_mask, taken, status); lists of ints."""
    B, max_blocks = len(ctx), len(table[0])
    table = [list(r) for r in table]
    slots = [[-1] * max_new for _ in range(B)]
    positions = [[-1] * max_new for _ in range(B)]
    masks = [[0] * max_new for _ in range(B)]
    status, off, taken = [], 0, 0
    n_free = max(0, min(n_free, len(free)))
    for b in range(B):
        c, n = ctx[b], new[b]
        if c < 0 or n < 0 or n > max_new or -(-(c + n) // page) > max_blocks:
            status.append(BAD_LENGTH)
            continue
        held = -(-c // page)
        need = -(-(c + n) // page) - held
        off += need
        if need and off > n_free:
            status.append(NO_BLOCKS)
            continue
        taken = off if need else taken
        for i in range(need):
            table[b][held + i] = free[off - need + i]
        bad = parents is not None and any(not -1 <= parents[b][t] < t for t in range(n))
        status.append(BAD_TREE if bad else OK)
        for t in range(n):
            block = table[b][(c + t) // page]
            slot = block * page + (c + t) % page
            slots[b][t] = slot if block >= 0 and slot < 1 << 31 else -1
            if bad:
                continue
            if parents is None:
                m = (2 << t) - 1
            else:
                parent = parents[b][t]
                m = (1 << t) | (masks[b][parent] if parent >= 0 else 0)
            masks[b][t] = m if t < 64 else 0
            positions[b][t] = c + (t if parents is None else bin(m).count("1") - 1)
    return {"table": table, "slots": slots, "positions": positions, "tree_mask": masks,
            "taken": taken, "status": status}


def attention(q, k, v, table, ctx, nodes, mask, scale):
    """q [B, T, Hq, D], k / v [blocks, page, Hk, D] float64, table / ctx / nodes ints, mask uint64
    [B, T] or None: (out, lse, weight) with weight = sum_i p_i |v_i|, the scale of the
    output's rounding errors, and reach = max_i scale sum_d |q_d k_id|, that of the scores'."""
    B, T, Hq, D = q.shape
    blocks, page, Hk, _ = k.shape
    G = Hq // Hk
    out, weight = np.zeros(q.shape), np.zeros(q.shape)
    lse, reach = np.full(q.shape[:3], -np.inf), np.zeros(q.shape[:3])
    for b in range(B):
        c, n = int(ctx[b]), int(nodes[b])
        if c < 0 or n < 0 or n > T or c + n > table.shape[1] * page:
            continue
        i = np.arange(c + n)
        block = table[b][i // page]
        held = (block >= 0) & (block < blocks)
        at = np.where(held, block, 0)
        kb, vb = k[at, i % page], v[at, i % page]                     # [L, Hk, D]
        for t in range(n):
            bits = int(mask[b, t]) if mask is not None else (2 << t) - 1
            seen = held.copy()
            for j in range(n):
                seen[c + j] &= bool((bits >> j) & 1)
            if not seen.any():
                continue
            for h in range(Hq):
                kk, vv = kb[seen, h // G], vb[seen, h // G]
                s = kk @ q[b, t, h] * scale
                top = s.max()
                p = np.exp(s - top)
                z = p.sum()
                out[b, t, h] = p @ vv / z
                weight[b, t, h] = p @ np.abs(vv) / z
                lse[b, t, h] = top + np.log(z)
                reach[b, t, h] = (np.abs(kk) @ np.abs(q[b, t, h])).max() * abs(scale)
    return out, lse, weight, reach


def logits(x, history, prompt_len, history_len, drafts, row_mask, R, F, P, bias_ids, bias_values,
           n_bias, words, mask_rows):
    """x float64 [B, rows, V]: (y, size) with size the sum of the magnitudes of the terms."""
    B, rows, V = x.shape
    y, size = x.copy(), np.abs(np.where(np.isfinite(x), x, 0))
    for b in range(B):
        hl = 0 if history is None else min(max(int(history_len[b]), 0), history.shape[1])
        pl = 0 if prompt_len is None else min(max(int(prompt_len[b]), 0), hl)
        r_, f_, p_ = (d if t is None else float(t[b]) for t, d in ((R, 1.0), (F, 0.0), (P, 0.0)))
        if not (np.isfinite(r_) and r_ > 0 and np.isfinite(f_) and np.isfinite(p_)):
            y[b] = -np.inf
            continue
        for r in range(rows):
            prompt, said = set(), {}
            for i in range(hl):
                t = int(history[b, i])
                if not 0 <= t < V:
                    continue
                if i < pl:
                    prompt.add(t)
                else:
                    said[t] = said.get(t, 0) + 1
            for j in range(0 if drafts is None else drafts.shape[1]):
                on = j < r if row_mask is None else (int(row_mask[b, r]) >> j) & 1
                t = int(drafts[b, j])
                if on and 0 <= t < V:
                    said[t] = said.get(t, 0) + 1
            z, m = y[b, r], size[b, r]
            for t in prompt | set(said):
                c = said.get(t, 0)
                z[t] = z[t] / r_ if z[t] > 0 else z[t] * r_
                z[t] -= f_ * c + (p_ if c else 0)
                m[t] = m[t] * max(r_, 1 / r_) + abs(f_) * c + abs(p_)
            nb = 0 if bias_ids is None else bias_ids.shape[1]
            if n_bias is not None:
                nb = min(max(int(n_bias[b]), 0), nb)
            for i in range(nb):
                t = int(bias_ids[b, i])
                if 0 <= t < V:
                    z[t] += float(bias_values[b, i])
                    m[t] += abs(float(bias_values[b, i]))
            if words is not None:
                w = b * rows + r if mask_rows is None else int(mask_rows[b, r])
                if 0 <= w < words.shape[0]:
                    on = np.unpackbits(np.ascontiguousarray(words[w]).astype("<u4").view(np.uint8),
                                       bitorder="little")[:V]
                    z[on == 0] = -np.inf
    return y, size
