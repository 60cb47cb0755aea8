"""Plain implementations in 64-bit floats of the rotation of heads, the rows
of a latent cache and attention over it.  Written from the formulas in
include/dspark.h."""
import math

import numpy as np


def frequencies(rot, base=1e4, scaling=None, factor=1.0, original_len=1.0, low=1.0, high=32.0):
    out = []
    for i in range(rot // 2):
        f = base ** (-2 * i / rot)
        if scaling == "linear":
            f /= factor
        if scaling == "parts":
            keep = min(max((original_len * f / (2 * math.pi) - low) / (high - low), 0.0), 1.0)
            f *= keep + (1 - keep) / factor
        out.append(f)
    return np.array(out)


def head(x, weight, eps, positions, freq, start, interleaved, magnitude):
    """x [n, heads, dim] float64: (y, size), size the magnitude of each element's terms.  Padding's
    rows are 0."""
    n, heads, dim = x.shape
    if weight is not None:
        x = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * weight
    y, size = x.copy(), np.abs(x)
    rot = 2 * len(freq)
    for i in range(rot // 2):
        a, b = (start + 2 * i, start + 2 * i + 1) if interleaved else \
            (start + i, start + i + rot // 2)
        angle = positions.astype(np.float64) * freq[i]
        c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
        y[..., a] = (x[..., a] * c - x[..., b] * s) * magnitude
        y[..., b] = (x[..., b] * c + x[..., a] * s) * magnitude
        size[..., a] = size[..., b] = (np.abs(x[..., a]) + np.abs(x[..., b])) * abs(magnitude)
    y[positions < 0] = 0
    size[positions < 0] = 0
    return y, size


def latent_attention(q, cache, table, ctx, nodes, mask, scale, latent):
    """q [B, T, H, W], cache [blocks, page, W] float64: (out, lse, weight, reach) as
    serving_ref.attention gives them."""
    B, T, H, W = q.shape
    blocks, page, _ = cache.shape
    out, weight = np.zeros((B, T, H, latent)), np.zeros((B, T, H, latent))
    lse, reach = np.full((B, T, H), -np.inf), np.zeros((B, T, H))
    for b in range(B):
        c, n = int(ctx[b]), int(nodes[b])
        if c < 0 or n < 0 or n > T or c + n > table.shape[1] * page:
            continue
        i = np.arange(c + n)
        block = table[b][i // page]
        held = (block >= 0) & (block < blocks)
        rows = cache[np.where(held, block, 0), i % page]              # [L, W]
        for t in range(n):
            bits = int(mask[b, t]) if mask is not None else (2 << t) - 1
            seen = held.copy()
            for j in range(n):
                seen[c + j] &= bool((bits >> j) & 1)
            if not seen.any():
                continue
            r = rows[seen]
            s = q[b, t] @ r.T * scale                                 # [H, L]
            top = s.max(-1, keepdims=True)
            p = np.exp(s - top)
            z = p.sum(-1, keepdims=True)
            out[b, t] = p @ r[:, :latent] / z
            weight[b, t] = p @ np.abs(r[:, :latent]) / z
            lse[b, t] = (top + np.log(z))[:, 0]
            reach[b, t] = (np.abs(q[b, t]) @ np.abs(r).T).max(-1) * abs(scale)
    return out, lse, weight, reach
