"""Latent attention over long texts in f16, whose weights lose bits below 2^-14
and are 0 below 2^-25 of the exponents' reference.

A weight is off by u = 2^-11 of it, and by 2^-25 at most where it is below
2^-14.  The reference is not above the row's largest score, so against Z, the
sum of the weights relative to that score, N of the latter move a result by
N 2^-25 max|v| / Z at most.  A product adds 16 positions to the accumulator,
which drops what lies 2^-24 below it: N / 16 times.  The rest of the bound is
that of test_gpu_latent_attention.  One key that outweighs all others hides up
to 2^-24 of its weight of each of them, as dspark.h says."""
import numpy as np
import pytest
import torch

import latent_ref as ref
from test_gpu_latent_attention import Case, f64

pytestmark = pytest.mark.gpu

N = 100_003


def check(c, got, small):
    out, lse, status = got
    want, wlse, weight, reach = ref.latent_attention(
        f64(c.q), f64(c.cache), c.table, c.ctx, c.nodes, None, c.scale, c.latent)
    u, W = 2.0 ** -11, c.q.shape[-1]
    score = W * 2.0 ** -23 * reach + 2.0 ** -20
    tol = (u * (weight * (1 + u) + np.abs(want)) + 2 * score[..., None] * weight +
           N / 16 * 2.0 ** -24 * weight + small(wlse) + 2.0 ** -25)
    err = np.abs(f64(out) - want)
    assert (err <= tol).all(), float((err / tol).max())
    assert (np.abs(f64(lse) - wlse) <= score + 2.0 ** -22 * np.abs(wlse) + 2.0 ** -18).all()
    assert (status == 0).all()


@pytest.mark.parametrize("latent,rope", [(512, 64), (256, 32)])
@pytest.mark.parametrize("spread", [0.2, 2.0])
def test_weights_below_the_normal_range(latent, rope, spread):
    c = Case([N - 1], [1], 1, heads=16, latent=latent, rope=rope, dtype=torch.float16, spread=spread,
             seed=latent, page=64)
    got = c.run()
    rows = f64(c.cache)[c.table[0, np.arange(N) // 64], np.arange(N) % 64]
    top = (f64(c.q)[0, 0] @ rows.T).max(-1) * c.scale
    most = np.abs(rows[:, :latent]).max()
    check(c, got, lambda lse: (N * most * 2.0 ** -25 / np.exp(lse - top))[..., None])


def test_one_key_outweighs_the_others():
    c = Case([N - 1], [1], 1, heads=4, dtype=torch.float16, page=64)
    c.scale = 1.0
    c.cache[..., 0] = 0
    c.cache[..., 1] = 1
    at = int(c.table[0, 700]), 5
    c.cache[at[0], at[1], 0] = 17.625                        # 2^25.4 times the others' weight
    c.cache[at[0], at[1], 1:] = 0
    c.q.zero_()
    c.q[..., 0] = 1
    got = c.run()
    most = float(c.cache[..., 1:512].abs().max())
    check(c, got, lambda lse: N * most * 2.0 ** -24)
