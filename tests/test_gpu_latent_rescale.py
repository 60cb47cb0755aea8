"""Latent attention where the reference of the exponents moves at every tile,
so that every accumulator is rescaled between two products, over and over:
the results in 64 bits, and the same bits from run to run."""
import numpy as np
import pytest
import torch

from test_gpu_latent_attention import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("latent,rope", [(512, 64), (256, 32), (320, 0)])
@pytest.mark.parametrize("T,heads", [(4, 32), (1, 16), (6, 32)])
def test_the_reference_moves_at_every_tile(dtype, latent, rope, T, heads):
    c = Case([25000, 3000], [T, max(1, T - 1)], T, heads=heads, latent=latent, rope=rope, dtype=dtype,
             page=32, seed=T, spread=0.5)
    c.scale = 1.0
    c.cache *= 0.125
    # a key's first element is 8 more with every tile of 128 positions, 11.5 units of log2 to a
    # row whose query has 1 there, half of it or nothing to others: multiples of 8 up to 1,568, exact
    for b in range(2):
        i = np.arange(int(c.ctx[b] + c.nodes[b]))
        block = torch.from_numpy(c.table[b][i // 32].astype(np.int64)).cuda()
        c.cache[block, torch.from_numpy(i % 32).cuda(), 0] = \
            torch.from_numpy(i // 128 * 8.0).cuda().to(dtype)
    rows = torch.arange(T * heads, device="cuda").view(T, heads)
    c.q[..., 0] = torch.tensor([1.0, 0.5, 0.0, 1.0], device="cuda").to(dtype)[rows % 4]
    want = c.run()
    c.check(want)
    a = c.device()
    for _ in range(20):
        got = c.call(*a)
        assert all(torch.equal(x, y) for x, y in zip(want, got))
