"""Large scales on scores of 0: every weight is the same, and nothing is NaN."""
import pytest
import torch

from test_gpu_tree_attention import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,T,heads,page", [(128, 1, 8, 16), (128, 6, 8, 16), (128, 40, 16, 16),
                                              (64, 2, 8, 16), (256, 6, 8, 16), (256, 6, 8, 12)])
@pytest.mark.parametrize("scale", [2.2e38, -2.2e38, 1e-44])
def test_zero_scores(dim, T, heads, page, scale):
    c = Case([50, 300], [T, T], T, dim=dim, heads=heads, page=page, mask="tree")
    c.q.zero_()
    c.scale = scale
    c.check(c.run(scale=scale))
