"""The rotation's table against exact arithmetic, on the host: no GPU."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import draft_sampling_verification_gb300 as ds
import latent_ref as ref
from draft_sampling_verification_gb300 import build

# 2 pi to 30 digits
TAU = Fraction(6283185307179586476925286766559, 10 ** 30)


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


def turns(table):
    return [int(t) & (2 ** 64 - 1) for t in table.tolist()]


@pytest.mark.parametrize("rot", [8, 16, 64, 128, 256])
@pytest.mark.parametrize("how", [
    dict(), dict(base=1e6), dict(base=10.0), dict(scaling="linear", factor=8.0),
    dict(scaling="parts", factor=32.0, original_len=4096), dict(
        base=5e5, scaling="parts", factor=8.0, original_len=8192, low=1.0, high=4.0)])
def test_frequencies(rot, how):
    """Within the roundings of the doubles: the power (one unit in the last place or two), the
    scaling's few operations and the division by 2 pi (8 units of 2^-53 in all), then 2^-65."""
    table = ds.rope_table(rot, device="cpu", **how)
    assert table.dtype is torch.int64 and table.shape == (rot // 2,)
    for got, f in zip(turns(table), ref.frequencies(rot, **how)):
        want = Fraction(float(f)) / TAU
        assert abs(Fraction(got, 2 ** 64) - want) <= want * Fraction(16, 2 ** 53) + \
            Fraction(1, 2 ** 65)


def test_given_frequencies():
    f = [1.0, 0.5, 7.0, 0.0]                     # 7 radians: more than one turn
    for given in (f, torch.tensor(f), np.array(f)):
        got = turns(ds.rope_table(8, inv_freq=given, device="cpu"))
        for g, x in zip(got, f):
            want = Fraction(x) / TAU % 1
            assert abs(Fraction(g, 2 ** 64) - want) <= Fraction(4, 2 ** 53)
    scaled = turns(ds.rope_table(8, inv_freq=f, scaling="linear", factor=2.0, device="cpu"))
    assert scaled == turns(ds.rope_table(8, inv_freq=[x / 2 for x in f], device="cpu"))


def test_refusals():
    for kw in (dict(rot_dim=0), dict(rot_dim=4), dict(rot_dim=12), dict(rot_dim=264),
               dict(rot_dim=-8), dict(base=0.0), dict(base=-1.0), dict(base=float("inf")),
               dict(base=float("nan")), dict(scaling="linear", factor=0.0),
               dict(scaling="linear", factor=float("nan")),
               dict(scaling="parts", factor=2.0, original_len=0.0),
               dict(scaling="parts", factor=2.0, original_len=9.0, low=3.0, high=3.0),
               dict(scaling="parts", factor=2.0, original_len=9.0, low=float("nan")),
               dict(scaling="dynamic"), dict(inv_freq=[1.0] * 3), dict(inv_freq=[1.0] * 5),
               dict(inv_freq=[1.0, -1.0, 1.0, 1.0]), dict(inv_freq=[1.0, float("nan"), 1.0, 1.0]),
               dict(inv_freq=[float("inf")] * 4)):
        with pytest.raises((RuntimeError, ValueError)):
            ds.rope_table(**{"rot_dim": 8, "device": "cpu", **kw})
