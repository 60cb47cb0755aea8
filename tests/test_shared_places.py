"""Outputs of the rotation whose rows share elements are refused, by the
binding and by the library, and those that only lie between one another's rows
are not: the binding's rule against every place of small layouts -- no GPU
needed."""
import ctypes

import pytest
import torch

import draft_sampling_verification_gb300 as ds
from draft_sampling_verification_gb300 import _lib, build
from test_other_device import HEADS, TURN, Current, called, on  # noqa: F401
from test_serving_abi import P, SIZE, caller

SHARED = [(64, 64), (64, 192), (0, 64), (256, 0), (32, 256), (256, 32), (192, 128),
          (160, 320)]                                   # two tokens' steps are one head's
APART = [(256, 64), (64, 256), (512, 128), (128, 512), (72, 288), (256, 320)]


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def shared(width, dims):
    """By going through all places; dims: (count, stride)."""
    places = [0]
    for count, stride in dims:
        places = [p + i * stride for p in places for i in range(count)]
    places.sort()
    return any(b - a < width for a, b in zip(places, places[1:]))


@pytest.mark.parametrize("token,head", SHARED + APART)
def test_the_binding(called, token, head):  # noqa: F811
    args = {k: on(Current, *shape, dtype=dtype) for k, (shape, dtype) in HEADS.items()
            if k not in ("k", "k_weight")}
    args["q"] = on(Current, 4, 4, 64)
    out = torch.zeros(5000, dtype=torch.bfloat16).as_strided((4, 4, 64), (token, head, 1))
    call = lambda: ds.dspark_qk_rotate(k=None, k_weight=None, k_out=None,       # noqa: E731
                                       q_out=out.as_subclass(Current), **args, **TURN)
    assert shared(64, [(4, token), (4, head)]) == ((token, head) in SHARED)
    if (token, head) in APART:
        call()
        assert called == ["dspark_qk_rotate"]
        return
    with pytest.raises(ValueError, match="must not overlap"):
        call()
    assert called == []


def test_the_binding_on_all_small_layouts():
    for n in (1, 2, 3, 5):
        for heads in (1, 2, 4):
            for token in range(0, 44, 4):
                for head in range(0, 44, 4):
                    # a dimension of one element has stride 0 there
                    a = (0, 0, token if n > 1 else 0, head if heads > 1 else 0, n, heads, 8)
                    want = shared(8, [(n, token), (heads, head)])
                    try:
                        ds._written("x", None, a)
                        assert not want, a
                    except ValueError:
                        assert want, a


@pytest.mark.parametrize("token,head", SHARED)
def test_the_library(lib, token, head):
    # arguments as in test_latent_abi, with 4 tokens and 4 heads; a good layout is not tried, as
    # it would be launched
    far = ctypes.c_void_p(1 << 20)
    call = caller(lib.dspark_qk_rotate, (P, P, 0, 512, 64, 512, 64, 4, 4, 4, 64, None, None, 1e-6, P,
                                         P, 0, 64, 0, 1.0, far, 256, 64, far, 256, 64, 0, None))
    assert call(a21=token, a22=head) == SIZE
    assert call(a24=token, a25=head) == SIZE
    call = caller(lib.dspark_rotate_write, (
        P, P, P, 0, 512, 64, 128, 64, 4, 4, 2, 64, None, None, 1e-6, P, P, 0, 64, 0, 1.0,
        far, 256, 64, P, P, 1, 2048, 128, 64, 5, 16, P, None, 4, None))
    assert call(a22=token, a23=head) == SIZE
