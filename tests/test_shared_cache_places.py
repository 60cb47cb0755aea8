"""The latent write and the write of rotated keys refuse a cache two of whose
rows share elements: the library's rule against every place of many layouts --
no GPU needed."""
import ctypes
import random

import pytest

from test_latent_abi import lib  # noqa: F401
from test_serving_abi import P, SIZE, caller
from test_shared_places import shared


@pytest.fixture(scope="module")
def latent_write(lib):  # noqa: F811
    # as in test_latent_abi; no tokens: nothing is launched where the cache is good
    return caller(lib.dspark_latent_write, (P, 576, P, 576, 0, 3, 512, 64, None, 1e-6, P, P, 0, 1.0,
                                            P, 1, 9216, 576, 5, 16, P, None, 0, None))


@pytest.mark.parametrize("block", [576, 1152, 8640, 9208])
def test_blocks_that_begin_inside_others(latent_write, block):
    assert latent_write(a16=block) == SIZE


@pytest.mark.parametrize("block,token", [(9216, 576), (9600, 576), (9216, 584), (576, 2880),
                                         (584, 2920), (1152, 5760)])
def test_rows_apart(latent_write, block, token):
    blocks, page = 5, 16
    want = shared(576, [(blocks, block), (page, token)])
    assert want == (block == 9216 and token == 584)
    assert latent_write(a16=block, a17=token) == (SIZE if want else 0)


def test_many_layouts(latent_write):
    rng = random.Random(1)
    seen = [0, 0]
    for _ in range(4000):
        blocks, page = rng.randint(1, 5), rng.randint(1, 5)
        block, token = 8 * rng.randint(0, 90), 8 * rng.randint(0, 90)
        want = shared(72, [(blocks, block), (page, token)])
        got = latent_write(a6=64, a7=8, a16=block, a17=token, a18=blocks, a19=page)
        assert got == (SIZE if want else 0), (blocks, page, block, token)
        seen[want] += 1
    assert min(seen) > 500


def test_layouts_of_the_largest_sizes(latent_write):
    """Products of counts and strides beyond 63 bits are no shorter for it."""
    big = 2 ** 63 - 8
    kw = dict(a18=2 ** 20, a19=1024)
    assert latent_write(a16=big, a17=576, **kw) == 0
    assert latent_write(a16=big, a17=big, **kw) == SIZE
    assert latent_write(a16=2 ** 62, a17=2 ** 61, **kw) == SIZE
    assert latent_write(a16=1024 * 2 ** 50, a17=2 ** 50, **kw) == 0


@pytest.fixture(scope="module")
def rotate_write(lib):  # noqa: F811
    # as in test_latent_abi, with no tokens
    return caller(lib.dspark_rotate_write, (
        P, P, P, 0, 512, 64, 128, 64, 3, 8, 2, 64, None, None, 1e-6, P, P, 0, 64, 0, 1.0,
        ctypes.c_void_p(32), 512, 64, P, P, 1, 2048, 128, 64, 5, 16, P, None, 0, None))


@pytest.mark.parametrize("block,token,head", [
    (2048, 128, 64), (2048, 64, 1024), (64, 640, 320), (128, 640, 64), (2048, 128, 0), (0, 128, 64),
    (1984, 128, 64), (128, 128, 64), (2048, 64, 64), (2048, 120, 64), (2048, 64, 960)])
def test_caches_of_heads(rotate_write, block, token, head):
    want = shared(64, [(5, block), (16, token), (2, head)])
    assert want == ((block, token, head) not in ((2048, 128, 64), (2048, 64, 1024), (64, 640, 320),
                                                 (128, 640, 64)))
    assert rotate_write(a27=block, a28=token, a29=head) == (SIZE if want else 0)


def test_many_caches_of_heads(rotate_write):
    rng = random.Random(2)
    seen = [0, 0]
    for _ in range(4000):
        count = [rng.randint(1, 4) for _ in range(3)]
        stride = [8 * rng.randint(0, 1 << rng.randint(2, 5)) for _ in range(3)]
        want = shared(16, list(zip(count, stride)))
        got = rotate_write(a11=16, a18=16, a30=count[0], a31=count[1], a10=count[2], a27=stride[0],
                           a28=stride[1], a29=stride[2])
        assert got == (SIZE if want else 0), (count, stride)
        seen[want] += 1
    assert min(seen) > 500
