"""The rotation, the latent cache's write and attention over it refuse bad
arguments on the host (negative return codes, nothing launched) -- no GPU
needed."""
import ctypes

import pytest

from draft_sampling_verification_gb300 import _lib, build
from test_serving_abi import ALIGN, ARG, DTYPE, NULL, ODD, P, SIZE, caller

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_qk_rotate(lib):
    # q, k, src, q token, head, k token, head, n, heads, kv heads, dim, qw, kw, eps, positions,
    # table, start, rot, interleaved, magnitude, q out, token, head, k out, token, head, out, stream
    call = caller(lib.dspark_qk_rotate, (P, P, 0, 512, 64, 512, 64, 3, 8, 2, 64, None, None, 1e-6, P,
                                         P, 0, 64, 0, 1.0, P, 512, 64, P, 512, 64, 0, None))
    for kw in (dict(a2=3), dict(a26=-1), dict(a2=1), dict(a2=1, a26=2), dict(a2=2, a26=1)):
        assert call(**kw) == DTYPE, kw
    for kw in (dict(a7=-1), dict(a8=-1), dict(a9=-1), dict(a8=65535), dict(a10=0), dict(a10=60),
               dict(a10=264), dict(a16=8), dict(a16=4, a17=56), dict(a17=12), dict(a17=-8),
               dict(a16=-8), dict(a17=72), dict(a3=-4), dict(a4=-4), dict(a5=-4), dict(a6=-4),
               dict(a21=-4), dict(a22=-4), dict(a24=-4), dict(a25=-4)):
        assert call(**kw) == SIZE, kw
    for kw in (dict(a13=-1.0), dict(a13=NAN), dict(a13=INF), dict(a19=NAN), dict(a19=INF),
               dict(a21=256), dict(a25=128), dict(a26=1)):           # in place, other places
        assert call(**kw) == ARG, kw
    for i in (0, 1, 14, 15, 20, 23):
        assert call(**{"a%d" % i: None}) == NULL, i
    eight = ctypes.c_void_p(24)
    for kw in (dict(a0=eight), dict(a1=eight), dict(a20=eight), dict(a23=eight), dict(a3=510),
               dict(a4=62), dict(a5=510), dict(a6=62), dict(a21=510), dict(a25=62), dict(a11=ODD),
               dict(a12=ODD), dict(a14=ODD), dict(a15=ctypes.c_void_p(20)),
               dict(a2=1, a26=1, a3=508)):
        assert call(**kw) == ALIGN, kw
    assert call(a7=0) == 0 and call(a8=0, a9=0) == 0


def test_rotate_write(lib):
    # q, k, v, src, q token, head, kv token, head, n src, heads, kv heads, dim, qw, kw, eps,
    # positions, table, start, rot, interleaved, magnitude, q out, token, head, kc, vc, dtype,
    # block, token, head, blocks, page, slots, rows, n, stream
    call = caller(lib.dspark_rotate_write, (
        P, P, P, 0, 512, 64, 128, 64, 3, 8, 2, 64, None, None, 1e-6, P, P, 0, 64, 0, 1.0,
        ctypes.c_void_p(32), 512, 64, P, P, 1, 2048, 128, 64, 5, 16, P, None, 3, None))
    for kw in (dict(a26=0), dict(a26=7), dict(a3=2), dict(a3=9)):
        assert call(**kw) == DTYPE, kw
    for kw in (dict(a30=0), dict(a31=0), dict(a31=1025), dict(a30=1 << 28), dict(a8=-1),
               dict(a34=-1), dict(a10=0), dict(a11=4), dict(a11=264), dict(a6=-8), dict(a7=-8),
               dict(a4=-8), dict(a27=-8), dict(a18=72), dict(a9=-1)):
        assert call(**kw) == SIZE, kw
    assert call(a33=P) == ARG and call(a14=NAN) == ARG and call(a20=INF) == ARG
    assert call(a21=P) == ARG                                        # fp32 queries in place
    for i in (0, 1, 2, 15, 16, 21, 24, 25, 32):
        assert call(**{"a%d" % i: None}) == NULL, i
    for kw in (dict(a0=ODD), dict(a1=ODD), dict(a2=ODD), dict(a24=ctypes.c_void_p(24)), dict(a6=126),
               dict(a22=508), dict(a27=2044), dict(a28=4), dict(a29=1), dict(a32=ODD), dict(a15=ODD)):
        assert call(**kw) == ALIGN, kw
    assert call(a34=0) == 0 and call(a8=0, a9=0) == 0


def test_latent_write(lib):
    # c, token, r, token, src, n src, latent, rope, weight, eps, positions, table, interleaved,
    # magnitude, cache, dtype, block, token, blocks, page, slots, rows, n, stream
    call = caller(lib.dspark_latent_write, (P, 576, P, 576, 0, 3, 512, 64, None, 1e-6, P, P, 0, 1.0,
                                            P, 1, 9216, 576, 5, 16, P, None, 3, None))
    for kw in (dict(a15=0), dict(a15=5), dict(a4=2), dict(a4=-1)):
        assert call(**kw) == DTYPE, kw
    for kw in (dict(a5=-1), dict(a22=-1), dict(a6=0), dict(a6=32), dict(a6=96), dict(a6=576),
               dict(a7=-8), dict(a7=4), dict(a7=72), dict(a1=-4), dict(a3=-4), dict(a16=-8),
               dict(a18=0), dict(a19=0), dict(a19=1025)):
        assert call(**kw) == SIZE, kw
    assert call(a9=NAN) == ARG and call(a13=NAN) == ARG and call(a9=-1.0) == ARG
    for i in (0, 2, 10, 11, 14, 20):
        assert call(**{"a%d" % i: None}) == NULL, i
    for kw in (dict(a0=ODD), dict(a2=ODD), dict(a1=574), dict(a3=574), dict(a14=ODD), dict(a16=9220),
               dict(a17=580), dict(a20=ODD), dict(a21=ODD), dict(a10=ODD), dict(a8=ODD),
               dict(a11=ctypes.c_void_p(20))):
        assert call(**kw) == ALIGN, kw
    assert call(a22=0) == 0 and call(a5=0) == 0


def test_latent_attention(lib):
    # q, dtype, req, node, head stride, B, nodes, heads, latent, rope, cache, block, token, blocks,
    # page, table, ld, max blocks, ctx, nodes, mask, scale, out, lse, status, workspace, stream
    call = caller(lib.dspark_latent_attention, (P, 1, 9216, 9216, 576, 1, 1, 16, 512, 64, P, 9216,
                                                576, 5, 16, P, 4, 4, P, P, None, 0.1, P, None, P, P,
                                                None))
    assert call(a1=0) == DTYPE and call(a1=3) == DTYPE
    for kw in (dict(a5=-1), dict(a5=65536), dict(a6=0), dict(a6=65), dict(a7=0), dict(a7=129),
               dict(a8=0), dict(a8=500), dict(a8=576), dict(a9=-8), dict(a9=4), dict(a9=72),
               dict(a12=568), dict(a11=568), dict(a13=0), dict(a14=0), dict(a14=12), dict(a14=1032),
               dict(a16=3), dict(a17=0), dict(a16=1 << 27, a17=1 << 27), dict(a2=-8), dict(a3=-8),
               dict(a4=-8), dict(a11=1 << 39)):
        assert call(**kw) == SIZE, kw
    for s in (NAN, INF, -INF, 2.4e38):
        assert call(a21=s) == ARG
    for i in (0, 10, 15, 18, 19, 22, 24, 25):
        assert call(**{"a%d" % i: None}) == NULL, i
    for kw in (dict(a0=ODD), dict(a10=ODD), dict(a22=ODD), dict(a25=ODD), dict(a15=ODD),
               dict(a18=ODD), dict(a19=ODD), dict(a20=ctypes.c_void_p(20)), dict(a23=ODD),
               dict(a24=ODD), dict(a2=9220), dict(a3=9220), dict(a4=580), dict(a11=9220),
               dict(a12=580)):
        assert call(**kw) == ALIGN, kw
    assert call(a5=0) == 0
    size = lib.dspark_latent_attention_workspace_bytes
    assert size(1, 1, 16, 512) > 0 and size(0, 1, 1, 64) > 0
    for a in ((1, 0, 16, 512), (1, 65, 16, 512), (1, 1, 0, 512), (1, 1, 129, 512), (1, 1, 16, 500),
              (-1, 1, 16, 512), (1, 1, 16, 576)):
        assert size(*a) == 0, a


def test_latent_write_refuses_a_cache_whose_rows_overlap(lib):
    # as in test_latent_write; n = 0: nothing is launched where the call is good
    call = caller(lib.dspark_latent_write, (P, 576, P, 576, 0, 3, 512, 64, None, 1e-6, P, P, 0, 1.0,
                                            P, 1, 9216, 576, 5, 16, P, None, 0, None))
    for kw in (dict(a17=568), dict(a17=0), dict(a16=568), dict(a16=0)):
        assert call(**kw) == SIZE, kw
    # one row, one block; blocks that lie between one another's rows
    for kw in (dict(a17=0, a19=1), dict(a16=0, a18=1), dict(a16=576, a17=2880)):
        assert call(**kw) == 0, kw
