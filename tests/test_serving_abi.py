"""The operators around a speculative step refuse bad arguments on the host
(negative return codes, nothing launched) -- no GPU needed."""
import ctypes

import pytest

from draft_sampling_verification_gb300 import _lib, build

P = ctypes.c_void_p(16)        # a non-null, aligned placeholder; never dereferenced
ODD = ctypes.c_void_p(18)
NULL, SIZE, DTYPE, ALIGN, ARG = -1, -2, -3, -5, -7


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def caller(f, ok):
    def call(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)
    return call


def test_cache_plan(lib):
    # ctx, new, B, max_new, page, table, ld, max_blocks, free, max_free, n_free, parents, slots,
    # positions, mask, taken, status, stream
    call = caller(lib.dspark_cache_plan, (P, P, 1, 6, 16, P, 4, 4, P, 9, None, None, P, None, None,
                                          P, P, None))
    for kw in (dict(a2=-1), dict(a3=0), dict(a3=(1 << 24) + 1), dict(a4=0), dict(a4=1025),
               dict(a7=0), dict(a6=3), dict(a9=-1), dict(a7=1 << 28, a6=1 << 28),
               dict(a2=1 << 30), dict(a3=65, a11=P), dict(a3=65, a14=P)):
        assert call(**kw) == SIZE, kw
    for i in (0, 1, 5, 8, 12, 15, 16):
        assert call(**{"a%d" % i: None}) == NULL
    for i in (0, 1, 5, 8, 10, 11, 12, 13, 15, 16):
        assert call(**{"a%d" % i: ODD}) == ALIGN
    assert call(a14=ctypes.c_void_p(20)) == ALIGN
    assert call(a2=0) == 0


def test_kv_write(lib):
    # k, v, src dtype, token, head stride, n_src, heads, dim, kc, vc, dtype, block, token, head
    # stride, blocks, page, slots, rows, n, stream
    call = caller(lib.dspark_kv_write, (P, P, 1, 128, 64, 3, 2, 64, P, P, 1, 2048, 128, 64, 5, 16,
                                        P, None, 3, None))
    assert call(a10=0) == DTYPE and call(a10=7) == DTYPE
    assert call(a2=2) == DTYPE and call(a2=9) == DTYPE     # f16 into a bf16 cache
    for kw in (dict(a14=0), dict(a15=0), dict(a15=1025), dict(a14=1 << 28), dict(a5=-1),
               dict(a18=-1), dict(a6=0), dict(a7=4), dict(a7=12), dict(a7=1032), dict(a3=-8),
               dict(a11=-8)):
        assert call(**kw) == SIZE, kw
    for kw in (dict(a11=2044), dict(a12=4), dict(a13=1), dict(a3=68), dict(a4=4), dict(a0=ODD),
               dict(a9=ctypes.c_void_p(24)), dict(a16=ODD), dict(a17=ODD)):
        assert call(**kw) == ALIGN, kw
    for i in (0, 1, 8, 9, 16):
        assert call(**{"a%d" % i: None}) == NULL
    assert call(a18=0) == 0 and call(a5=0) == 0


def test_tree_attention(lib):
    # q, dtype, req, node, head stride, B, nodes, heads, kv_heads, dim, kc, vc, block, token, head
    # stride, blocks, page, table, ld, max_blocks, ctx, nodes, mask, scale, out, lse, status, ws,
    # stream
    call = caller(lib.dspark_tree_attention,
                  (P, 1, 6144, 1024, 128, 1, 6, 8, 2, 128, P, P, 4096, 256, 128, 5, 16, P, 4, 4, P,
                   P, None, 0.1, P, None, P, P, None))
    assert call(a1=0) == DTYPE and call(a1=3) == DTYPE
    for kw in (dict(a5=-1), dict(a5=65536), dict(a6=0), dict(a6=65), dict(a7=9), dict(a7=0),
               dict(a8=0), dict(a7=130), dict(a9=96), dict(a9=0), dict(a15=0), dict(a16=0),
               dict(a16=1025), dict(a19=0), dict(a18=3), dict(a2=-8), dict(a12=-8),
               dict(a18=1 << 28, a19=1 << 28)):
        assert call(**kw) == SIZE, kw
    assert call(a23=float("nan")) == ARG and call(a23=float("inf")) == ARG
    for kw in (dict(a2=6140), dict(a3=4), dict(a4=1), dict(a12=4), dict(a0=ODD),
               dict(a10=ctypes.c_void_p(24)), dict(a17=ODD), dict(a22=ctypes.c_void_p(20)),
               dict(a24=ctypes.c_void_p(24)), dict(a25=ODD), dict(a27=ctypes.c_void_p(24))):
        assert call(**kw) == ALIGN, kw
    for i in (0, 10, 11, 17, 20, 21, 24, 26, 27):
        assert call(**{"a%d" % i: None}) == NULL
    assert call(a5=0) == 0
    w = lib.dspark_tree_attention_workspace_bytes
    assert w(1, 6, 8, 2, 128) > 0 and w(1, 6, 8, 3, 128) == 0 and w(1, 65, 8, 2, 128) == 0


def test_logits_process(lib):
    # x, dtype, ld, B, rows, V, history, ld, prompt, len, drafts, n, row mask, R, F, P, bias ids,
    # values, max, n, words, ld, n_masks, mask rows, out, ld, status, stream
    call = caller(lib.dspark_logits_process,
                  (P, 1, 64, 1, 6, 64, P, 9, P, P, P, 5, P, P, P, P, P, P, 3, P, P, 2, 4, P,
                   ctypes.c_void_p(4096), 64, P, None))
    assert call(a1=2) == DTYPE                             # half-precision logits
    for kw in (dict(a5=0), dict(a5=131073), dict(a2=63), dict(a25=63), dict(a3=-1), dict(a3=65536),
               dict(a4=0), dict(a4=65), dict(a11=65), dict(a11=-1), dict(a18=-1), dict(a18=65536),
               dict(a7=-1), dict(a7=1 << 24), dict(a21=1), dict(a22=0)):
        assert call(**kw) == SIZE, kw
    for i in (0, 9, 10, 16, 17, 24, 26):
        assert call(**{"a%d" % i: None}) == NULL
    assert call(a24=P, a25=65) == ARG                      # in place with another stride
    for i in (6, 8, 9, 10, 13, 14, 15, 16, 17, 19, 20, 23, 26):
        assert call(**{"a%d" % i: ODD}) == ALIGN
    assert call(a12=ctypes.c_void_p(20)) == ALIGN and call(a0=ctypes.c_void_p(17)) == ALIGN
    assert call(a3=0) == 0
