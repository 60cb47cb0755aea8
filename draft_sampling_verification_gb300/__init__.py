"""GB300 draft sampling and verification (dyadic24-standard-v1).

Thin Python binding of the C ABI in ``include/dspark.h``: the functions named
like the C calls (``dspark_q_build``, ``dspark_draft_sample``,
``dspark_verify_greedy``, ``dspark_verify_ratio``, ``dspark_target_probs``,
``dspark_cache_plan``, ``dspark_kv_write``, ``dspark_tree_attention``,
``dspark_logits_process``)
take torch CUDA tensors, pass their device pointers, sizes and the current
stream to libdspark.so, and raise on a nonzero return.  Every step of the
path runs in the library's CUDA kernels; torch only provides device memory
and streams.  The lower-case helpers (``q_build`` ...) allocate the outputs
with torch and call the same entry points.
"""
from __future__ import annotations

import ctypes
import functools
import inspect

import torch

from . import _lib

M = 1 << 24
F32, BF16, F16 = 0, 1, 2
ST_OK, ST_NONFINITE, ST_ZERO_MASS, ST_ALLOC_INCONSISTENT = 0, 1, 2, 3
ST_BAD_TEMPERATURE, ST_BAD_Q, ST_BAD_DRAFT, ST_TIMEOUT, ST_INTERNAL = 4, 5, 6, 7, 8
ST_BAD_CHECKSUM, ST_NO_BLOCKS, ST_BAD_LENGTH, ST_BAD_TREE, ST_BAD_PENALTY = 9, 10, 11, 12, 13
MAX_NODES = 64
FLAG_AMBIG_ACCEPT, FLAG_NEAR_BOUNDARY, FLAG_DEGENERATE = 1, 2, 4
SCHEDULE_AUTO, SCHEDULE_ONE_LAUNCH, SCHEDULE_SEPARATE = 0, 1, 2
PURPOSE_PROPOSAL, PURPOSE_ACCEPT, PURPOSE_RESIDUAL, PURPOSE_BONUS, PURPOSE_MATCH = 0, 1, 2, 3, 4

__all__ = ["dspark_q_build", "dspark_q_build_sample", "dspark_draft_sample", "dspark_verify_greedy",
           "dspark_verify_ratio", "dspark_verify", "dspark_verify_stats", "verify_stats",
           "dspark_target_probs", "dspark_spec_step",
           "dspark_spec_step_schedule", "dspark_spec_step_noalloc", "dspark_q_pack",
           "dspark_q_validate", "dspark_verify_match", "verify_match", "dspark_q_chain_sample",
           "q_chain_sample", "dspark_q_build_sample_sharded", "dspark_q_sharded_workspace_bytes",
           "q_build_sample_sharded", "dspark_spec_step_host",
           "dspark_spec_step_host_staging_bytes", "q_build",
           "draft_sample", "verify_greedy", "verify_ratio", "target_probs", "q_build_sample",
           "spec_step", "version", "dspark_cache_plan", "cache_plan", "dspark_kv_write", "kv_write",
           "dspark_tree_attention", "dspark_tree_attention_workspace_bytes", "tree_attention",
           "dspark_logits_process", "logits_process"]


def version() -> str:
    return _lib.load().dspark_version().decode()


def _call(name, *args):
    rc = getattr(_lib._lib or _lib.load(), name)(*args)
    if rc != 0:
        raise RuntimeError("%s failed with code %d" % (name, rc))


def _stream(stream):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    return ctypes.c_void_p(t.data_ptr())


def _dtype_code(t):
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError("logits must be float32 or bfloat16, got %s" % t.dtype)


def _uniform(t, dims, what):
    """(count, step) of what lies along t's first `dims` dimensions: one after the other, `step`
    apart (0 for one alone).  A dimension of one element may have any stride."""
    shape, strides, n, step = t.shape, t.stride(), 1, 0
    for i in range(dims - 1, -1, -1):
        if shape[i] > 1:
            if n == 1:
                step = strides[i]
            elif n and strides[i] != step * n:
                raise ValueError("%s must be uniformly strided" % what)
        n *= shape[i]
    return n, step


def _rows(t):
    """(rows, V, ld) of a logit tensor whose rows are uniformly strided."""
    if t.dim() >= 2 and t.is_contiguous() and t.shape[-1] > 0:
        V = t.shape[-1]
        return t.numel() // V, V, V
    if t.dim() < 2 or t.stride(-1) != 1:
        raise ValueError("logit rows must be contiguous in their last dimension")
    V = t.shape[-1]
    rows, ld = _uniform(t, t.dim() - 1, "logit rows")
    return rows, V, ld if rows > 1 else V


def _i32(t):
    if t is not None and t.dtype not in (torch.int32, torch.uint32):
        raise TypeError("expected an int32/uint32 tensor")
    return _ptr(t)


# ------------------------------------------------------------ C-named calls
def dspark_q_build(draft_logits, temperature, top_k, counts, sparse_ids, nnz, row_status,
                   stream=None):
    rows, V, ld = _rows(draft_logits)
    _call("dspark_q_build", _ptr(draft_logits), _dtype_code(draft_logits), ld, rows, V,
          _ptr(temperature), int(top_k), _i32(counts), _i32(sparse_ids), _i32(nnz),
          _i32(row_status), _stream(stream))


def dspark_q_build_sample(draft_logits, B, depth, temperature, top_k, seed, request_ids, counts,
                          sparse_ids, nnz, draft_tokens, row_status, stream=None):
    rows, V, ld = _rows(draft_logits)
    if rows != B * depth:
        raise ValueError("draft_logits must hold B*depth rows")
    _call("dspark_q_build_sample", _ptr(draft_logits), _dtype_code(draft_logits), ld, int(B),
          int(depth), V, _ptr(temperature), int(top_k), int(seed) & (2 ** 64 - 1),
          _i32(request_ids), _i32(counts), _i32(sparse_ids), _i32(nnz), _i32(draft_tokens),
          _i32(row_status), _stream(stream))


def dspark_draft_sample(counts, sparse_ids, nnz, top_k, B, depth, V, seed, request_ids,
                        draft_tokens, row_status, stream=None):
    _call("dspark_draft_sample", _i32(counts), _i32(sparse_ids), _i32(nnz), int(top_k), int(B),
          int(depth), int(V), int(seed) & (2 ** 64 - 1), _i32(request_ids), _i32(draft_tokens),
          _i32(row_status), _stream(stream))


def dspark_verify_greedy(target_logits, B, depth, draft_tokens, accept_len, committed,
                         req_status, stream=None):
    rows, V, ld = _rows(target_logits)
    if rows != B * (depth + 1):
        raise ValueError("target_logits must hold B*(depth+1) rows")
    _call("dspark_verify_greedy", _ptr(target_logits), _dtype_code(target_logits), ld, int(B),
          int(depth), V, _i32(draft_tokens), _i32(accept_len), _i32(committed),
          _i32(req_status), _stream(stream))


def dspark_verify_ratio(target_logits, B, depth, draft_tokens, counts, sparse_ids, nnz, top_k,
                        seed, request_ids, accept_len, committed, flags, req_status,
                        stream=None):
    rows, V, ld = _rows(target_logits)
    if rows != B * (depth + 1):
        raise ValueError("target_logits must hold B*(depth+1) rows")
    _call("dspark_verify_ratio", _ptr(target_logits), _dtype_code(target_logits), ld, int(B),
          int(depth), V, _i32(draft_tokens), _i32(counts), _i32(sparse_ids), _i32(nnz),
          int(top_k), int(seed) & (2 ** 64 - 1), _i32(request_ids), _i32(accept_len),
          _i32(committed), _i32(flags), _i32(req_status), _stream(stream))


def dspark_verify(target_logits, B, depth, draft_tokens, greedy_out=None, ratio_out=None,
                  counts=None, sparse_ids=None, nnz=None, top_k=0, seed=0, request_ids=None,
                  stream=None):
    """Both verification modes in one pass.  greedy_out = (accept_len,
    committed, status) or None; ratio_out = (accept_len, committed, flags,
    status) or None, with counts / sparse_ids / nnz / top_k / seed /
    request_ids as in dspark_verify_ratio."""
    rows, V, ld = _rows(target_logits)
    if rows != B * (depth + 1):
        raise ValueError("target_logits must hold B*(depth+1) rows")
    g = greedy_out or (None, None, None)
    r = ratio_out or (None, None, None, None)
    _call("dspark_verify", _ptr(target_logits), _dtype_code(target_logits), ld, int(B),
          int(depth), V, _i32(draft_tokens), _i32(counts), _i32(sparse_ids), _i32(nnz),
          int(top_k), int(seed) & (2 ** 64 - 1), _i32(request_ids), _i32(g[0]), _i32(g[1]),
          _i32(g[2]), _i32(r[0]), _i32(r[1]), _i32(r[2]), _i32(r[3]), _stream(stream))


def dspark_spec_step_noalloc(draft_logits, target_logits, B, depth, temperature, seed,
                             request_ids, counts, draft_tokens, row_status, greedy_out=None,
                             ratio_out=None, stream=None, schedule=0):
    """dspark_spec_step with the library's own device scratch array instead
    of a workspace (calls on one device must not overlap)."""
    rd, V, ld_d = _rows(draft_logits)
    rt, Vt, ld_t = _rows(target_logits)
    if rd != B * depth or rt != B * (depth + 1) or Vt != V:
        raise ValueError("draft_logits must hold B*depth rows and target_logits B*(depth+1) rows "
                         "of the same V")
    g = greedy_out or (None, None, None)
    r = ratio_out or (None, None, None, None)
    _call("dspark_spec_step_noalloc", _ptr(draft_logits), _dtype_code(draft_logits), ld_d,
          _ptr(target_logits), _dtype_code(target_logits), ld_t, int(B), int(depth), V,
          _ptr(temperature), int(seed) & (2 ** 64 - 1), _i32(request_ids), _i32(counts),
          _i32(draft_tokens), _i32(row_status), _i32(g[0]), _i32(g[1]), _i32(g[2]), _i32(r[0]),
          _i32(r[1]), _i32(r[2]), _i32(r[3]), int(schedule), _stream(stream))


def _host(t):
    if t is None:
        return None
    if t.is_cuda or not t.is_contiguous():
        raise ValueError("expected a contiguous host tensor")
    return ctypes.c_void_p(t.data_ptr())


def dspark_spec_step_host_staging_bytes(B, depth, V, draft_dtype, target_dtype):
    return int(_lib.load().dspark_spec_step_host_staging_bytes(int(B), int(depth), int(V),
                                                               int(draft_dtype), int(target_dtype)))


def dspark_spec_step_host(draft_logits, target_logits, B, depth, temperature, seed, request_ids,
                          draft_tokens, row_status, staging, greedy_out=None, ratio_out=None,
                          stream=None, schedule=0):
    """dspark_spec_step on host tensors (page-locked for asynchronous copies):
    draft_logits [B*depth, V] and target_logits [B*(depth+1), V] (float32 or
    bfloat16), temperature / request_ids (or None), host outputs; staging is
    a device uint8 tensor of dspark_spec_step_host_staging_bytes bytes."""
    V = draft_logits.shape[-1]
    if (draft_logits.numel() != B * depth * V or target_logits.numel() != B * (depth + 1) * V
            or target_logits.shape[-1] != V):
        raise ValueError("draft_logits must hold B*depth rows and target_logits B*(depth+1) rows "
                         "of the same V")
    g = greedy_out or (None, None, None)
    r = ratio_out or (None, None, None, None)
    _call("dspark_spec_step_host", _host(draft_logits), _dtype_code(draft_logits),
          _host(target_logits), _dtype_code(target_logits), int(B), int(depth), int(V),
          _host(temperature), int(seed) & (2 ** 64 - 1), _host(request_ids), _host(draft_tokens),
          _host(row_status), _host(g[0]), _host(g[1]), _host(g[2]), _host(r[0]), _host(r[1]),
          _host(r[2]), _host(r[3]), _ptr(staging), int(schedule), _stream(stream))


def dspark_spec_step_schedule(B, depth):
    """The schedule dspark_spec_step takes with SCHEDULE_AUTO (host only)."""
    rc = _lib.load().dspark_spec_step_schedule(int(B), int(depth))
    if rc < 0:
        raise ValueError("dspark_spec_step_schedule: error %d" % rc)
    return rc


def dspark_verify_match(target_logits, B, depth, draft_tokens, seed, request_ids, accept_len,
                        committed, flags, req_status, stream=None):
    rows, V, ld = _rows(target_logits)
    if rows != B * (depth + 1):
        raise ValueError("target_logits must hold B*(depth+1) rows")
    _call("dspark_verify_match", _ptr(target_logits), _dtype_code(target_logits), ld, int(B),
          int(depth), V, _i32(draft_tokens), int(seed) & (2 ** 64 - 1), _i32(request_ids),
          _i32(accept_len), _i32(committed), _i32(flags), _i32(req_status), _stream(stream))


def dspark_q_chain_sample(draft_logits, B, depth, temperature, bias, anchors, seed,
                          request_ids, workspace, counts, draft_tokens, row_status, margins=None,
                          stream=None):
    """draft_logits [B*depth, V] (or [B, depth, V]); bias [n_bias, V] fp32 or None;
    anchors int32 [B]; workspace unused (may be None)."""
    rows, V, ld = _rows(draft_logits)
    if rows != B * depth:
        raise ValueError("draft_logits must hold B*depth rows")
    nb, bld = (0, V) if bias is None else (bias.shape[0], bias.stride(0))
    _call("dspark_q_chain_sample", _ptr(draft_logits), _dtype_code(draft_logits), ld, int(B),
          int(depth), V, _ptr(temperature), _ptr(bias), bld, nb, _i32(anchors),
          int(seed) & (2 ** 64 - 1), _i32(request_ids), _ptr(workspace), _i32(counts),
          _i32(draft_tokens), _i32(row_status), _ptr(margins), _stream(stream))


def dspark_q_sharded_workspace_bytes(n_rows):
    return int(_lib.load().dspark_q_sharded_workspace_bytes(int(n_rows)))


def dspark_q_build_sample_sharded(draft_logits, B, depth, n_shards, temperature, top_k, seed,
                                  request_ids, counts, sparse_ids, nnz, draft_tokens, row_status,
                                  workspace, stream=None):
    rows, V, ld = _rows(draft_logits)
    if rows != B * depth:
        raise ValueError("draft_logits must hold B*depth rows")
    _call("dspark_q_build_sample_sharded", _ptr(draft_logits), _dtype_code(draft_logits), ld,
          int(B), int(depth), V, int(n_shards), _ptr(temperature), int(top_k),
          int(seed) & (2 ** 64 - 1), _i32(request_ids), _i32(counts), _i32(sparse_ids), _i32(nnz),
          _i32(draft_tokens), _i32(row_status), _ptr(workspace), _stream(stream))


def dspark_q_pack(counts, sparse_ids, nnz, top_k, V, q_out, checksum_out, stream=None):
    """counts [n_rows, V] (dense) or [n_rows, top_k] with sparse_ids / nnz;
    q_out float32 of the same shape; checksum_out int64 [n_rows] (holding the
    uint64 checksums)."""
    _call("dspark_q_pack", _i32(counts), _i32(sparse_ids), _i32(nnz), int(top_k),
          counts.shape[0], int(V), _ptr(q_out), _ptr(checksum_out), _stream(stream))


def dspark_q_validate(q, sparse_ids, nnz, top_k, V, tokens, expect, counts_out, row_status,
                      stream=None):
    """q float32 [n_rows, width]; tokens int32 [n_rows] or None; expect int64
    [n_rows] or None; counts_out int32 [n_rows, width] or None."""
    n_rows = q.shape[0]
    _call("dspark_q_validate", _ptr(q), _i32(sparse_ids), _i32(nnz), int(top_k), n_rows, int(V),
          _i32(tokens), _ptr(expect), _i32(counts_out), _i32(row_status), _stream(stream))


def dspark_verify_stats(flags, stats, stream=None):
    """flags: int32 / uint32 [B] (device); stats: int32 [3] (device)."""
    _call("dspark_verify_stats", _ptr(flags), int(flags.numel()), _ptr(stats), _stream(stream))


def dspark_target_probs(target_logits, p_out, argmax, row_status, stream=None):
    rows, V, ld = _rows(target_logits)
    _call("dspark_target_probs", _ptr(target_logits), _dtype_code(target_logits), ld, rows, V,
          _ptr(p_out), _i32(argmax), _i32(row_status), _stream(stream))


def dspark_spec_step(draft_logits, target_logits, B, depth, temperature, seed, request_ids, counts,
                     draft_tokens, row_status, greedy_out=None, ratio_out=None, workspace=None,
                     stream=None, schedule=0):
    """greedy_out = (accept_len, committed, status) or None; ratio_out =
    (accept_len, committed, flags, status) or None; workspace: >= B + 1 int32
    (allocated here when None); schedule: SCHEDULE_AUTO, SCHEDULE_ONE_LAUNCH
    or SCHEDULE_SEPARATE."""
    rd, V, ld_d = _rows(draft_logits)
    rt, Vt, ld_t = _rows(target_logits)
    if rd != B * depth or rt != B * (depth + 1) or Vt != V:
        raise ValueError("draft_logits must hold B*depth rows and target_logits B*(depth+1) rows "
                         "of the same V")
    g = greedy_out or (None, None, None)
    r = ratio_out or (None, None, None, None)
    if workspace is None:
        workspace = _empty((B + 1,), torch.int32, draft_logits.device)
    _call("dspark_spec_step", _ptr(draft_logits), _dtype_code(draft_logits), ld_d,
          _ptr(target_logits), _dtype_code(target_logits), ld_t, int(B), int(depth), V,
          _ptr(temperature), int(seed) & (2 ** 64 - 1), _i32(request_ids), _i32(counts),
          _i32(draft_tokens), _i32(row_status), _i32(g[0]), _i32(g[1]), _i32(g[2]), _i32(r[0]),
          _i32(r[1]), _i32(r[2]), _i32(r[3]), _i32(workspace), int(schedule), _stream(stream))


def _arg(name, t, dtype, shape):
    """The pointer of an optional contiguous CUDA tensor of this dtype and shape."""
    if t is None:
        return None
    if t.dtype is dtype and t.is_cuda and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    raise ValueError("%s must be a contiguous CUDA tensor of shape %s" % (name, tuple(shape)))


_HALF = {torch.bfloat16: BF16, torch.float16: F16}


def _cache_args(k_cache, v_cache):
    """(dtype code, k pointer, v pointer, block / token / head strides) of the two caches
    [n_blocks, page_size, n_heads, head_dim]: any strides, the same for both, the last one 1."""
    if k_cache.dtype not in _HALF or v_cache.dtype is not k_cache.dtype:
        raise TypeError("the caches must both be bfloat16 or float16")
    st = k_cache.stride()
    if (k_cache.dim() != 4 or v_cache.shape != k_cache.shape or v_cache.stride() != st
            or st[3] != 1):
        raise ValueError("the caches must be [n_blocks, page_size, n_heads, head_dim] of the same "
                         "shape and strides, contiguous in head_dim")
    if not (k_cache.is_cuda and v_cache.is_cuda):
        raise ValueError("expected a CUDA tensor")
    return _HALF[k_cache.dtype], k_cache.data_ptr(), v_cache.data_ptr(), st[0], st[1], st[2]


def dspark_cache_plan(ctx_len, new_len, max_new, page_size, block_table, free_blocks, n_free,
                      parents, slots, positions, tree_mask, taken, req_status, stream=None):
    """ctx_len / new_len / req_status int32 [B]; block_table int32 [B, max_blocks] (rows may be
    strided), updated in place; free_blocks int32 [max_free]; n_free int32 [1] or None; parents
    int32 [B, max_new] or None; slots int32 [B, max_new]; positions the same or None; tree_mask
    int64 [B, max_new] (holding the uint64 masks) or None; taken int32 [1]."""
    i32, cells = torch.int32, (ctx_len.shape[0], max_new)
    _cache_plan(ctx_len, new_len, max_new, page_size, block_table, free_blocks, n_free, parents,
                _arg("slots", slots, i32, cells), _arg("positions", positions, i32, cells),
                _arg("tree_mask", tree_mask, torch.int64, cells), _arg("taken", taken, i32, (1,)),
                _arg("req_status", req_status, i32, cells[:1]), stream)
    if not cells[0] and taken is not None:  # nothing is launched for an empty batch
        with torch.cuda.stream(stream):
            taken.zero_()


def _table_args(block_table, B):
    """(pointer, row stride, max_blocks) of a block table int32 [B, max_blocks]."""
    if (block_table.dtype is not torch.int32 or block_table.dim() != 2
            or block_table.shape[0] != B or block_table.stride(1) != 1
            or not block_table.is_cuda):
        raise ValueError("block_table must be an int32 CUDA tensor [B, max_blocks]")
    wide = block_table.shape[1]
    return block_table.data_ptr(), block_table.stride(0) if B > 1 else wide, wide


def _cache_plan(ctx_len, new_len, max_new, page_size, block_table, free_blocks, n_free, parents,
                slots, positions, tree_mask, taken, req_status, stream):
    """The call, with the outputs as pointers."""
    i32, B = torch.int32, ctx_len.shape[0]
    table, ld, wide = _table_args(block_table, B)
    n = free_blocks.shape[0]
    _call("dspark_cache_plan", _arg("ctx_len", ctx_len, i32, (B,)),
          _arg("new_len", new_len, i32, (B,)), B, max_new, page_size, table, ld, wide,
          _arg("free_blocks", free_blocks, i32, (n,)), n, _arg("n_free", n_free, i32, (1,)),
          _arg("parents", parents, i32, (B, max_new)), slots, positions, tree_mask, taken,
          req_status, _stream(stream))


def dspark_kv_write(k, v, k_cache, v_cache, slots, rows=None, stream=None):
    """k, v [.., n_heads, head_dim] (tokens uniformly strided; the same shape and strides), float32
    or the caches' type; k_cache, v_cache [n_blocks, page_size, n_heads, head_dim]; slots int32 of
    n_tokens; rows int32 of n_tokens or None (then n_tokens is the number of source tokens)."""
    code, kp, vp, sb, st, sh = _cache_args(k_cache, v_cache)
    if k.dim() < 3 or v.shape != k.shape or k.stride(-1) != 1 or v.stride(-1) != 1:
        raise ValueError("k and v must have the same shape [.., n_heads, head_dim], contiguous in "
                         "head_dim")
    if k.shape[-2:] != k_cache.shape[-2:]:
        raise ValueError("k and v must have the caches' heads and head_dim")
    if v.dtype is not k.dtype or (k.dtype is not torch.float32 and k.dtype is not k_cache.dtype):
        raise TypeError("k and v must be float32 or of the caches' type")
    if v.stride() != k.stride() and any(
            a != b and size > 1 for a, b, size in zip(k.stride(), v.stride(), k.shape)):
        raise ValueError("k and v must have the same strides")
    n, step = _uniform(k, k.dim() - 2, "the tokens of k and v")
    if not (k.is_cuda and v.is_cuda):
        raise ValueError("expected a CUDA tensor")
    if rows is None and slots.numel() != n:
        raise ValueError("slots must hold one slot for each token")
    _call("dspark_kv_write", k.data_ptr(), v.data_ptr(),
          F32 if k.dtype is torch.float32 else code, step,
          k.stride(-2) if k.shape[-2] > 1 else 0, n, k.shape[-2], k.shape[-1], kp, vp, code, sb,
          st, sh, k_cache.shape[0], k_cache.shape[1],
          _arg("slots", slots, torch.int32, slots.shape),
          _arg("rows", rows, torch.int32, slots.shape), slots.numel(), _stream(stream))


@functools.lru_cache(maxsize=256)
def dspark_tree_attention_workspace_bytes(B, nodes, n_heads, n_kv_heads, head_dim):
    return int(_lib.load().dspark_tree_attention_workspace_bytes(B, nodes, n_heads, n_kv_heads,
                                                                 head_dim))


def dspark_tree_attention(q, k_cache, v_cache, block_table, ctx_len, n_nodes, tree_mask, scale,
                          out, lse, req_status, workspace, stream=None):
    """q [B, nodes, n_heads, head_dim] (strided, contiguous in head_dim) of the caches' type;
    block_table int32 [B, max_blocks] (rows may be strided); ctx_len / n_nodes / req_status int32
    [B]; tree_mask int64 [B, nodes] (holding the uint64 masks) or None; out like q, contiguous;
    lse float32 [B, nodes, n_heads] or None; workspace: uint8, at least
    dspark_tree_attention_workspace_bytes bytes."""
    B, nodes, heads = q.shape[:3]
    need = dspark_tree_attention_workspace_bytes(B, nodes, heads, k_cache.shape[2], q.shape[3])
    if workspace.numel() * workspace.element_size() < need:
        raise ValueError("the workspace is too small")
    _tree_attention(q, k_cache, v_cache, block_table, ctx_len, n_nodes, tree_mask, scale,
                    _arg("out", out, q.dtype, q.shape),
                    _arg("lse", lse, torch.float32, (B, nodes, heads)),
                    _arg("req_status", req_status, torch.int32, (B,)), _ptr(workspace), stream)


def _tree_attention(q, k_cache, v_cache, block_table, ctx_len, n_nodes, tree_mask, scale, out,
                    lse, req_status, workspace, stream):
    """The call, with outputs and workspace as pointers."""
    code, kp, vp, sb, st, sh = _cache_args(k_cache, v_cache)
    i32, strides = torch.int32, q.stride()
    if q.dim() != 4 or q.dtype is not k_cache.dtype or strides[3] != 1 or not q.is_cuda:
        raise ValueError("q must be a CUDA tensor [B, nodes, n_heads, head_dim] of the caches' "
                         "type, contiguous in head_dim")
    B, nodes, heads, dim = q.shape
    n_blocks, page, kv_heads, kv_dim = k_cache.shape
    if kv_dim != dim:
        raise ValueError("q and the caches must have the same head_dim")
    table, ld, wide = _table_args(block_table, B)
    _call("dspark_tree_attention", q.data_ptr(), code, strides[0], strides[1], strides[2], B,
          nodes, heads, kv_heads, dim, kp, vp, sb, st, sh, n_blocks, page, table, ld, wide,
          _arg("ctx_len", ctx_len, i32, (B,)), _arg("n_nodes", n_nodes, i32, (B,)),
          _arg("tree_mask", tree_mask, torch.int64, (B, nodes)), scale, out, lse, req_status,
          workspace, _stream(stream))


def dspark_logits_process(logits, history, prompt_len, history_len, draft_tokens, row_mask,
                          repetition, frequency, presence, bias_ids, bias_values, n_bias,
                          mask_words, mask_rows, out, req_status, stream=None):
    """logits [B, rows, V] float32 or bfloat16, rows uniformly strided; out the same (or logits
    itself).  Optional (None): history int32 [B, history_ld] with history_len (and prompt_len)
    int32 [B]; draft_tokens int32 [B, n_drafts]; row_mask int64 [B, rows] (holding the uint64
    masks); repetition / frequency / presence float32 [B]; bias_ids int32 and bias_values float32
    [B, max_bias] with n_bias int32 [B]; mask_words int32 [n_masks, words] (rows may be strided)
    with mask_rows int32 [B, rows].  req_status int32 [B]."""
    if logits.dim() != 3 or out.shape != logits.shape or out.dtype is not logits.dtype:
        raise ValueError("logits must be [B, rows, V], and out of the same shape and type")
    n, V, ld = _rows(logits)
    ld_out = ld if out is logits else _rows(out)[2]
    B, rows = logits.shape[:2]
    i32, f32, one, per = torch.int32, torch.float32, (B,), (B, rows)
    wide = 0 if history is None else history.shape[-1]
    drafts = 0 if draft_tokens is None else draft_tokens.shape[-1]
    biases = 0 if bias_ids is None else bias_ids.shape[-1]
    if mask_words is None:
        wp, wld, n_masks = None, 0, 0
    else:
        n_masks, words = mask_words.shape
        if (mask_words.dtype not in (i32, torch.uint32) or mask_words.stride(1) != 1
                or not mask_words.is_cuda or words < (V + 31) // 32):
            raise ValueError("mask_words must be an int32 CUDA tensor [n_masks, ceil(V / 32)]")
        wp, wld = mask_words.data_ptr(), mask_words.stride(0) if n_masks > 1 else words
    _call("dspark_logits_process", _ptr(logits), _dtype_code(logits), ld if n > 1 else V, B, rows,
          V, _arg("history", history, i32, (B, wide)), wide,
          _arg("prompt_len", prompt_len, i32, one), _arg("history_len", history_len, i32, one),
          _arg("draft_tokens", draft_tokens, i32, (B, drafts)), drafts,
          _arg("row_mask", row_mask, torch.int64, per), _arg("repetition", repetition, f32, one),
          _arg("frequency", frequency, f32, one), _arg("presence", presence, f32, one),
          _arg("bias_ids", bias_ids, i32, (B, biases)),
          _arg("bias_values", bias_values, f32, (B, biases)), biases,
          _arg("n_bias", n_bias, i32, one), wp, wld, n_masks,
          _arg("mask_rows", mask_rows, i32, per), _ptr(out), ld_out if n > 1 else V,
          _arg("req_status", req_status, i32, one), _stream(stream))


# --------------------------------------------------- allocating helpers
def _on_stream(helper):
    """Runs an allocating helper with its `stream` as torch's current one, so that outputs and
    workspaces are that stream's memory: of another stream's they could be given to its next
    tensor while the kernels that write them are still to come.  (The helpers of a few us enter
    the stream themselves: this wrapper costs 0.3.)"""
    at = list(inspect.signature(helper).parameters).index("stream")

    @functools.wraps(helper)
    def call(*args, **kw):
        stream = args[at] if len(args) > at else kw.get("stream")
        if stream is None:
            return helper(*args, **kw)
        with torch.cuda.stream(stream):
            return helper(*args, **kw)

    return call


def _empty(shape, dtype, device):
    return torch.empty(shape, dtype=dtype, device=device)


@_on_stream
def q_build(draft_logits, temperature=None, top_k=0, stream=None):
    """draft_logits [..., V]; returns dict(counts, ids, nnz, status) (rows flattened)."""
    rows, V, _ = _rows(draft_logits)
    dev = draft_logits.device
    if top_k > 0:
        counts = _empty((rows, top_k), torch.int32, dev)
        ids = _empty((rows, top_k), torch.int32, dev)
        nnz = _empty((rows,), torch.int32, dev)
    else:
        counts = _empty((rows, V), torch.int32, dev)
        ids = nnz = None
    status = _empty((rows,), torch.int32, dev)
    dspark_q_build(draft_logits, temperature, top_k, counts, ids, nnz, status, stream)
    return {"counts": counts, "ids": ids, "nnz": nnz, "status": status, "top_k": top_k}


@_on_stream
def q_build_sample(draft_logits, B, depth, seed, temperature=None, top_k=0, request_ids=None,
                   stream=None):
    """Fused q build + draft draw; returns (q dict, tokens [B, depth])."""
    rows, V, _ = _rows(draft_logits)
    dev = draft_logits.device
    if top_k > 0:
        counts = _empty((rows, top_k), torch.int32, dev)
        ids = _empty((rows, top_k), torch.int32, dev)
        nnz = _empty((rows,), torch.int32, dev)
    else:
        counts = _empty((rows, V), torch.int32, dev)
        ids = nnz = None
    status = _empty((rows,), torch.int32, dev)
    tokens = _empty((B, depth), torch.int32, dev)
    dspark_q_build_sample(draft_logits, B, depth, temperature, top_k, seed, request_ids, counts,
                          ids, nnz, tokens, status, stream)
    return {"counts": counts, "ids": ids, "nnz": nnz, "status": status, "top_k": top_k}, tokens


@_on_stream
def spec_step(draft_logits, target_logits, B, depth, seed, temperature=None, request_ids=None,
              modes=("greedy", "ratio"), stream=None, schedule=0):
    """Fused q build + draft draw + verification (dense q).  Returns (q dict,
    tokens [B, depth], {mode: outputs as verify_greedy / verify_ratio})."""
    rows, V, _ = _rows(draft_logits)
    dev = draft_logits.device
    counts = _empty((rows, V), torch.int32, dev)
    status = _empty((rows,), torch.int32, dev)
    tokens = _empty((B, depth), torch.int32, dev)
    outs = {}
    if "greedy" in modes:
        outs["greedy"] = (_empty((B,), torch.int32, dev), _empty((B, depth + 1), torch.int32, dev),
                          _empty((B,), torch.int32, dev))
    if "ratio" in modes:
        outs["ratio"] = (_empty((B,), torch.int32, dev), _empty((B, depth + 1), torch.int32, dev),
                         _empty((B,), torch.int32, dev), _empty((B,), torch.int32, dev))
    dspark_spec_step(draft_logits, target_logits, B, depth, temperature, seed, request_ids, counts,
                     tokens, status, outs.get("greedy"), outs.get("ratio"), stream=stream,
                     schedule=schedule)
    q = {"counts": counts, "ids": None, "nnz": None, "status": status, "top_k": 0}
    return q, tokens, outs


@_on_stream
def verify_match(target_logits, draft_tokens, seed, request_ids=None, stream=None):
    """Stochastic verification; returns (accept_len, committed, flags, status)."""
    B, depth = draft_tokens.shape
    dev = target_logits.device
    acc = _empty((B,), torch.int32, dev)
    com = _empty((B, depth + 1), torch.int32, dev)
    fl = _empty((B,), torch.int32, dev)
    st = _empty((B,), torch.int32, dev)
    dspark_verify_match(target_logits, B, depth, draft_tokens, seed, request_ids, acc, com, fl, st,
                        stream)
    return acc, com, fl, st


@_on_stream
def q_chain_sample(draft_logits, B, depth, seed, anchors, bias=None, temperature=None,
                   request_ids=None, stream=None):
    """The Markov-conditioned draft chain; returns (q dict, tokens [B, depth],
    margins [B, depth])."""
    rows, V, _ = _rows(draft_logits)
    dev = draft_logits.device
    counts = _empty((rows, V), torch.int32, dev)
    status = _empty((rows,), torch.int32, dev)
    tokens = _empty((B, depth), torch.int32, dev)
    margins = _empty((B, depth), torch.float32, dev)
    dspark_q_chain_sample(draft_logits, B, depth, temperature, bias, anchors, seed, request_ids,
                          None, counts, tokens, status, margins, stream)
    q = {"counts": counts, "ids": None, "nnz": None, "status": status, "top_k": 0}
    return q, tokens, margins


@_on_stream
def q_build_sample_sharded(draft_logits, B, depth, n_shards, seed, temperature=None, top_k=0,
                           request_ids=None, stream=None):
    """The vocabulary-sharded emulation of q_build_sample."""
    rows, V, _ = _rows(draft_logits)
    dev = draft_logits.device
    ws = _empty((dspark_q_sharded_workspace_bytes(rows),), torch.uint8, dev)
    if top_k > 0:
        counts = _empty((rows, top_k), torch.int32, dev)
        ids = _empty((rows, top_k), torch.int32, dev)
        nnz = _empty((rows,), torch.int32, dev)
    else:
        counts = _empty((rows, V), torch.int32, dev)
        ids = nnz = None
    status = _empty((rows,), torch.int32, dev)
    tokens = _empty((B, depth), torch.int32, dev)
    dspark_q_build_sample_sharded(draft_logits, B, depth, n_shards, temperature, top_k, seed,
                                  request_ids, counts, ids, nnz, tokens, status, ws, stream)
    return {"counts": counts, "ids": ids, "nnz": nnz, "status": status, "top_k": top_k}, tokens


@_on_stream
def q_pack(q, V, stream=None):
    """Wire form of a q dict from q_build: (q float32 of the counts' shape,
    checksums int64 [n_rows] holding the uint64 bit patterns)."""
    counts = q["counts"]
    qf = _empty(counts.shape, torch.float32, counts.device)
    cs = _empty((counts.shape[0],), torch.int64, counts.device)
    dspark_q_pack(counts, q["ids"], q["nnz"], q["top_k"], V, qf, cs, stream)
    return qf, cs


@_on_stream
def q_validate(qf, V, ids=None, nnz=None, top_k=0, tokens=None, expect=None, stream=None):
    """Validation of received q rows: (status int32 [n_rows], recovered counts
    int32 of qf's shape)."""
    counts = _empty(qf.shape, torch.int32, qf.device)
    st = _empty((qf.shape[0],), torch.int32, qf.device)
    dspark_q_validate(qf, ids, nnz, top_k, V, tokens, expect, counts, st, stream)
    return st, counts


@_on_stream
def draft_sample(q, B, depth, V, seed, request_ids=None, stream=None):
    dev = q["counts"].device
    tokens = _empty((B * depth,), torch.int32, dev)
    status = _empty((B * depth,), torch.int32, dev)
    dspark_draft_sample(q["counts"], q["ids"], q["nnz"], q["top_k"], B, depth, V, seed,
                        request_ids, tokens, status, stream)
    return tokens.view(B, depth), status.view(B, depth)


@_on_stream
def verify_greedy(target_logits, drafts, stream=None):
    B, depth = drafts.shape
    dev = target_logits.device
    acc = _empty((B,), torch.int32, dev)
    com = _empty((B, depth + 1), torch.int32, dev)
    st = _empty((B,), torch.int32, dev)
    dspark_verify_greedy(target_logits, B, depth, drafts, acc, com, st, stream)
    return acc, com, st


@_on_stream
def verify_ratio(target_logits, drafts, q, seed, request_ids=None, stream=None):
    B, depth = drafts.shape
    dev = target_logits.device
    acc = _empty((B,), torch.int32, dev)
    com = _empty((B, depth + 1), torch.int32, dev)
    fl = _empty((B,), torch.int32, dev)
    st = _empty((B,), torch.int32, dev)
    dspark_verify_ratio(target_logits, B, depth, drafts, q["counts"], q["ids"], q["nnz"],
                        q["top_k"], seed, request_ids, acc, com, fl, st, stream)
    return acc, com, fl, st


@_on_stream
def verify_stats(flags, stream=None):
    """Counts of the requests with each DSPARK_FLAG_* bit in flags [B]: a
    tensor [3] (ambiguous decisions, draws near a boundary, degenerate
    residuals)."""
    stats = _empty((3,), torch.int32, flags.device)
    dspark_verify_stats(flags, stats, stream)
    return stats


@_on_stream
def target_probs(target_logits, want_p=True, stream=None):
    rows, V, _ = _rows(target_logits)
    dev = target_logits.device
    p = _empty((rows, V), torch.float32, dev) if want_p else None
    am = _empty((rows,), torch.int32, dev)
    st = _empty((rows,), torch.int32, dev)
    dspark_target_probs(target_logits, p, am, st, stream)
    return p, am, st


def cache_plan(ctx_len, new_len, max_new, page_size, block_table, free_blocks, n_free=None,
               parents=None, stream=None):
    """Grants the step's blocks and maps its new tokens; returns dict(block_table (the caller's,
    updated), slots, positions [B, max_new], taken [1], status [B]) and, for max_new <= 64,
    tree_mask int64 [B, max_new]."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return cache_plan(ctx_len, new_len, max_new, page_size, block_table, free_blocks,
                              n_free, parents)
    B, dev, i32 = ctx_len.shape[0], ctx_len.device, torch.int32
    slots, taken, status = (_empty((B, max_new), i32, dev), _empty((1,), i32, dev),
                            _empty((B,), i32, dev))
    positions = torch.empty_like(slots)
    mask = _empty((B, max_new), torch.int64, dev) if max_new <= MAX_NODES else None
    _cache_plan(ctx_len, new_len, max_new, page_size, block_table, free_blocks, n_free, parents,
                slots.data_ptr(), positions.data_ptr(), None if mask is None else mask.data_ptr(),
                taken.data_ptr(), status.data_ptr(), stream)
    if not B:
        taken.zero_()
    out = {"block_table": block_table, "slots": slots, "positions": positions, "taken": taken,
           "status": status}
    if mask is not None:
        out["tree_mask"] = mask
    return out


def kv_write(k, v, k_cache, v_cache, slots, rows=None, stream=None):
    """Writes tokens' keys and values into their slots; returns the two caches."""
    dspark_kv_write(k, v, k_cache, v_cache, slots, rows, stream)
    return k_cache, v_cache


def tree_attention(q, k_cache, v_cache, block_table, ctx_len, n_nodes, tree_mask=None, scale=None,
                   stream=None):
    """Attention of the nodes over the cache (scale 1 / sqrt(head_dim) when None); returns (out
    like q, lse [B, nodes, n_heads], status [B])."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return tree_attention(q, k_cache, v_cache, block_table, ctx_len, n_nodes, tree_mask,
                                  scale)
    B, nodes, heads, dim = q.shape
    dev = q.device
    out = _empty((B, nodes, heads, dim), q.dtype, dev)
    lse = _empty((B, nodes, heads), torch.float32, dev)
    st = _empty((B,), torch.int32, dev)
    ws = _empty((dspark_tree_attention_workspace_bytes(B, nodes, heads, k_cache.shape[2], dim),),
                torch.uint8, dev)
    _tree_attention(q, k_cache, v_cache, block_table, ctx_len, n_nodes, tree_mask,
                    dim ** -0.5 if scale is None else scale, out.data_ptr(), lse.data_ptr(),
                    st.data_ptr(), ws.data_ptr(), stream)
    return out, lse, st


def logits_process(logits, history=None, prompt_len=None, history_len=None, draft_tokens=None,
                   row_mask=None, repetition=None, frequency=None, presence=None, bias_ids=None,
                   bias_values=None, n_bias=None, mask_words=None, mask_rows=None, out=None,
                   stream=None):
    """Penalties, biases and grammar masks on logits [B, rows, V]; returns (out (a new tensor when
    None; logits itself for in place), status [B])."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return logits_process(logits, history, prompt_len, history_len, draft_tokens, row_mask,
                                  repetition, frequency, presence, bias_ids, bias_values, n_bias,
                                  mask_words, mask_rows, out)
    if out is None:
        out = _empty(logits.shape, logits.dtype, logits.device)
    st = _empty((logits.shape[0],), torch.int32, logits.device)
    dspark_logits_process(logits, history, prompt_len, history_len, draft_tokens, row_mask,
                          repetition, frequency, presence, bias_ids, bias_values, n_bias,
                          mask_words, mask_rows, out, st, stream)
    return out, st
