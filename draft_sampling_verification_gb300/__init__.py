"""GB300 draft sampling and verification (dyadic24-standard-v1).

Thin Python binding of the C ABI in ``include/dspark.h``: the functions named
like the C calls (``dspark_q_build``, ``dspark_draft_sample``,
``dspark_verify_greedy``, ``dspark_verify_ratio``, ``dspark_target_probs``,
``dspark_cache_plan``, ``dspark_kv_write``, ``dspark_tree_attention``,
``dspark_logits_process``, ``dspark_qk_rotate``, ``dspark_rotate_write``,
``dspark_latent_write``, ``dspark_latent_attention``)
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
ROPE_PLAIN, ROPE_LINEAR, ROPE_PARTS = 0, 1, 2
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
           "dspark_logits_process", "logits_process", "dspark_rope_table", "rope_table",
           "dspark_qk_rotate", "qk_rotate", "dspark_rotate_write", "rotate_write",
           "dspark_latent_write", "latent_write", "dspark_latent_attention",
           "dspark_latent_attention_workspace_bytes", "latent_attention"]


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


def dspark_rope_table(rot_dim, base, scaling, factor, original_len, low, high, inv_freq, table):
    """table: host int64 [rot_dim / 2] (holding the uint64 turns); inv_freq: host float64
    [rot_dim / 2] or None.  The one call that needs no GPU."""
    pairs = (rot_dim // 2,)
    for name, t, dtype in (("inv_freq", inv_freq, torch.float64), ("table", table, torch.int64)):
        if t is not None and (t.dtype is not dtype or tuple(t.shape) != pairs):
            raise ValueError("%s must be %s of shape %s" % (name, dtype, pairs))
    _call("dspark_rope_table", int(rot_dim), float(base), int(scaling), float(factor),
          float(original_len), float(low), float(high), _host(inv_freq), _host(table))


def _here(*tensors):
    """Refuses tensors of another device than the current one, which the calls launch on.  Given
    every tensor of a call, outputs and workspace among them: the kernels get bare pointers."""
    device = torch._C._cuda_getDevice()
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError("tensors must be on the current CUDA device")


_ELEMENTS = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}


def _head_args(name, t):
    """(dtype code, pointer, token stride, head stride, tokens, heads, head_dim) of a tensor
    [.., n_heads, head_dim] whose tokens are uniformly strided."""
    code, shape, strides = _ELEMENTS.get(t.dtype), t.shape, t.stride()
    if code is None:
        raise TypeError("%s must be float32, bfloat16 or float16, got %s" % (name, t.dtype))
    if len(shape) < 3 or (strides[-1] != 1 and shape[-1] > 1) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor [.., n_heads, head_dim], contiguous in head_dim"
                         % name)
    heads, dim = shape[-2:]
    if len(shape) == 3:
        n, step = shape[0], strides[0]
    else:
        n, step = _uniform(t, len(shape) - 2, "the tokens of " + name)
    return code, t.data_ptr(), step if n > 1 else 0, strides[-2] if heads > 1 else 0, n, heads, dim


def _written(name, t, heads):
    """Refuses an output whose elements share a place, by the arguments of _head_args."""
    _, _, token, head, n, n_heads, dim = heads
    (near, few), (far, many) = sorted(((head, n_heads), (token, n)))
    shared = few > 0 < many and ((few > 1 and near < dim) or (many > 1 and far < dim))
    if not shared and few > 1 < many:
        # i steps of the farther dimension, as many as steps of the nearer one can lead back from
        for i in range(1, min(many, ((few - 1) * near + dim - 1) // far + 1)):
            j = i * far // near
            shared = shared or any(k < few and abs(i * far - k * near) < dim for k in (j, j + 1))
    if shared:
        raise ValueError("the tokens and heads of %s must not overlap" % name)


def _table_arg(table, rot_start):
    """(pointer, rot_start, rot_dim) of a rotation's table (None: no rotation)."""
    if table is None:
        return None, 0, 0
    return _arg("table", table, torch.int64, table.shape), rot_start, 2 * table.numel()


def _fresh(t, dtype):
    """A new tensor for the output of t, and its _head_args: whole rows one after the other."""
    out = torch.empty(t.shape, dtype=dtype, device=t.device)
    heads, dim = t.shape[-2:]
    return out, (_ELEMENTS.get(dtype), out.data_ptr(), heads * dim, dim, None, heads, dim)


_NONE = (0, None, 0, 0, 0, 0, 0)


def dspark_qk_rotate(q, k, positions, table, q_weight, k_weight, eps, rot_start, interleaved,
                     magnitude, q_out, k_out, stream=None):
    """q, k [.., n_heads, head_dim] (either may be None, with its output) of one type, with the
    same tokens and head_dim; positions int32 of n_tokens; table int64 [rot_dim / 2] of
    rope_table, on the device, or None (norms alone); weights float32 [head_dim] or None; q_out,
    k_out like q, k in shape, of one type: the sources' or, for float32 sources, a 16-bit one."""
    outs = []
    for name, t, o in (("q_out", q, q_out), ("k_out", k, k_out)):
        if t is None:
            outs.append(_NONE)
            continue
        _here(o)
        outs.append(_head_args(name, o))
        if o.shape != t.shape:
            raise ValueError("%s must have its source's shape" % name)
        _written(name, o, outs[-1])
    if q is not None and k is not None and outs[0][0] != outs[1][0]:
        raise TypeError("q_out and k_out must have the same type")
    _qk_rotate(q, k, positions, table, q_weight, k_weight, eps, rot_start, interleaved, magnitude,
               *outs, stream)


def _qk_rotate(q, k, positions, table, q_weight, k_weight, eps, rot_start, interleaved, magnitude,
               q_out, k_out, stream):
    """The call, with the outputs as _head_args."""
    a, b = (_NONE if t is None else _head_args(n, t) for n, t in (("q", q), ("k", k)))
    some, code = (a, q_out[0]) if q is not None else (b, k_out[0])
    if some is _NONE:
        raise ValueError("q or k is needed")
    if q is not None and k is not None and (a[0] != b[0] or a[4] != b[4] or a[6] != b[6]):
        raise ValueError("q and k must have the same type, tokens and head_dim")
    _here(q, k, positions, table, q_weight if q is not None else None,
          k_weight if k is not None else None)
    n, dim = some[4], some[6]
    tp, start, rot = _table_arg(table, rot_start)
    _call("dspark_qk_rotate", a[1], b[1], some[0], a[2], a[3], b[2], b[3], n, a[5], b[5], dim,
          _arg("q_weight", q_weight, torch.float32, (dim,)),
          _arg("k_weight", k_weight, torch.float32, (dim,)), eps,
          _positions(positions, n), tp, start, rot, interleaved, magnitude, q_out[1], q_out[2],
          q_out[3], k_out[1], k_out[2], k_out[3], code, _stream(stream))


def _positions(positions, n):
    if positions.numel() != n:
        raise ValueError("positions must hold one position for each token")
    return _arg("positions", positions, torch.int32, positions.shape)


def dspark_rotate_write(q, k, v, positions, table, k_cache, v_cache, slots, rows, q_weight,
                        k_weight, eps, rot_start, interleaved, magnitude, q_out, stream=None):
    """q [.., n_heads, head_dim] or None (with q_out), k, v [.., n_kv_heads, head_dim] of the same
    strides, all float32 or the caches' type; positions, slots int32 of n_tokens; rows int32 of
    n_tokens (q None) or None (then n_tokens is the number of tokens of k, and of q); the caches as
    in dspark_kv_write; q_out like q, of the caches' type; the rest as in dspark_qk_rotate."""
    o = _NONE
    if q is not None:
        _here(q_out)
        o = _head_args("q_out", q_out)
        if q_out.shape != q.shape:
            raise ValueError("q_out must have q's shape")
        _written("q_out", q_out, o)
    _rotate_write(q, k, v, positions, table, k_cache, v_cache, slots, rows, q_weight, k_weight, eps,
                  rot_start, interleaved, magnitude, o, stream)


def _rotate_write(q, k, v, positions, table, k_cache, v_cache, slots, rows, q_weight, k_weight, eps,
                  rot_start, interleaved, magnitude, q_out, stream):
    """The call, with q_out as _head_args."""
    code, kp, vp, sb, st, sh = _cache_args(k_cache, v_cache)
    x = _head_args("k", k)
    if v.shape != k.shape or v.dtype is not k.dtype or not v.is_cuda:
        raise ValueError("k and v must be CUDA tensors of the same shape and type")
    if v.stride() != k.stride() and any(
            i != j and size > 1 for i, j, size in zip(k.stride(), v.stride(), k.shape)):
        raise ValueError("k and v must have the same strides")
    _here(q, k, v, k_cache, v_cache, positions, table, slots, rows, k_weight,
          q_weight if q is not None else None)
    n_blocks, page, kv_heads, dim = k_cache.shape
    if x[5] != kv_heads or x[6] != dim:
        raise ValueError("k and v must have the caches' heads and head_dim")
    if x[0] != F32 and x[0] != code:
        raise TypeError("q, k and v must be float32 or of the caches' type")
    n = slots.numel()
    if rows is None and n != x[4]:
        raise ValueError("slots must hold one slot for each token")
    a = _NONE
    if q is not None:
        a = _head_args("q", q)
        if a[0] != x[0] or a[4] != n or a[6] != dim:
            raise ValueError("q and k must have the same type, tokens and head_dim")
        if q_out[0] != code:
            raise ValueError("q_out must have the caches' type")
    tp, start, rot = _table_arg(table, rot_start)
    _call("dspark_rotate_write", a[1], x[1], v.data_ptr(), x[0], a[2], a[3], x[2], x[3], x[4],
          a[5], kv_heads, dim, _arg("q_weight", q_weight, torch.float32, (dim,)),
          _arg("k_weight", k_weight, torch.float32, (dim,)), eps, _positions(positions, n), tp,
          start, rot, interleaved, magnitude, q_out[1], q_out[2], q_out[3], kp, vp, code, sb, st,
          sh, n_blocks, page, _arg("slots", slots, torch.int32, slots.shape),
          _arg("rows", rows, torch.int32, slots.shape), n, _stream(stream))


def _latent_cache_args(cache):
    """(dtype code, pointer, block stride, token stride) of a cache [n_blocks, page_size, width]."""
    if cache.dtype not in _HALF:
        raise TypeError("the cache must be bfloat16 or float16")
    if cache.dim() != 3 or cache.stride(2) != 1 or not cache.is_cuda:
        raise ValueError("the cache must be a CUDA tensor [n_blocks, page_size, latent_dim + "
                         "rope_dim], contiguous in its last dimension")
    blocks, page, width = cache.shape
    # a dimension of one element may have any stride
    token = cache.stride(1) if page > 1 else width
    return (_HALF[cache.dtype], cache.data_ptr(),
            cache.stride(0) if blocks > 1 else max(token, page * token), token)


def _token_args(name, t):
    """(pointer, token stride, tokens, width) of a tensor [.., width] of uniformly strided tokens."""
    if t.dim() < 2 or (t.stride(-1) != 1 and t.shape[-1] > 1) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor [.., width], contiguous in its last dimension"
                         % name)
    n, step = _uniform(t, t.dim() - 1, "the tokens of " + name)
    return t.data_ptr(), step, n, t.shape[-1]


def dspark_latent_write(c, k_rope, positions, table, cache, slots, rows, weight, eps, interleaved,
                        magnitude, stream=None):
    """c [.., latent_dim] and k_rope [.., rope_dim] (None: rope_dim 0) of the same tokens, float32
    or the cache's type; cache [n_blocks, page_size, latent_dim + rope_dim]; positions, slots int32
    of n_tokens; rows int32 of n_tokens or None (then n_tokens is the number of source tokens);
    table int64 [rope_dim / 2] of rope_table, on the device; weight float32 [latent_dim] or None."""
    code, cp, sb, st = _latent_cache_args(cache)
    p, step, n_src, latent = _token_args("c", c)
    rp, r_step, rope = None, 0, 0
    if k_rope is not None:
        rp, r_step, n_rope, rope = _token_args("k_rope", k_rope)
        if n_rope != n_src or k_rope.dtype is not c.dtype:
            raise ValueError("c and k_rope must have the same tokens and type")
        if table is None or 2 * table.numel() != rope:
            raise ValueError("table must hold one entry for each pair of k_rope")
    _here(c, k_rope, cache, positions, table, slots, rows, weight)
    if c.dtype is not torch.float32 and c.dtype is not cache.dtype:
        raise TypeError("c must be float32 or of the cache's type")
    if cache.shape[2] != latent + rope:
        raise ValueError("the cache's rows must hold c and k_rope")
    n = slots.numel()
    if rows is None and n != n_src:
        raise ValueError("slots must hold one slot for each token")
    _call("dspark_latent_write", p, step, rp, r_step, _ELEMENTS[c.dtype], n_src, latent, rope,
          _arg("weight", weight, torch.float32, (latent,)), eps, _positions(positions, n),
          _table_arg(table, 0)[0] if rope else None, int(interleaved), magnitude, cp, code, sb, st,
          cache.shape[0], cache.shape[1], _arg("slots", slots, torch.int32, slots.shape),
          _arg("rows", rows, torch.int32, slots.shape), n, _stream(stream))


@functools.lru_cache(maxsize=256)
def dspark_latent_attention_workspace_bytes(B, nodes, n_heads, latent_dim):
    return int(_lib.load().dspark_latent_attention_workspace_bytes(B, nodes, n_heads, latent_dim))


def dspark_latent_attention(q, cache, block_table, ctx_len, n_nodes, latent_dim, tree_mask, scale,
                            out, lse, req_status, workspace, stream=None):
    """q [B, nodes, n_heads, latent_dim + rope_dim] (strided, contiguous in its last dimension) of
    the cache's type; cache [n_blocks, page_size, latent_dim + rope_dim]; out [B, nodes, n_heads,
    latent_dim] and lse float32 [B, nodes, n_heads] (or None) contiguous; workspace: uint8, at
    least dspark_latent_attention_workspace_bytes bytes; the rest as in dspark_tree_attention."""
    B, nodes, heads = q.shape[:3]
    need = dspark_latent_attention_workspace_bytes(B, nodes, heads, latent_dim)
    if workspace.numel() * workspace.element_size() < need:
        raise ValueError("the workspace is too small")
    _here(out, lse, req_status, workspace)
    _latent_attention(q, cache, block_table, ctx_len, n_nodes, latent_dim, tree_mask, scale,
                      _arg("out", out, q.dtype, (B, nodes, heads, latent_dim)),
                      _arg("lse", lse, torch.float32, (B, nodes, heads)),
                      _arg("req_status", req_status, torch.int32, (B,)), _ptr(workspace), stream)


def _latent_attention(q, cache, block_table, ctx_len, n_nodes, latent_dim, tree_mask, scale, out,
                      lse, req_status, workspace, stream):
    """The call, with outputs and workspace as pointers."""
    code, cp, sb, st = _latent_cache_args(cache)
    i32, strides = torch.int32, q.stride()
    if q.dim() != 4 or q.dtype is not cache.dtype or strides[3] != 1 or not q.is_cuda:
        raise ValueError("q must be a CUDA tensor [B, nodes, n_heads, latent_dim + rope_dim] of "
                         "the cache's type, contiguous in its last dimension")
    _here(q, cache, block_table, ctx_len, n_nodes, tree_mask)
    B, nodes, heads, width = q.shape
    n_blocks, page, row = cache.shape
    if row != width:
        raise ValueError("q and the cache's rows must have the same width")
    # a dimension of one element may have any stride
    req, node, head = (st if n > 1 else width for st, n in zip(strides, q.shape[:3]))
    table, ld, wide = _table_args(block_table, B)
    _call("dspark_latent_attention", q.data_ptr(), code, req, node, head, B, nodes, heads,
          latent_dim, width - latent_dim, cp, sb, st, n_blocks, page, table, ld, wide,
          _arg("ctx_len", ctx_len, i32, (B,)), _arg("n_nodes", n_nodes, i32, (B,)),
          _arg("tree_mask", tree_mask, torch.int64, (B, nodes)), scale, out, lse, req_status,
          workspace, _stream(stream))


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


_SCALINGS = {None: ROPE_PLAIN, "linear": ROPE_LINEAR, "parts": ROPE_PARTS}


def rope_table(rot_dim, base=10000.0, scaling=None, factor=1.0, original_len=1.0, low=1.0,
               high=32.0, inv_freq=None, device=None):
    """The table of a rotation of rot_dim elements, int64 [rot_dim / 2] on the device (the current
    CUDA device when None), made once and kept.  scaling: None, "linear" or "parts" (linear in the
    turns over original_len; models whose ramp is linear in the pair's index give inv_freq); inv_freq:
    radians a position, a sequence or a tensor, in place of base's."""
    if scaling not in _SCALINGS:
        raise ValueError("scaling must be None, 'linear' or 'parts', got %r" % (scaling,))
    if inv_freq is not None:
        inv_freq = torch.as_tensor(inv_freq).detach().to("cpu", torch.float64).contiguous()
    table = torch.empty((rot_dim // 2,), dtype=torch.int64)
    dspark_rope_table(rot_dim, base, _SCALINGS[scaling], factor, original_len, low, high, inv_freq,
                      table)
    return table.to("cuda" if device is None else device)


def qk_rotate(q, k, positions, table, q_weight=None, k_weight=None, eps=1e-6, rot_start=0,
              interleaved=False, magnitude=1.0, out=None, stream=None):
    """Norms (with weights) and rotates queries and keys [.., n_heads, head_dim] (either may be
    None) by their tokens' positions; returns (q_out, k_out): new tensors, or the pair `out`, which
    may be (q, k) themselves."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return qk_rotate(q, k, positions, table, q_weight, k_weight, eps, rot_start,
                             interleaved, magnitude, out)
    if out is None:
        (a, x), (b, y) = ((None, _NONE) if t is None else _fresh(t, t.dtype) for t in (q, k))
        _qk_rotate(q, k, positions, table, q_weight, k_weight, eps, rot_start, interleaved,
                   magnitude, x, y, stream)
        return a, b
    dspark_qk_rotate(q, k, positions, table, q_weight, k_weight, eps, rot_start, interleaved,
                     magnitude, out[0], out[1], stream)
    return out[0], out[1]


def rotate_write(q, k, v, positions, table, k_cache, v_cache, slots, rows=None, q_weight=None,
                 k_weight=None, eps=1e-6, rot_start=0, interleaved=False, magnitude=1.0, out=None,
                 stream=None):
    """qk_rotate whose keys go to their slots of the cache, with the values; returns (q_out (a new
    tensor of the caches' type, `out`, or None without q), k_cache, v_cache)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return rotate_write(q, k, v, positions, table, k_cache, v_cache, slots, rows, q_weight,
                                k_weight, eps, rot_start, interleaved, magnitude, out)
    if out is None:
        out, o = (None, _NONE) if q is None else _fresh(q, k_cache.dtype)
        _rotate_write(q, k, v, positions, table, k_cache, v_cache, slots, rows, q_weight, k_weight,
                      eps, rot_start, interleaved, magnitude, o, stream)
    else:
        dspark_rotate_write(q, k, v, positions, table, k_cache, v_cache, slots, rows, q_weight,
                            k_weight, eps, rot_start, interleaved, magnitude, out, stream)
    return out, k_cache, v_cache


def latent_write(c, k_rope, positions, table, cache, slots, rows=None, weight=None, eps=1e-6,
                 interleaved=False, magnitude=1.0, stream=None):
    """Writes tokens' normed latent vectors and rotated parts into their slots; returns the cache."""
    dspark_latent_write(c, k_rope, positions, table, cache, slots, rows, weight, eps, interleaved,
                        magnitude, stream)
    return cache


def latent_attention(q, cache, block_table, ctx_len, n_nodes, latent_dim, scale, tree_mask=None,
                     stream=None):
    """Attention of the nodes over a latent cache, absorbed form; returns (out [B, nodes, n_heads,
    latent_dim], lse [B, nodes, n_heads], status [B])."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return latent_attention(q, cache, block_table, ctx_len, n_nodes, latent_dim, scale,
                                    tree_mask)
    B, nodes, heads = q.shape[:3]
    dev = q.device
    out = _empty((B, nodes, heads, latent_dim), q.dtype, dev)
    lse = _empty((B, nodes, heads), torch.float32, dev)
    st = _empty((B,), torch.int32, dev)
    ws = _empty((dspark_latent_attention_workspace_bytes(B, nodes, heads, latent_dim),),
                torch.uint8, dev)
    _latent_attention(q, cache, block_table, ctx_len, n_nodes, latent_dim, tree_mask, scale,
                      out.data_ptr(), lse.data_ptr(), st.data_ptr(), ws.data_ptr(), stream)
    return out, lse, st
