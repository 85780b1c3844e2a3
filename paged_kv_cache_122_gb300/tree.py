"""Torch-facing binding of tree verification and cross attention
(``include/pagedkv_tree.h``).

A step over trees of drafted tokens: append the nodes (``rope_and_cache``), attend
(``paged_attention_tree``), find the path the target model agrees with
(``accept_tree``), move its rows together (``keep_tokens``, or all layers at once
with ``pk_keep_tokens_layers``) and give the pages behind them back
(``BlockManager.truncate``).  As in ``api``, every function marshals arguments into
one C call; names follow the C entry points, and the unprefixed names are the same
calls.
"""
from __future__ import annotations

import functools
from typing import Optional, Tuple

import torch

from . import _native
from ._native import check, load
from .api import _at, _empty_like, _layers, _need, _on, _raw_stream
from .fp8 import _NOTHING, _bound, _workspace

_MAX_TREE = 8192        # nodes of a tree in pk_accept_tree


@functools.lru_cache(maxsize=256)
def pk_tree_workspace_bytes(num_heads: int, num_kv_heads: int, head_dim: int, max_q_len: int, max_seq_len: int) -> int:
    return int(load().pk_tree_workspace_bytes(num_heads, num_kv_heads, head_dim, max_q_len, max_seq_len))


def _args(q, cu_q_lens, max_q_len, k_cache, v_cache, block_tables, seq_lens, scale, out_dtype, max_seq_len, out,
          workspace, stream):
    """Checks what the two attention calls share; returns the output and the
    arguments before and after the mask."""
    dev = q.device
    _need(q, "q", torch.bfloat16, 3)
    _need(cu_q_lens, "cu_q_lens", torch.int32, 1, dev)
    _need(k_cache, "k_cache", torch.bfloat16, 4, dev)
    _need(v_cache, "v_cache", torch.bfloat16, 4, dev)
    _need(block_tables, "block_tables", torch.int32, 2, dev)
    _need(seq_lens, "seq_lens", torch.int32, 1, dev)
    T, H, D = shape = q.shape
    P, B, Hkv, Dk = pool = k_cache.shape
    N, MB = block_tables.shape
    if v_cache.shape != pool or Dk != D:
        raise ValueError("k_cache / v_cache / q shapes disagree")
    if seq_lens.numel() != N or cu_q_lens.numel() != N + 1:
        raise ValueError("seq_lens / cu_q_lens do not match the block tables' batch")
    given = out is not None
    if not given:
        out = _empty_like(q, out_dtype, stream)
    elif out.shape != shape:
        raise ValueError("out must have q's shape")
    if out.dtype is torch.bfloat16:
        dtype = _native.PK_BF16
    elif out.dtype is torch.float32:
        dtype = _native.PK_FP32
    else:
        raise TypeError("out must be bf16 or fp32")
    if given:
        _need(out, "out", out.dtype, 3, dev)
    max_seq_len = _bound(MB * B if max_seq_len is None else max_seq_len)
    max_q_len = _bound(max_q_len)
    nbytes = pk_tree_workspace_bytes(H, Hkv, D, max_q_len, max_seq_len)
    if workspace is None:
        workspace = _workspace(dev, nbytes, stream)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    elif workspace.nbytes < nbytes:
        raise ValueError("workspace too small")
    head = (out.data_ptr(), dtype, q.data_ptr(), T, cu_q_lens.data_ptr(), max_q_len)
    tail = (k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(), MB, seq_lens.data_ptr(), max_seq_len, N, H,
            Hkv, D, P, B, float(scale), _at(workspace), 0 if workspace is None else workspace.nbytes)
    return dev, out, head, tail


def pk_paged_attention_tree(q: torch.Tensor, cu_q_lens: torch.Tensor, max_q_len: int, tree_mask: torch.Tensor,
                            k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                            seq_lens: torch.Tensor, scale: float, *, out_dtype=torch.bfloat16,
                            max_seq_len: Optional[int] = None, out: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of each sequence's newest tokens (rows cu_q_lens[s] .. cu_q_lens[s+1]-1
    of q [total_q, H, D] bf16, a tree of drafts already in the cache) to its whole
    context and to the nodes i whose bit i % 64 of word i // 64 is set in the row's
    ``tree_mask`` [total_q, words] int64.  See the C header."""
    dev, out, head, tail = _args(q, cu_q_lens, max_q_len, k_cache, v_cache, block_tables, seq_lens, scale, out_dtype,
                                 max_seq_len, out, workspace, stream)
    _need(tree_mask, "tree_mask", torch.int64, 2, dev)
    rows, words = tree_mask.shape
    if rows != q.shape[0]:
        raise ValueError("tree_mask must have one row per query row")
    st = _on(dev, load().pk_paged_attention_tree, *head, tree_mask.data_ptr(), words, *tail, _raw_stream(dev, stream))
    check("pk_paged_attention_tree", st)
    return out


paged_attention_tree = pk_paged_attention_tree


def pk_paged_attention_cross(q: torch.Tensor, cu_q_lens: torch.Tensor, max_q_len: int, k_cache: torch.Tensor,
                             v_cache: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor, scale: float, *,
                             out_dtype=torch.bfloat16, max_seq_len: Optional[int] = None,
                             out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                             stream=None) -> torch.Tensor:
    """Attention of any number of query rows per sequence (rows cu_q_lens[s] ..
    cu_q_lens[s+1]-1 of q) to all of the sequence's seq_lens[s] keys (an encoder's
    states): no causal limit.  See the C header."""
    dev, out, head, tail = _args(q, cu_q_lens, max_q_len, k_cache, v_cache, block_tables, seq_lens, scale, out_dtype,
                                 max_seq_len, out, workspace, stream)
    st = _on(dev, load().pk_paged_attention_cross, *head, *tail, _raw_stream(dev, stream))
    check("pk_paged_attention_cross", st)
    return out


paged_attention_cross = pk_paged_attention_cross


def pk_selftest_cross_wait_timeout(q: torch.Tensor, cu_q_lens: torch.Tensor, max_q_len: int, k_cache: torch.Tensor,
                                   v_cache: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor,
                                   scale: float, stall_tile: int, wait_limit_us: int, *, out_dtype=torch.bfloat16,
                                   max_seq_len: Optional[int] = None, out: Optional[torch.Tensor] = None,
                                   workspace: Optional[torch.Tensor] = None, stream=None) -> int:
    """Self-test of the bounded waits (see the C header): a cross-attention call whose
    CTA 0 stops copying keys at ``stall_tile``, so that its waits give up after
    ``wait_limit_us``.  Returns the call's status."""
    dev, out, head, tail = _args(q, cu_q_lens, max_q_len, k_cache, v_cache, block_tables, seq_lens, scale, out_dtype,
                                 max_seq_len, out, workspace, stream)
    return int(_on(dev, load().pk_selftest_cross_wait_timeout, *head, *tail, int(stall_tile), int(wait_limit_us),
                   _raw_stream(dev, stream)))


def pk_selftest_cross_stale_lengths(q: torch.Tensor, cu_q_lens: torch.Tensor, max_q_len: int, k_cache: torch.Tensor,
                                    v_cache: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor,
                                    scale: float, stale_seq_lens: torch.Tensor, stale_cu_q_lens: torch.Tensor, *,
                                    out_dtype=torch.bfloat16, max_seq_len: Optional[int] = None,
                                    out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                                    stream=None) -> int:
    """Self-test of the second look at the lengths (see the C header): a cross-attention
    call whose first plan is made from the stale arrays.  Returns the call's status."""
    dev, out, head, tail = _args(q, cu_q_lens, max_q_len, k_cache, v_cache, block_tables, seq_lens, scale, out_dtype,
                                 max_seq_len, out, workspace, stream)
    for stale, name, like in ((stale_seq_lens, "stale_seq_lens", seq_lens), (stale_cu_q_lens, "stale_cu_q_lens", cu_q_lens)):
        _need(stale, name, torch.int32, 1, dev)
        if stale.numel() != like.numel():
            raise ValueError(f"{name} must have as many entries as the true one")
    return int(_on(dev, load().pk_selftest_cross_stale_lengths, *head, *tail[:-2], stale_seq_lens.data_ptr(),
                   stale_cu_q_lens.data_ptr(), *tail[-2:], _raw_stream(dev, stream)))


def pk_accept_tree(draft_tokens: torch.Tensor, parents: torch.Tensor, target_tokens: torch.Tensor,
                   cu_q_lens: torch.Tensor, max_q_len: int, seq_lens: torch.Tensor, *,
                   stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """The accepted path of each tree: from its node 0 on, the lowest child whose
    drafted token is the target's choice after its parent.  ``draft_tokens`` and
    ``target_tokens`` [total_q] int64, ``parents`` [total_q] int32 (within the tree),
    ``seq_lens`` with the whole tree.  Returns (accepted [N, max_q_len] int32, -1
    behind the path; num_accepted [N] int32; next_tokens [N] int64; the lengths
    after the step [N] int32).  See the C header."""
    if not isinstance(seq_lens, torch.Tensor):
        raise TypeError("seq_lens must be a torch.Tensor")
    dev = seq_lens.device
    _need(seq_lens, "seq_lens", torch.int32, 1)
    _need(draft_tokens, "draft_tokens", torch.int64, 1, dev)
    _need(parents, "parents", torch.int32, 1, dev)
    _need(target_tokens, "target_tokens", torch.int64, 1, dev)
    _need(cu_q_lens, "cu_q_lens", torch.int32, 1, dev)
    N, T = seq_lens.numel(), draft_tokens.numel()
    if cu_q_lens.numel() != N + 1:
        raise ValueError("cu_q_lens must have one entry more than sequences")
    if parents.numel() != T or target_tokens.numel() != T:
        raise ValueError("draft_tokens / parents / target_tokens must have one entry per node")
    max_q_len = _bound(max_q_len)
    if max_q_len < 0:
        raise ValueError("max_q_len must not be negative")
    if max_q_len > _MAX_TREE:                                # (before the results are allocated)
        check("pk_accept_tree", _native.PK_ERR_UNSUPPORTED)
    with torch.cuda.stream(stream) if stream is not None else _NOTHING:
        # (From a tensor at hand: torch.empty with a device takes 2 us longer.)
        accepted = seq_lens.new_empty((N, max_q_len))
        num = torch.empty_like(seq_lens)
        following = torch.empty_like(seq_lens, dtype=torch.int64)
        lens = torch.empty_like(seq_lens)
    if stream is not None:
        for t in (accepted, num, following, lens):
            t.record_stream(torch.cuda.current_stream(dev))
    st = _on(dev, load().pk_accept_tree, accepted.data_ptr(), num.data_ptr(), following.data_ptr(), lens.data_ptr(),
             draft_tokens.data_ptr(), parents.data_ptr(), target_tokens.data_ptr(), T, cu_q_lens.data_ptr(), max_q_len,
             seq_lens.data_ptr(), N, _raw_stream(dev, stream))
    check("pk_accept_tree", st)
    return accepted, num, following, lens


accept_tree = pk_accept_tree


def _keep_args(block_tables, seq_lens, cu_q_lens, accepted, num_accepted, dev):
    _need(block_tables, "block_tables", torch.int32, 2, dev)
    _need(seq_lens, "seq_lens", torch.int32, 1, dev)
    _need(cu_q_lens, "cu_q_lens", torch.int32, 1, dev)
    _need(accepted, "accepted", torch.int32, 2, dev)
    _need(num_accepted, "num_accepted", torch.int32, 1, dev)
    N, MB = block_tables.shape
    if seq_lens.numel() != N or cu_q_lens.numel() != N + 1 or num_accepted.numel() != N or accepted.shape[0] != N:
        raise ValueError("seq_lens / cu_q_lens / accepted / num_accepted do not match the block tables' batch")
    return N, (block_tables.data_ptr(), MB, seq_lens.data_ptr(), cu_q_lens.data_ptr(), accepted.data_ptr(),
               accepted.shape[1], num_accepted.data_ptr())


def pk_keep_tokens(k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor,
                   cu_q_lens: torch.Tensor, accepted: torch.Tensor, num_accepted: torch.Tensor, stream=None) -> None:
    """Move the accepted nodes' K and V rows to the front of their tree's place in the
    cache, in place.  ``seq_lens`` are the lengths with the whole tree; ``accepted``
    and ``num_accepted`` as ``accept_tree`` gives them.  See the C header."""
    dev = k_cache.device
    _need(k_cache, "k_cache", torch.bfloat16, 4, dev)
    _need(v_cache, "v_cache", torch.bfloat16, 4, dev)
    P, B, Hkv, D = k_cache.shape
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache / v_cache shapes disagree")
    N, lists = _keep_args(block_tables, seq_lens, cu_q_lens, accepted, num_accepted, dev)
    st = _on(dev, load().pk_keep_tokens, k_cache.data_ptr(), v_cache.data_ptr(), *lists, N, Hkv, D, P, B,
             _raw_stream(dev, stream))
    check("pk_keep_tokens", st)


keep_tokens = pk_keep_tokens


def pk_keep_tokens_layers(k_cache_layers, v_cache_layers, block_tables: torch.Tensor, seq_lens: torch.Tensor,
                          cu_q_lens: torch.Tensor, accepted: torch.Tensor, num_accepted: torch.Tensor,
                          stream=None) -> None:
    """``keep_tokens`` on every layer in one launch.  Caches are lists of per-layer
    tensors or prebuilt ``LayerPointers``.  See the C header."""
    kc, vc = _layers(k_cache_layers), _layers(v_cache_layers)
    if len(kc) != len(vc) or kc.shape != vc.shape or len(kc.shape) != 4:
        raise ValueError("k / v cache layers disagree")
    dev = kc.device
    if vc.device != dev:
        raise ValueError(f"v cache layers are on {vc.device}, expected {dev}")
    P, B, Hkv, D = kc.shape
    N, lists = _keep_args(block_tables, seq_lens, cu_q_lens, accepted, num_accepted, dev)
    st = _on(dev, load().pk_keep_tokens_layers, kc.ptrs.data_ptr(), vc.ptrs.data_ptr(), *lists, N, len(kc), Hkv, D, P, B,
             _raw_stream(dev, stream))
    check("pk_keep_tokens_layers", st)
