"""Torch-facing binding of the 8-bit paged cache (``include/pagedkv_fp8.h``).

The caches are ``torch.float8_e4m3fn`` tensors [num_blocks, num_kv_heads,
block_size, head_dim] with float32 scales [num_blocks, num_kv_heads]: a stored
value stands for itself times its scale.  As in ``api``, every function
marshals arguments into one C call; names follow the C entry points, and the
unprefixed names are the same calls.
"""
from __future__ import annotations

import contextlib
import functools
from typing import Optional, Tuple

import torch

from . import _native
from ._native import check, load
from .api import _at, _empty_like, _need, _on, _raw_stream, _rope_args, new_workspace, workspace_for

FP8 = torch.float8_e4m3fn
_NOTHING = contextlib.nullcontext()


def new_cache_fp8(num_blocks: int, num_kv_heads: int, block_size: int, head_dim: int, device
                  ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """An empty 8-bit cache: (k_cache, v_cache, k_scales, v_scales)."""
    shape = (num_blocks, num_kv_heads, block_size, head_dim)
    caches = [torch.zeros(shape, dtype=torch.uint8, device=device).view(FP8) for _ in range(2)]
    scales = [torch.ones(shape[:2], dtype=torch.float32, device=device) for _ in range(2)]
    return caches[0], caches[1], scales[0], scales[1]


def _bound(x) -> int:
    """A length bound as the C calls take it: what does not fit 32 bits stays as far
    out as it can be (ctypes would take it modulo 2^32)."""
    return max(-1, min(int(x), 0x7FFFFFFF))


def _need_cache(k_cache, v_cache, k_scales, v_scales, dev):
    tensor, index = torch.Tensor, dev.index
    if (isinstance(k_cache, tensor) and isinstance(v_cache, tensor) and isinstance(k_scales, tensor)
            and isinstance(v_scales, tensor) and k_cache.dtype is FP8 and v_cache.dtype is FP8
            and k_scales.dtype is torch.float32 and v_scales.dtype is torch.float32 and k_cache.is_contiguous()
            and v_cache.is_contiguous() and k_scales.is_contiguous() and v_scales.is_contiguous()
            and k_cache.get_device() == v_cache.get_device() == k_scales.get_device() == v_scales.get_device() == index):
        shape, scales = k_cache.shape, k_scales.shape
        if len(shape) == 4 and v_cache.shape == shape and scales == shape[:2] and v_scales.shape == scales:
            return shape
    # Something is wrong: what, and where.
    _need(k_cache, "k_cache", FP8, 4, dev)
    _need(v_cache, "v_cache", FP8, 4, dev)
    _need(k_scales, "k_scales", torch.float32, 2, dev)
    _need(v_scales, "v_scales", torch.float32, 2, dev)
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must have the same shape")
    raise ValueError(f"scales must be [num_blocks, num_kv_heads] = {tuple(k_cache.shape[:2])}")


def pk_rope_and_cache_fp8(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor,
                          v_cache: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor,
                          block_tables: torch.Tensor, seq_lens: torch.Tensor,
                          inv_freq: Optional[torch.Tensor] = None, *, cu_q_lens: Optional[torch.Tensor] = None,
                          max_q_len: Optional[int] = None, positions: Optional[torch.Tensor] = None,
                          interleaved: bool = False, factor: float = 1.0, q_out: Optional[torch.Tensor] = None,
                          stream=None) -> Optional[torch.Tensor]:
    """Rotate q and k, append k and v to the 8-bit cache and return the rotated
    queries.  Rows cu_q_lens[s] .. cu_q_lens[s+1]-1 are sequence s's newest
    tokens (``cu_q_lens`` None: one a sequence), ``seq_lens`` the lengths after
    the append; the positions are those in the block table unless given.  The
    other arguments are those of ``rope_and_cache``.  See the C header."""
    dev = k_cache.device
    P, Hc, B, Dc = _need_cache(k_cache, v_cache, k_scales, v_scales, dev)
    _need(block_tables, "block_tables", torch.int32, 2, dev)
    _need(seq_lens, "seq_lens", torch.int32, 1, dev)
    (T, Hkv, D), q_out, H, rot, strides = _rope_args(q, k, v, inv_freq, q_out, dev, stream)
    N, MB = block_tables.shape
    if Hc != Hkv or Dc != D:
        raise ValueError("k / v / cache shapes disagree")
    if seq_lens.numel() != N:
        raise ValueError("seq_lens do not match the block tables' batch")
    if cu_q_lens is None:
        if T != N:
            raise ValueError("without cu_q_lens every sequence has one new token")
        max_q_len = 1
    else:
        _need(cu_q_lens, "cu_q_lens", torch.int32, 1, dev)
        if cu_q_lens.numel() != N + 1:
            raise ValueError("cu_q_lens must have one entry more than sequences")
        if max_q_len is None:
            max_q_len = T
    if positions is not None:
        _need(positions, "positions", torch.int64, 1, dev)
        if positions.numel() != T:
            raise ValueError("positions must have one entry per token")
    st = _on(dev, load().pk_rope_and_cache_fp8, _at(q_out), _at(q), k.data_ptr(), v.data_ptr(), *strides,
             k_cache.data_ptr(), v_cache.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(),
             block_tables.data_ptr(), MB, seq_lens.data_ptr(), _at(cu_q_lens), _bound(max_q_len), N, _at(positions),
             _at(inv_freq), rot, int(interleaved), float(factor), T, H, Hkv, D, P, B, _raw_stream(dev, stream))
    check("pk_rope_and_cache_fp8", st)
    return q_out


rope_and_cache_fp8 = pk_rope_and_cache_fp8


@functools.lru_cache(maxsize=256)
def pk_decode_fp8_workspace_bytes(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int,
                                  max_seq_len: int) -> int:
    return int(load().pk_decode_fp8_workspace_bytes(num_seqs, num_heads, num_kv_heads, head_dim, max_seq_len))


def _workspace(dev, nbytes: int, stream) -> Optional[torch.Tensor]:
    """The cached workspace of the stream; while it is being captured, one from
    the graph's own pool, so that two graphs never share one."""
    if nbytes == 0:
        return None
    with torch.cuda.stream(stream) if stream is not None else _NOTHING:
        return new_workspace(nbytes, dev) if torch._C._cuda_isCurrentStreamCapturing() else workspace_for(dev, nbytes, stream)


def _attend(name, out, q, cu_q_lens, max_q_len, k_cache, v_cache, k_scales, v_scales, block_tables, seq_lens, scale,
            out_dtype, max_seq_len, workspace, stream):
    dev = q.device
    _need(q, "q", torch.bfloat16, 3)
    P, Hkv, B, Dk = _need_cache(k_cache, v_cache, k_scales, v_scales, dev)
    _need(block_tables, "block_tables", torch.int32, 2, dev)
    _need(seq_lens, "seq_lens", torch.int32, 1, dev)
    T, H, D = shape = q.shape
    N, MB = block_tables.shape
    if Dk != D:
        raise ValueError("k_cache / v_cache / q shapes disagree")
    if seq_lens.numel() != N:
        raise ValueError("seq_lens do not match the block tables' batch")
    if cu_q_lens is None:
        if T != N:
            raise ValueError("q must have one row per sequence")
    else:
        _need(cu_q_lens, "cu_q_lens", torch.int32, 1, dev)
        if cu_q_lens.numel() != N + 1:
            raise ValueError("cu_q_lens must have one entry more than sequences")
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
    nbytes = pk_decode_fp8_workspace_bytes(N, H, Hkv, D, max_seq_len)
    if workspace is None:
        workspace = _workspace(dev, nbytes, stream)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    elif workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError("workspace too small")
    tail = (k_cache.data_ptr(), v_cache.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), block_tables.data_ptr(),
            MB, seq_lens.data_ptr(), max_seq_len, N, H, Hkv, D, P, B, float(scale), _at(workspace),
            0 if workspace is None else workspace.nbytes, _raw_stream(dev, stream))
    if cu_q_lens is None:
        st = _on(dev, load().pk_paged_attention_decode_fp8, out.data_ptr(), dtype, q.data_ptr(), *tail)
    else:
        st = _on(dev, load().pk_paged_attention_multi_query_fp8, out.data_ptr(), dtype, q.data_ptr(), T,
                 cu_q_lens.data_ptr(), _bound(max_q_len), *tail)
    check(name, st)
    return out


def pk_paged_attention_decode_fp8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                  k_scales: torch.Tensor, v_scales: torch.Tensor, block_tables: torch.Tensor,
                                  seq_lens: torch.Tensor, scale: float, *, out_dtype=torch.bfloat16,
                                  max_seq_len: Optional[int] = None, out: Optional[torch.Tensor] = None,
                                  workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Decode attention of q [N, H, D] bf16 over the 8-bit paged cache; returns
    [N, H, D] (bf16 or fp32).  See the C header."""
    return _attend("pk_paged_attention_decode_fp8", out, q, None, 1, k_cache, v_cache, k_scales, v_scales,
                   block_tables, seq_lens, scale, out_dtype, max_seq_len, workspace, stream)


paged_attention_decode_fp8 = pk_paged_attention_decode_fp8


def _selftest_args(out, q, k_cache, v_cache, k_scales, v_scales, block_tables, seq_lens, scale, max_seq_len):
    N, H, D = q.shape
    P, Hkv, B, _ = k_cache.shape
    return (out.data_ptr(), _native.PK_FP32 if out.dtype == torch.float32 else _native.PK_BF16, q.data_ptr(),
            k_cache.data_ptr(), v_cache.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), block_tables.data_ptr(),
            block_tables.shape[1], seq_lens.data_ptr(), _bound(max_seq_len), N, H, Hkv, D, P, B, float(scale))


def pk_selftest_decode_fp8_wait_timeout(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                        k_scales: torch.Tensor, v_scales: torch.Tensor, block_tables: torch.Tensor,
                                        seq_lens: torch.Tensor, scale: float, max_seq_len: int, workspace: torch.Tensor,
                                        stall_tile: int, wait_limit_us: int, stream=None) -> int:
    """Self-test of the bounded waits (see the C header): a decode call whose CTA 0
    stops issuing copies at ``stall_tile``, so that its waits give up after
    ``wait_limit_us``.  Returns the call's status."""
    return int(_on(q.device, load().pk_selftest_decode_fp8_wait_timeout,
                   *_selftest_args(out, q, k_cache, v_cache, k_scales, v_scales, block_tables, seq_lens, scale, max_seq_len),
                   workspace.data_ptr(), workspace.nbytes, int(stall_tile), int(wait_limit_us), _raw_stream(q.device, stream)))


def pk_selftest_decode_fp8_stale_lengths(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                         k_scales: torch.Tensor, v_scales: torch.Tensor, block_tables: torch.Tensor,
                                         seq_lens: torch.Tensor, scale: float, max_seq_len: int,
                                         stale_seq_lens: torch.Tensor, workspace: torch.Tensor, stream=None) -> int:
    """Self-test of the second look at the lengths (see the C header): a decode call
    that plans first from ``stale_seq_lens``.  Returns the call's status."""
    return int(_on(q.device, load().pk_selftest_decode_fp8_stale_lengths,
                   *_selftest_args(out, q, k_cache, v_cache, k_scales, v_scales, block_tables, seq_lens, scale, max_seq_len),
                   stale_seq_lens.data_ptr(), workspace.data_ptr(), workspace.nbytes, _raw_stream(q.device, stream)))


def pk_paged_attention_multi_query_fp8(q: torch.Tensor, cu_q_lens: torch.Tensor, max_q_len: int,
                                       k_cache: torch.Tensor, v_cache: torch.Tensor, k_scales: torch.Tensor,
                                       v_scales: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor,
                                       scale: float, *, out_dtype=torch.bfloat16, max_seq_len: Optional[int] = None,
                                       out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                                       stream=None) -> torch.Tensor:
    """Causal attention of a few new tokens per sequence (rows cu_q_lens[s] ..
    cu_q_lens[s+1]-1 of q) over the 8-bit paged cache; at most 16 query columns
    (tokens, rounded up to a power of two, times heads per KV head).  Wider
    blocks: ``gather_kv_fp8``, then ``paged_attention_multi_query``."""
    if cu_q_lens is None:
        raise TypeError("cu_q_lens must be a torch.Tensor")
    return _attend("pk_paged_attention_multi_query_fp8", out, q, cu_q_lens, max_q_len, k_cache, v_cache, k_scales,
                   v_scales, block_tables, seq_lens, scale, out_dtype, max_seq_len, workspace, stream)


paged_attention_multi_query_fp8 = pk_paged_attention_multi_query_fp8


def pk_gather_kv_fp8(k_cache: torch.Tensor, v_cache: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor,
                     block_tables: torch.Tensor, seq_lens: torch.Tensor, cu_seq_lens: torch.Tensor,
                     out_k: torch.Tensor, out_v: torch.Tensor, *, max_seq_len: Optional[int] = None,
                     stream=None) -> None:
    """Write the sequences' K and V rows as bf16 to rows cu_seq_lens[s] + j of
    out_k and out_v ([rows, Hkv, D]).  See the C header."""
    dev = k_cache.device
    P, Hkv, B, D = _need_cache(k_cache, v_cache, k_scales, v_scales, dev)
    _need(block_tables, "block_tables", torch.int32, 2, dev)
    _need(seq_lens, "seq_lens", torch.int32, 1, dev)
    _need(cu_seq_lens, "cu_seq_lens", torch.int64, 1, dev)
    _need(out_k, "out_k", torch.bfloat16, 3, dev)
    _need(out_v, "out_v", torch.bfloat16, 3, dev)
    N, MB = block_tables.shape
    if seq_lens.numel() != N or cu_seq_lens.numel() != N:
        raise ValueError("seq_lens / cu_seq_lens do not match the block tables' batch")
    rows, heads, width = out_k.shape
    if out_k.shape != out_v.shape or (heads, width) != (Hkv, D):
        raise ValueError("out_k and out_v must be [rows, num_kv_heads, head_dim]")
    if max_seq_len is None:
        max_seq_len = MB * B
    st = _on(dev, load().pk_gather_kv_fp8, out_k.data_ptr(), out_v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
             k_scales.data_ptr(), v_scales.data_ptr(), block_tables.data_ptr(), MB, seq_lens.data_ptr(),
             cu_seq_lens.data_ptr(), rows, _bound(max_seq_len), N, Hkv, D, P, B, _raw_stream(dev, stream))
    check("pk_gather_kv_fp8", st)


gather_kv_fp8 = pk_gather_kv_fp8


def pk_copy_blocks_fp8(k_cache: torch.Tensor, v_cache: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor,
                       src_dst_pairs: torch.Tensor, stream=None) -> None:
    """Copy whole blocks and their scales for every (src, dst) row of an int64
    [n, 2] tensor.  See the C header."""
    dev = k_cache.device
    P, Hkv, B, D = _need_cache(k_cache, v_cache, k_scales, v_scales, dev)
    _need(src_dst_pairs, "src_dst_pairs", torch.int64, 2, dev)
    n, two = src_dst_pairs.shape
    if two != 2:
        raise ValueError("src_dst_pairs must be [n, 2]")
    st = _on(dev, load().pk_copy_blocks_fp8, k_cache.data_ptr(), v_cache.data_ptr(), k_scales.data_ptr(),
             v_scales.data_ptr(), src_dst_pairs.data_ptr(), n, Hkv, D, P, B, _raw_stream(dev, stream))
    check("pk_copy_blocks_fp8", st)


copy_blocks_fp8 = pk_copy_blocks_fp8


def pk_swap_blocks_fp8(dst, src, pairs: torch.Tensor, stream=None) -> None:
    """Copy whole blocks and their scales from pool ``src`` to pool ``dst``
    (each a (k_cache, v_cache, k_scales, v_scales); CUDA tensors or pinned CPU
    tensors) for every (src, dst) row of an int64 [n, 2] device tensor.  See
    the C header."""
    if not isinstance(pairs, torch.Tensor) or not pairs.is_cuda:
        raise ValueError("pairs must be a CUDA tensor")
    dev = pairs.device
    _need(pairs, "pairs", torch.int64, 2, dev)
    if pairs.shape[1] != 2:
        raise ValueError("pairs must be [n, 2]")
    for name, pool in (("dst", dst), ("src", src)):
        if len(pool) != 4:
            raise ValueError(f"{name} must be (k_cache, v_cache, k_scales, v_scales)")
        for what, t, dtype, ndim in zip(("k_cache", "v_cache", "k_scales", "v_scales"), pool,
                                        (FP8, FP8, torch.float32, torch.float32), (4, 4, 2, 2)):
            if t.dtype != dtype or t.dim() != ndim or not t.is_contiguous():
                raise ValueError(f"{name} {what} must be a contiguous {dtype} tensor of {ndim} dims")
            if not (t.is_cuda and t.device == dev) and not (t.device.type == "cpu" and t.is_pinned()):
                raise ValueError(f"{name} {what} must be on {dev} or in pinned host memory")
        if pool[0].shape != pool[1].shape or any(tuple(x.shape) != tuple(pool[0].shape[:2]) for x in pool[2:]):
            raise ValueError(f"the shapes of pool {name} disagree")
    if src[0].shape[1:] != dst[0].shape[1:]:
        raise ValueError("pool shapes disagree")
    P_src, Hkv, B, D = src[0].shape
    st = _on(dev, load().pk_swap_blocks_fp8, *(t.data_ptr() for t in dst), *(t.data_ptr() for t in src),
             pairs.data_ptr(), pairs.shape[0], Hkv, D, B, P_src, dst[0].shape[0], _raw_stream(dev, stream))
    check("pk_swap_blocks_fp8", st)


swap_blocks_fp8 = pk_swap_blocks_fp8
