"""Float64 references of tree attention, cross attention, the accepted path and the
move of its rows.  TEST INFRASTRUCTURE ONLY (see the package docstring): plain
definitions, no splitting, no online softmax, nothing shared with the library.
"""
from __future__ import annotations

from typing import List, Optional, Sequence, Tuple

import numpy as np

from .paged_ref import bf16_bits_to_f64, gather_sequence


def masked_attention(q_bits: np.ndarray, k_cache_bits: np.ndarray, v_cache_bits: np.ndarray, block_tables: np.ndarray,
                     seq_lens: Sequence[int], cu_q_lens: Sequence[int], scale: float, block_size: int,
                     tree_mask: Optional[np.ndarray] = None) -> Tuple[np.ndarray, np.ndarray, np.ndarray, np.ndarray]:
    """Attention of query rows cu_q_lens[s] .. to the sequence's keys: with
    ``tree_mask`` [total_q, words] (uint64) the rows are its newest tokens and see the
    context and the nodes whose bit is set, without it they see every key.

    Returns out [total_q, H, D] float64 (zeros where a row sees nothing) and, for the
    error bound, sum p |v - out|, sum p |v| (same shape) and the largest
    scale * sum |q| |k| over the keys a row sees ([total_q, H]).
    """
    Tq, H, D = q_bits.shape
    Hkv = k_cache_bits.shape[2]
    G = H // Hkv
    out, spread, size = (np.zeros((Tq, H, D)) for _ in range(3))
    most = np.zeros((Tq, H))
    q_all = bf16_bits_to_f64(q_bits)
    for s in range(len(seq_lens)):
        L, q0, q1 = int(seq_lens[s]), int(cu_q_lens[s]), int(cu_q_lens[s + 1])
        n = q1 - q0
        if n == 0 or L == 0:
            continue
        sees = np.ones((n, L), dtype=bool)
        if tree_mask is not None:
            for r in range(n):
                for i in range(n):
                    sees[r, L - n + i] = bool((int(tree_mask[q0 + r, i // 64]) >> (i % 64)) & 1)
        for h in range(Hkv):
            K = bf16_bits_to_f64(gather_sequence(k_cache_bits, block_tables[s], L, block_size, h))
            V = bf16_bits_to_f64(gather_sequence(v_cache_bits, block_tables[s], L, block_size, h))
            for g in range(h * G, (h + 1) * G):
                q = q_all[q0:q1, g]
                with np.errstate(invalid="ignore", over="ignore"):
                    x = np.where(sees, scale * (q @ K.T), -np.inf)
                top = x.max(axis=1, keepdims=True)
                p = np.where(sees, np.exp(x - np.where(np.isfinite(top), top, 0.0)), 0.0)
                total = p.sum(axis=1, keepdims=True)
                p = np.divide(p, total, out=np.zeros_like(p), where=total > 0)
                o = p @ V
                out[q0:q1, g] = o
                size[q0:q1, g] = p @ np.abs(V)
                for r in range(n):
                    spread[q0 + r, g] = p[r] @ np.abs(V - o[r])
                mag = np.where(sees, abs(scale) * (np.abs(q) @ np.abs(K).T), 0.0)
                most[q0:q1, g] = np.nan_to_num(mag).max(axis=1)
    return out, spread, size, most


def ancestors_mask(parents: Sequence[int], words: int) -> np.ndarray:
    """[nodes, words] uint64: bit i of row r is set where node i is r or above it."""
    seen: List[int] = []
    for r, p in enumerate(parents):
        seen.append((seen[p] if p >= 0 else 0) | (1 << r))
    return np.array([[(m >> (64 * w)) & ((1 << 64) - 1) for w in range(words)] for m in seen],
                    dtype=np.uint64).reshape(len(seen), words)


def accept(tokens: Sequence[int], parents: Sequence[int], targets: Sequence[int]) -> List[int]:
    """The accepted path of one tree: from node 0, again and again the lowest child
    whose token is the target's after the node."""
    path: List[int] = [0] if len(tokens) else []
    while path:
        at = path[-1]
        nxt = [c for c in range(at + 1, len(tokens)) if parents[c] == at and tokens[c] == targets[at]]
        if not nxt:
            break
        path.append(nxt[0])
    return path


def keep(cache_bits: np.ndarray, block_tables: np.ndarray, seq_lens: Sequence[int], cu_q_lens: Sequence[int],
         paths: Sequence[Sequence[int]], block_size: int) -> np.ndarray:
    """A copy of the cache in which the rows of each path lie together."""
    out = cache_bits.copy()
    for s, path in enumerate(paths):
        base = int(seq_lens[s]) - (int(cu_q_lens[s + 1]) - int(cu_q_lens[s]))
        for i, node in enumerate(path):
            src, dst = base + node, base + i
            out[block_tables[s][dst // block_size], dst % block_size] = \
                cache_bits[block_tables[s][src // block_size], src % block_size]
    return out


def bound(out: np.ndarray, spread: np.ndarray, size: np.ndarray, most: np.ndarray, keys: int, head_dim: int,
          bf16_out: bool) -> np.ndarray:
    """What an element may be off by where weights are rounded to bf16 and sums are
    fp32.  With weights w_j (1 + d_j), |d_j| <= e, the mean of v moves by at most
    e sum p |v - out| / (1 - e).  e: half a step of bf16, 2^-8 (8 significant bits: the
    numbers from 1 to 2 are 2^-7 apart); scores that are D fp32 sums, each off by at most a step (2^-23) of the
    running magnitude; 2^-16 for the exponent's fma (arguments below 2^7, 2^-24 of
    them) and 2^x (2^-22).  The sums over the keys add keys + 8 steps of sum p |v|, the
    output half a step of bf16 (2^-8 of the power of two at or below it)."""
    e = 2.0 ** -8 + head_dim * 2.0 ** -23 * most[..., None] + 2.0 ** -16
    tol = e / (1.0 - e) * spread + (keys + 8) * 2.0 ** -23 * size
    if bf16_out:
        mag = np.abs(out) + tol
        tol = tol + np.where(mag > 0, 2.0 ** (np.floor(np.log2(np.where(mag > 0, mag, 1.0))) - 8), 0.0)
    return tol + 1e-37


__all__ = ["masked_attention", "ancestors_mask", "accept", "keep", "bound"]
