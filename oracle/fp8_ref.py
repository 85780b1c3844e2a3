"""Float64 reference of the 8-bit paged cache and of rotary positions.

Written from the definitions in ``include/pagedkv.h`` (pk_rope_and_cache) and
``include/pagedkv_fp8.h``; shares no code with the library.  Caches are numpy
uint8 arrays [num_blocks, num_kv_heads, block_size, head_dim] of e4m3 bytes,
scales float32 [num_blocks, num_kv_heads].
"""
from __future__ import annotations

import math
from typing import Optional, Sequence

import numpy as np


def _e4m3_table() -> np.ndarray:
    out = np.empty(256)
    for b in range(256):
        sign = -1.0 if b & 0x80 else 1.0
        e, m = (b >> 3) & 15, b & 7
        if e == 15 and m == 7:
            out[b] = np.nan
        elif e == 0:
            out[b] = sign * m * 2.0 ** -9
        else:
            out[b] = sign * (8 + m) * 2.0 ** (e - 10)
    return out


E4M3 = _e4m3_table()


def e4m3_decode(b: np.ndarray) -> np.ndarray:
    return E4M3[np.asarray(b, dtype=np.uint8)]


def e4m3_step(x: np.ndarray) -> np.ndarray:
    """Spacing of the e4m3 values around |x| (up to 448)."""
    ax = np.abs(x)
    e = np.floor(np.log2(np.where(ax > 0, ax, 1.0)))
    e = np.where(np.ldexp(1.0, e.astype(int)) > ax, e - 1, e)          # log2 may round up at a power of two
    return np.ldexp(1.0, (np.clip(np.where(ax > 0, e, -6), -6, 8) - 3).astype(int))


def e4m3_encode(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 byte, ties to even, at most +-448; what is not finite becomes NaN."""
    x = np.asarray(x, dtype=np.float64)
    ok = np.isfinite(x)
    y = np.clip(np.where(ok, x, 0.0), -448.0, 448.0)
    step = e4m3_step(y)
    y = np.clip(np.rint(y / step) * step, -448.0, 448.0)
    mag = np.abs(y)
    e = np.floor(np.log2(np.where(mag >= 2.0 ** -6, mag, 1.0)))
    normal = mag >= 2.0 ** -6
    byte = np.where(normal, (e + 7) * 8 + (mag / 2.0 ** e - 1.0) * 8, mag * 2.0 ** 9).astype(np.uint8)
    byte = byte | np.where(np.signbit(x), 0x80, 0).astype(np.uint8)
    return np.where(ok, byte, 0x7F).astype(np.uint8)


def rope(x: np.ndarray, positions: Sequence[int], inv_freq: Optional[np.ndarray], interleaved: bool = False,
         factor: float = 1.0) -> np.ndarray:
    """x [T, heads, D] float64 with its first 2 * len(inv_freq) elements rotated."""
    y = np.array(x, dtype=np.float64)
    if inv_freq is None or len(inv_freq) == 0:
        return y
    r = len(inv_freq)
    angle = np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(inv_freq, dtype=np.float32).astype(np.float64)
    c, s = np.cos(angle)[:, None] * factor, np.sin(angle)[:, None] * factor
    first = slice(0, 2 * r, 2) if interleaved else slice(0, r)
    second = slice(1, 2 * r, 2) if interleaved else slice(r, 2 * r)
    x1, x2 = y[..., first].copy(), y[..., second].copy()
    y[..., first], y[..., second] = x1 * c - x2 * s, x2 * c + x1 * s
    return y


def largest_square(x: np.ndarray, rot: int, interleaved: bool, factor: float) -> np.ndarray:
    """m2 over the tokens and elements of x [n, heads, D], [heads], as the header
    defines it: sums and products rounded to 32 bits, what is not finite left out."""
    x = np.asarray(x, dtype=np.float64)
    a = x[..., :rot]
    x1, x2 = (a[..., 0::2], a[..., 1::2]) if interleaved else (a[..., :rot // 2], a[..., rot // 2:])
    top = float(np.finfo(np.float32).max)

    def square(u, v):
        ok = np.isfinite(u) & np.isfinite(v)
        m = np.where(ok, u, 0.0) ** 2 + np.where(ok, v, 0.0) ** 2
        with np.errstate(over="ignore"):
            return m.astype(np.float32)                        # infinity where it overflows
    pairs = square(x1, x2).reshape(*x.shape[:2], -1)
    rest = square(x[..., rot:], np.zeros_like(x[..., rot:]))
    out = np.zeros(x.shape[1], dtype=np.float32)
    if pairs.size:
        f2 = np.float32(np.float32(factor) * np.float32(factor))
        with np.errstate(over="ignore"):
            out = np.maximum(out, pairs.max(axis=(0, 2)) * f2)
    if rest.size:
        out = np.maximum(out, rest.max(axis=(0, 2)))
    return np.minimum(out, np.float32(top))


def needed_scale(m2: float) -> float:
    """The smallest 2^e, -64 <= e <= 64, with m2 <= (448 * 2^e)^2, by trying them."""
    for e in range(-64, 64):
        if float(m2) <= (448.0 * 2.0 ** e) ** 2:
            return 2.0 ** e
    return 2.0 ** 64


def append_fp8(k, v, k_cache, v_cache, k_scales, v_scales, tables, seq_lens, cu_q_lens, inv_freq=None,
               interleaved: bool = False, factor: float = 1.0, positions=None):
    """The append on copies of the caches: (k_cache, v_cache, k_scales, v_scales,
    exact), where exact[name] lists (block, row, values / scale) of the new rows
    before they are rounded, [Hkv, D]."""
    k_cache, v_cache, k_scales, v_scales = (np.array(x) for x in (k_cache, v_cache, k_scales, v_scales))
    B = k_cache.shape[2]
    rot = 0 if inv_freq is None else 2 * len(inv_freq)
    exact = {"k": [], "v": []}
    for s, L in enumerate(seq_lens):
        r0, r1 = int(cu_q_lens[s]), int(cu_q_lens[s + 1])
        at, start = int(L) - (r1 - r0), int(L) - (r1 - r0)
        while at < L:
            end = min(int(L), (at // B + 1) * B)
            rows = slice(r0 + at - start, r0 + end - start)
            block, off = int(tables[s][at // B]), at % B
            pos = np.arange(at, end) if positions is None else np.asarray(positions)[rows]
            for name, x, cache, scales in (("k", k, k_cache, k_scales), ("v", v, v_cache, v_scales)):
                m2 = largest_square(x[rows], rot if name == "k" else 0, interleaved, factor)
                y = rope(x[rows], pos, inv_freq if name == "k" else None, interleaved, factor)
                for h in range(cache.shape[1]):
                    scale = needed_scale(m2[h])
                    if off:
                        had = float(scales[block, h])
                        if not 2.0 ** -64 <= had <= 2.0 ** 64:
                            cache[block, h, :off] = 0x7F       # what they stood for is not known
                        elif had >= scale:
                            scale = had
                        else:
                            cache[block, h, :off] = e4m3_encode(e4m3_decode(cache[block, h, :off]) * (had / scale))
                    scales[block, h] = scale
                    cache[block, h, off:off + end - at] = e4m3_encode(y[:, h] / scale)
                for i in range(end - at):
                    exact[name].append((block, off + i, y[i] / scales[block].astype(np.float64)[:, None]))
            at = end
    return k_cache, v_cache, k_scales, v_scales, exact


def rows_fp8(cache: np.ndarray, scales: np.ndarray, table: Sequence[int], length: int) -> np.ndarray:
    """[length, Hkv, D] values of a sequence's tokens."""
    B = cache.shape[2]
    blocks = [int(b) for b in table[:-(-int(length) // B)]]
    if not blocks:
        return np.zeros((0, cache.shape[1], cache.shape[3]))
    x = e4m3_decode(cache[blocks]) * scales[blocks].astype(np.float64)[:, :, None, None]
    return x.transpose(0, 2, 1, 3).reshape(-1, cache.shape[1], cache.shape[3])[:length]


def attention_fp8(q, k_cache, v_cache, k_scales, v_scales, tables, seq_lens, cu_q_lens, scale: float):
    """Causal attention of each sequence's newest tokens, float64: (out [total_q,
    H, D], spread [total_q, H, D], scores), spread = sum p |v|, scores the
    largest sum |q||k| * |scale| a row met (both for error bounds)."""
    q = np.asarray(q, dtype=np.float64)
    out, spread = np.zeros_like(q), np.zeros_like(q)
    scores = 0.0
    H = q.shape[1]
    for s, L in enumerate(seq_lens):
        r0, r1 = int(cu_q_lens[s]), int(cu_q_lens[s + 1])
        K = rows_fp8(k_cache, k_scales, tables[s], L)
        V = rows_fp8(v_cache, v_scales, tables[s], L)
        G = H // K.shape[1]
        for r in range(r0, r1):
            n = int(L) - (r1 - r0) + (r - r0) + 1
            if n <= 0:
                continue
            for h in range(H):
                k, v = K[:n, h // G], V[:n, h // G]
                z = scale * (k @ q[r, h])
                scores = max(scores, float(np.max(np.abs(k) @ np.abs(q[r, h])) * abs(scale)))
                p = np.exp(z - z.max())
                p /= p.sum()
                out[r, h], spread[r, h] = p @ v, p @ np.abs(v)
    return out, spread, scores


def attention_floor(q, k_cache, v_cache, k_scales, v_scales, tables, seq_lens, cu_q_lens, scale: float) -> np.ndarray:
    """[total_q, H, D]: the largest p_j vs_j of a row times sum_j |stored v_j|.
    A weight p_j vs_j is kept to 2^-24 of the row's largest one beside its relative
    error, so 2^-24 of this is what the row's small weights can lose together:
    attention_bound's last term, with ``length`` 1 and this as ``largest_v``.  (That
    term as such takes p_j vs_j <= largest vs, which a long context is far below.)"""
    q = np.asarray(q, dtype=np.float64)
    out = np.zeros_like(q)
    for s, L in enumerate(seq_lens):
        r0, r1 = int(cu_q_lens[s]), int(cu_q_lens[s + 1])
        K, ones = rows_fp8(k_cache, k_scales, tables[s], L), np.ones_like(v_scales)
        V = np.abs(rows_fp8(v_cache, ones, tables[s], L))
        B = k_cache.shape[2]
        G = q.shape[1] // K.shape[1]
        vs = np.repeat(np.stack([v_scales[int(b)].astype(np.float64) for b in tables[s][:-(-int(L) // B)]]), B, axis=0) if L else None
        for r in range(r0, r1):
            n = int(L) - (r1 - r0) + (r - r0) + 1
            for h in range(q.shape[1]) if n > 0 else ():
                z = scale * (K[:n, h // G] @ q[r, h])
                p = np.exp(z - z.max())
                out[r, h] = np.max(p * vs[:n, h // G]) / p.sum() * V[:n, h // G].sum(axis=0)
    return out


def attention_bound(out, spread, scores: float, length: int, largest_v: float, bf16_out: bool,
                    weight_error: float = 2.0 ** -9 + 2.0 ** -11) -> np.ndarray:
    """How far the kernel's result may be from ``out``.  A weight is used to
    ``weight_error`` + 2^-18 (exponential and 32-bit arithmetic) of itself and to
    2^-24 of the largest one; a score is off by at most 2^-20 of sum |q||k| (query
    terms to 2^-22 of the row's largest, 32-bit sums), which moves numerator and
    denominator alike.  The kernel's weights are to 2^-11 (fp16, which three e5m2
    terms hold exactly); the default also covers three e4m3 terms, 2^-9 more."""
    weight = weight_error + 2.0 ** -18 + 2.0 * math.expm1(scores * 2.0 ** -20)
    tol = weight * (spread + np.abs(out)) + length * 2.0 ** -24 * largest_v
    return tol + (2.0 ** -8 * (np.abs(out) + tol) if bf16_out else 2.0 ** -23 * np.abs(out))
