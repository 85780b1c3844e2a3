"""Inputs shared by the tests of rotary positions and of the 8-bit cache."""
from __future__ import annotations

import numpy as np
import torch

import paged_kv_cache_122_gb300 as pk
from oracle import fp8_ref as R

DEV = "cuda:0"


def tables(rng, lens, B, spare=3, pad=-1):
    """Shuffled block tables for ``lens`` and the pool they come from."""
    need = [-(-int(n) // B) for n in lens]
    pool = sum(need) + spare
    ids = rng.permutation(pool).astype(np.int32)
    bt = np.full((len(lens), max(1, max(need))), pad, dtype=np.int32)
    k = 0
    for s, n in enumerate(need):
        bt[s, :n] = ids[k:k + n]
        k += n
    return bt, pool


def cache(rng, pool, Hkv, B, D, spread=1.0):
    """Random e4m3 bytes (no NaN) and power-of-two scales around 2^-7."""
    b = rng.integers(0, 256, size=(pool, Hkv, B, D), dtype=np.uint8)
    b = np.where((b & 0x7F) == 0x7F, b & 0x80, b).astype(np.uint8)
    # Magnitudes like quantised normal values: most exponents in the upper half.
    b = np.where((b & 0x78) < 0x38, (b & 0x87) | 0x40, b).astype(np.uint8)
    scales = np.exp2(rng.integers(-9, -6, size=(pool, Hkv))).astype(np.float32) * np.float32(spread)
    return b, scales


def to_dev(x):
    t = torch.from_numpy(np.ascontiguousarray(x)).to(DEV)
    return t


def to_cache(b):
    return to_dev(b).view(torch.float8_e4m3fn)


def cache_bytes(t):
    return t.view(torch.uint8).cpu().numpy()


def bf16(rng, *shape, scale=1.0):
    """Random bf16 values: (device tensor, float64 array)."""
    t = torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16)
    return t.to(DEV), t.double().numpy()


def cu_of(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def attention_case(seed, lens, qlens, G, Hkv, D, B, qscale=2.0, pad=-1):
    rng = np.random.default_rng(seed)
    bt, pool = tables(rng, lens, B, pad=pad)
    kb, ks = cache(rng, pool, Hkv, B, D)
    vb, vs = cache(rng, pool, Hkv, B, D)
    cu = cu_of(qlens)
    q, q64 = bf16(rng, int(cu[-1]), G * Hkv, D, scale=qscale)
    return dict(bt=bt, pool=pool, kb=kb, vb=vb, ks=ks, vs=vs, cu=cu, q=q, q64=q64, lens=np.asarray(lens, np.int32),
                scale=1.0 / np.sqrt(D), qmax=max(qlens) if len(qlens) else 0,
                dev=dict(k=to_cache(kb), v=to_cache(vb), ks=to_dev(ks), vs=to_dev(vs), bt=to_dev(bt),
                         sl=to_dev(np.asarray(lens, np.int32)), cu=to_dev(cu)))


def attend(c, out_dtype=torch.float32, multi=False, **kw):
    d = c["dev"]
    if multi:
        return pk.paged_attention_multi_query_fp8(c["q"], d["cu"], c["qmax"], d["k"], d["v"], d["ks"], d["vs"], d["bt"],
                                                  d["sl"], c["scale"], out_dtype=out_dtype, **kw)
    return pk.paged_attention_decode_fp8(c["q"], d["k"], d["v"], d["ks"], d["vs"], d["bt"], d["sl"], c["scale"],
                                         out_dtype=out_dtype, **kw)


def check_attention(c, out, what="", kb=None, vb=None, ks=None, vs=None):
    """The kernel's output against the float64 attention, within its derived bound."""
    vs = c["vs"] if vs is None else vs
    ref, spread, scores = R.attention_fp8(c["q64"], c["kb"] if kb is None else kb, c["vb"] if vb is None else vb,
                                          c["ks"] if ks is None else ks, vs, c["bt"], c["lens"], c["cu"], c["scale"])
    got = out.double().cpu().numpy()
    tol = R.attention_bound(ref, spread, scores, int(max(c["lens"], default=0)), float(448 * vs.max()),
                            out.dtype == torch.bfloat16)
    err = np.abs(got - ref)
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    worst = np.unravel_index(np.argmax(err - tol), err.shape)
    assert np.all(err <= tol), f"{what}: off by {err[worst]:.3e}, {tol[worst]:.3e} allowed at {worst}"
