"""Attention cases in which every 128-token tile shows in the result.

The values of tile t are one constant at element t % D and zero elsewhere, so an
element is the weight of L / (128 D) tiles: one that is lost, or joined with a
wrong weight, moves it by far more than the error bound, however long the
context (random values average out, and there a lost tile hides in the bound).
The value scales are all 2^-7, so that no tile's share is small.
"""
from __future__ import annotations

import numpy as np

from fp8lib import attention_case, cache, cu_of, tables, to_cache, to_dev
from oracle import fp8_ref as R

TILE = 128


def tile_values(vb, bt, lens):
    """Values 128 at element t % D of tile t's rows."""
    vb = np.zeros_like(vb)
    B, D = vb.shape[2:]
    for s, n in enumerate(lens):
        for j in range(-(-int(n) // B)):
            vb[bt[s, j], :, :, (j * B // TILE) % D] = 0x70
    return vb


def host_case(seed, lens, G, Hkv, D, B):
    """The same on the host alone."""
    rng = np.random.default_rng(seed)
    bt, pool = tables(rng, lens, B)
    kb, ks = cache(rng, pool, Hkv, B, D)
    vs = np.full_like(ks, 2.0 ** -7)
    q64 = rng.standard_normal((len(lens), G * Hkv, D))
    return dict(bt=bt, kb=kb, vb=tile_values(kb, bt, lens), ks=ks, vs=vs, q64=q64, lens=np.asarray(lens, np.int32),
                cu=cu_of([1] * len(lens)), scale=1.0 / np.sqrt(D))


def sharp_case(seed, lens, qlens, G, Hkv, D, B):
    c = attention_case(seed, lens, qlens, G, Hkv, D, B, qscale=1.0)
    c["vb"], c["vs"] = tile_values(c["vb"], c["bt"], lens), np.full_like(c["vs"], 2.0 ** -7)
    c["dev"].update(v=to_cache(c["vb"]), vs=to_dev(c["vs"]))
    return c


def reference(c, **kw):
    """(result, how far off it may be in fp32)."""
    args = (c["q64"], c["kb"], c["vb"], c["ks"], c["vs"], c["bt"], c["lens"], c["cu"], c["scale"])
    ref, spread, scores = R.attention_fp8(*args)
    return ref, R.attention_bound(ref, spread, scores, 1, R.attention_floor(*args), False, **kw)


def check_sharp(c, out, what=""):
    ref, tol = reference(c)
    err = np.abs(out.double().cpu().numpy() - ref)
    worst = np.unravel_index(np.argmax(err - tol), err.shape)
    assert np.all(err <= tol), f"{what}: off by {err[worst]:.3e}, {tol[worst]:.3e} allowed at {worst}"
