"""Small weights of the 8-bit attention: a long flat tail under one peak.

The tail's tokens all have the same weight, so that its rounding does not average
out: the result is the tail's share, off by as much as one weight is.  Many
sequences share the pages, so that a CTA walks whole sequences and the tail is
weighed against the peak (a sequence cut into short parts has parts without the
peak, whose weights are 1).
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_122_gb300 as pk
from fp8lib import DEV, attention_case, to_cache, to_dev
from fp8sharp import reference

pytestmark = pytest.mark.gpu

SHAPES = [(1, 2, 128), (4, 2, 64), (8, 1, 128), (16, 1, 128), (8, 2, 64)]     # G, KV heads, D


def tail_case(L, G, Hkv, D, peaks, scale, vs=1.0):
    """Keys 1.0 times peaks[token] at element 0, queries 1.0 there; a peak's values are 0, the others' 1."""
    c = attention_case(1, [L], [1], G, Hkv, D, 16)
    c["kb"][:], c["vb"][:] = 0, 0x38
    for token, byte in peaks.items():
        block, row = c["bt"][0, token // 16], token % 16
        c["kb"][block, :, row, 0] = byte
        c["vb"][block, :, row] = 0
    c["ks"][:], c["vs"][:] = 1.0, vs
    c["q64"] = np.zeros_like(c["q64"])
    c["q64"][0, :, 0] = 1.0
    c["scale"] = float(np.float32(scale))
    return c


def check_shared(c, sequences, what):
    """`sequences` sequences over the same pages: every row within the bound, a weight
    being off by 2^-11 of itself, and the sums of 500 products of 32 tokens by 2^-12
    (32-bit additions that may cut off: 500 x 2^-23, with room)."""
    ref, tol = reference(c, weight_error=2.0 ** -11 + 2.0 ** -12)
    q = torch.from_numpy(c["q64"]).to(torch.bfloat16).to(DEV).expand(sequences, -1, -1).contiguous()
    bt = to_dev(np.repeat(c["bt"], sequences, axis=0))
    sl = to_dev(np.repeat(c["lens"], sequences))
    out = pk.paged_attention_decode_fp8(q, to_cache(c["kb"]), to_cache(c["vb"]), to_dev(c["ks"]), to_dev(c["vs"]), bt, sl,
                                        c["scale"], out_dtype=torch.float32)
    err = np.abs(out.double().cpu().numpy() - ref)
    assert np.all(err <= tol), f"{what}: {np.max(err / tol):.2f} times what is allowed ({np.max(err / np.abs(ref)):.1e} of the result)"
    assert pk.pk_get_device_error() == 0


@pytest.mark.parametrize("bits", [10.3, 12.0, 13.67, 14.9, 15.91, 16.9, 17.9])
@pytest.mark.parametrize("G,Hkv,D", SHAPES)
def test_a_tail_keeps_its_share(G, Hkv, D, bits):
    # Down to where the bound's floor (2^-24 of the peak, a token) is a hundredth of the tail.
    L = int(min(2.0 ** bits, 16000))
    for peak in (0, L // 2, L - 1):
        c = tail_case(L, G, Hkv, D, {peak: 0x38}, bits * np.log(2.0))
        check_shared(c, 700 // Hkv, f"tail at 2^-{bits}, peak at {peak} of {L}")


@pytest.mark.parametrize("vs", [2.0 ** -40, 0.7, 3.0 * 2.0 ** 20, 2.0 ** -64, 2.0 ** 64])
def test_under_any_value_scale(vs):
    check_shared(tail_case(12000, 4, 1, 128, {5000: 0x38}, 13.67 * np.log(2.0), vs), 700, f"value scale {vs}")


@pytest.mark.parametrize("step", [0.5, 1.0, 3.0, 5.0])
@pytest.mark.parametrize("G,Hkv,D", SHAPES)
def test_peaks_that_rise(G, Hkv, D, step):
    # A peak every third tile, growing: the reference moves or not, and the tail
    # keeps its share either way.
    L = 6000
    peaks = {token: 0x20 + 2 * i for i, token in enumerate(range(100, L, 384))}    # 2^-3 to 2
    check_shared(tail_case(L, G, Hkv, D, peaks, step), 700 // Hkv, f"step {step}")
