"""Merges of the 8-bit attention's cut sequences, in cases where every tile shows."""
import numpy as np
import pytest
import torch

import paged_kv_cache_122_gb300 as pk
from fp8lib import DEV, attend, check_attention, to_cache, to_dev
from fp8sharp import check_sharp, sharp_case
from oracle import fp8_ref as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,G,Hkv,D,B", [
    ([40000], 16, 1, 64, 8),                                    # one sequence over every CTA
    ([131072], 4, 1, 128, 16), ([131072], 1, 1, 128, 32),
    ([40001], 4, 2, 64, 16), ([20000, 9001, 31000], 8, 2, 128, 16),
    ([70000, 129, 70000], 2, 3, 64, 32),
    ([300] * 700, 4, 1, 128, 16), ([300] * 700, 8, 2, 64, 8),   # cut in two, many times
    ([257 + 90 * i for i in range(60)], 16, 2, 128, 16),
])
def test_every_part_counts(lens, G, Hkv, D, B):
    c = sharp_case(len(lens) + G, lens, [1] * len(lens), G, Hkv, D, B)
    out = attend(c)
    check_sharp(c, out, f"{len(lens)} sequences")
    assert torch.equal(out, attend(c))
    assert pk.pk_get_device_error() == 0


@pytest.mark.parametrize("lens,q,G,Hkv,D,B", [([50000, 3000], 2, 8, 1, 128, 16), ([30000] * 2, 4, 2, 2, 64, 32),
                                              ([400] * 300, 3, 4, 1, 64, 8)])
def test_every_part_counts_with_several_queries(lens, q, G, Hkv, D, B):
    c = sharp_case(q, lens, [q] * len(lens), G, Hkv, D, B)
    check_sharp(c, attend(c, multi=True), f"{q} queries")
    assert pk.pk_get_device_error() == 0


@pytest.mark.parametrize("G,Hkv,D", [(4, 1, 128), (16, 1, 64), (4, 2, 64)])
def test_references_that_rise_along_the_sequence(G, Hkv, D):
    # Keys grow towards the end: every part has another reference, and tiles of one
    # part move it; the weights still reach over all parts (e^3 from first to last).
    L = 30000
    c = sharp_case(3, [L], [1], G, Hkv, D, 16)
    q = np.zeros_like(c["q64"])
    q[0, :, 0] = np.linspace(1.0, 3.0, G * Hkv)
    c["kb"][:] = 0
    levels = np.array([2.0 ** -6 * m for m in range(1, 65)])    # 0 to 1 in steps that e4m3 holds to 2^-4
    pages = -(-L // 16)
    for j in range(pages):
        c["kb"][c["bt"][0, j], :, :, 0] = R.e4m3_encode(levels[j * 64 // pages])[()]
    c["ks"][:], c["scale"] = 1.0, 1.0
    c["q64"], c["q"] = q, torch.from_numpy(q).to(torch.bfloat16).to(DEV)
    c["q64"] = c["q"].double().cpu().numpy()
    c["dev"].update(k=to_cache(c["kb"]), ks=to_dev(c["ks"]))
    check_sharp(c, attend(c), "rising")
    check_attention(c, attend(c), "rising")
    assert pk.pk_get_device_error() == 0
