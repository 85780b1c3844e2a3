"""Attention over an 8-bit cache whose value scales span the whole accepted
range, 2^-64 to 2^64.

With equal scores every token has its share of the denominator whatever its
value scale, so a block at one end must weigh as much there as one at the other.
The value rows are positive: the result is then as large as the sum of
magnitudes that bounds its error (fp8_ref.attention_bound), and a share that is
lost shows as a factor.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_122_gb300 as pk
from fp8lib import DEV, attend, attention_case, check_attention, to_cache, to_dev

pytestmark = pytest.mark.gpu

LOW, HIGH = 2.0 ** -64, 2.0 ** 64


def _positive(c, scale_of, seed=0):
    """Positive values, small scores, and scale_of(sequence, page) for every block."""
    rng = np.random.default_rng(seed)
    c["vb"] = (rng.integers(0x50, 0x70, size=c["vb"].shape)).astype(np.uint8)
    c["ks"][:] = 2.0 ** -9
    for s, n in enumerate(c["lens"]):
        for j in range(-(-int(n) // c["kb"].shape[2])):
            c["vs"][c["bt"][s, j]] = np.float32(scale_of(s, j))
    c["dev"].update(v=to_cache(c["vb"]), ks=to_dev(c["ks"]), vs=to_dev(c["vs"]))
    return c


@pytest.mark.parametrize("D,Hkv,G", [(128, 2, 1), (128, 1, 4), (64, 2, 4), (64, 3, 8), (128, 2, 16), (64, 2, 16)])
@pytest.mark.parametrize("low_first", [True, False])
def test_both_ends_in_one_tile(D, Hkv, G, low_first):
    c = attention_case(1, [32, 20, 128], [1] * 3, G, Hkv, D, 16, qscale=0.1)
    _positive(c, lambda s, j: LOW if (j % 2 == 0) == low_first else HIGH)
    check_attention(c, attend(c), f"one tile, low first {low_first}")
    assert pk.pk_get_device_error() == 0


@pytest.mark.parametrize("D,Hkv,G", [(128, 1, 4), (64, 2, 4), (128, 1, 16)])
@pytest.mark.parametrize("kind", ["by tile", "halves up", "halves down", "random"])
def test_both_ends_across_tiles_and_parts(D, Hkv, G, kind):
    # Three tiles a sequence, some of them cut between two CTAs; one sequence over dozens.
    rng = np.random.default_rng(5)
    coin = rng.integers(0, 2, size=4096)
    for lens in ([384] * 500, [5000], [300, 9000, 64]):
        def scale_of(s, j):
            tile, tiles = j // 8, -(-lens[s] // 128)
            high = {"by tile": tile % 2, "halves up": tile >= tiles / 2, "halves down": tile < tiles / 2,
                    "random": coin[(s * 7 + j) % 4096]}[kind]
            return HIGH if high else LOW
        c = attention_case(2, lens, [1] * len(lens), G, Hkv, D, 16, qscale=0.1)
        _positive(c, scale_of)
        out = attend(c)
        check_attention(c, out, f"{len(lens)} sequences, {kind}")
        assert torch.equal(out, attend(c))
    assert pk.pk_get_device_error() == 0


def test_ends_that_are_no_powers_of_two_and_shares_far_apart():
    # 1.9 x 2^63 and 1.1 x 2^-64; scores that leave the low blocks all of the
    # weight but for 2^-20.
    c = attention_case(3, [700, 64], [1] * 2, 4, 2, 128, 16, qscale=0.1)
    _positive(c, lambda s, j: 1.9 * 2.0 ** 63 if j % 3 == 1 else 1.1 * 2.0 ** -64)
    check_attention(c, attend(c), "no powers of two")
    c = attention_case(4, [256], [1], 1, 1, 128, 16, qscale=0.0)
    _positive(c, lambda s, j: HIGH if j < 8 else LOW)
    c["kb"][:] = 0
    for j in range(8, 16):
        c["kb"][c["bt"][0, j], 0, :, 0] = 0x38                  # 1.0
    c["ks"][:] = 1.0
    c["q64"][0, 0, 0] = 14.0
    c["q"] = torch.from_numpy(c["q64"]).to(torch.bfloat16).to(DEV)
    c["scale"] = 1.0                                            # the low blocks' score: 14 = ln 2^20.2
    c["dev"].update(k=to_cache(c["kb"]), ks=to_dev(c["ks"]))
    check_attention(c, attend(c), "shares far apart")
    assert pk.pk_get_device_error() == 0


@pytest.mark.parametrize("G,q", [(4, 2), (8, 2)])
def test_both_ends_with_several_queries(G, q):
    c = attention_case(6, [40, 300, 700], [q] * 3, G, 2, 64, 16, qscale=0.1)
    _positive(c, lambda s, j: HIGH if j % 2 else LOW)
    check_attention(c, attend(c, multi=True), f"G={G}, {q} queries")
    assert pk.pk_get_device_error() == 0
