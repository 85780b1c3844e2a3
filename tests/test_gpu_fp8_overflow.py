"""The 8-bit append where a pair's squares pass the fp32 range."""
import numpy as np
import pytest
import torch

import paged_kv_cache_122_gb300 as pk
from fp8lib import DEV
from oracle import fp8_ref as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
def test_a_pair_whose_squares_overflow_keeps_its_value_under_a_small_factor(interleaved):
    # x = 2^65: x^2 is beyond 32 bits, factor^2 x^2 = 2^96 would not be.  The
    # result, 2^48 at most, must not be cut off below that.
    x = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device=DEV)
    x[0, 0, 0], x[0, 0, 40] = 2.0 ** 65, 3.0
    freq = torch.ones(16, device=DEV)
    cache = pk.new_cache_fp8(1, 1, 16, 64, DEV)
    f = 2.0 ** -17
    pk.rope_and_cache_fp8(None, x, x, *cache, torch.zeros(1, 1, dtype=torch.int32, device=DEV),
                          torch.ones(1, dtype=torch.int32, device=DEV), freq, interleaved=interleaved, factor=f)
    empty = np.zeros((1, 1, 16, 64), np.uint8)
    ones = np.ones((1, 1), np.float32)
    x64 = x.double().cpu().numpy()
    kb, vb, ks, vs, _ = R.append_fp8(x64, x64, empty, empty, ones, ones, [[0]], [1], [0, 1], np.ones(16, np.float32),
                                     interleaved, f)
    assert cache[2].item() == ks[0, 0] == 2.0 ** 56 and cache[3].item() == vs[0, 0]
    assert np.array_equal(cache[0].view(torch.uint8).cpu().numpy(), kb)
    held = R.e4m3_decode(kb)[0, 0, 0, 0] * ks[0, 0]
    assert abs(held - 2.0 ** 48) <= 2.0 ** 46                   # half a step of e4m3 at that scale
    assert pk.pk_get_device_error() == 0
