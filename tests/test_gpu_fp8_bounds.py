"""Bounds of the 8-bit cache's calls that do not fit 32 bits."""
import numpy as np
import pytest
import torch

import paged_kv_cache_122_gb300 as pk
from fp8lib import DEV, attend, attention_case, bf16

pytestmark = pytest.mark.gpu


def test_bounds_beyond_32_bits_are_not_taken_modulo():
    c = attention_case(2, [40, 17], [2, 1], 4, 2, 64, 16)
    want = attend(c, multi=True)
    c["qmax"] = (1 << 32) + 2
    with pytest.raises(pk.PagedKVError, match="UNSUPPORTED"):   # far more than 16 columns
        attend(c, multi=True)
    c["qmax"] = 2
    for bound in ((1 << 32) + 16, 1 << 32, -(1 << 32) + 16):    # not what the tables hold
        with pytest.raises(pk.PagedKVError, match="SHAPE"):
            attend(c, multi=True, max_seq_len=bound)
    assert torch.equal(attend(c, multi=True), want)
    # A bound that is only a bound: the append takes any that is large enough.
    k, v = (bf16(np.random.default_rng(3), 3, 2, 64)[0] for _ in range(2))
    got = []
    for bound in (2, 1 << 31, (1 << 32) + 1):
        cache = pk.new_cache_fp8(c["pool"], 2, 16, 64, DEV)
        pk.rope_and_cache_fp8(None, k, v, *cache, c["dev"]["bt"], c["dev"]["sl"], cu_q_lens=c["dev"]["cu"], max_q_len=bound)
        got.append([x.view(torch.uint8) for x in cache])
        assert pk.pk_get_device_error() == 0
    for other in got[1:]:
        assert all(torch.equal(x, y) for x, y in zip(got[0], other))
    rows = [torch.zeros(57, 2, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    with pytest.raises(pk.PagedKVError, match="SHAPE"):
        pk.gather_kv_fp8(c["dev"]["k"], c["dev"]["v"], c["dev"]["ks"], c["dev"]["vs"], c["dev"]["bt"], c["dev"]["sl"],
                         torch.tensor([0, 40], device=DEV), *rows, max_seq_len=(1 << 32) + 40)
