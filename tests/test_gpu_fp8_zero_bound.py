"""Attention over the 8-bit cache with max_seq_len = 0: every sequence is empty
for the call.  The same rows are written and the same faults reported as with a
bound above 0 and lengths of 0."""
import pytest
import torch

import paged_kv_cache_122_gb300 as pk
from fp8lib import DEV, attend, attention_case

pytestmark = pytest.mark.gpu
N = pk._native


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("G,Hkv,D", [(4, 2, 64), (2, 3, 128)])
def test_decode(dtype, G, Hkv, D):
    c = attention_case(1, [0, 0, 0], [1] * 3, G, Hkv, D, 16)
    for lens, err in (([0, 0, 0], 0), ([0, 5, 0], N.DEVERR_SEQ_LEN), ([0, 0, -1], N.DEVERR_SEQ_LEN)):
        c["dev"]["sl"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        room = torch.full((5, G * Hkv, D), 9.0, dtype=dtype, device=DEV)
        attend(c, out=room[1:4], max_seq_len=0)
        assert torch.all(room[1:4] == 0) and torch.all(room[0] == 9.0) and torch.all(room[4] == 9.0)
        assert pk.pk_get_device_error() == err


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_several_queries(dtype):
    # Rows that no sequence owns, behind the last one and between, and those of
    # a sequence whose rows are bad stay as they were.
    c = attention_case(2, [0, 0, 0], [2, 0, 3], 4, 2, 64, 16)
    for cu, zero in (([0, 2, 2, 5], [0, 1, 2, 3, 4]), ([0, 2, 2, 3], [0, 1, 2]), ([0, 0, 0, 0], []), ([1, 3, 2, 4], [1, 2, 2, 3]),
                     ([0, 1, 2, 99], [0, 1]), ([-2, 0, 2, 4], [0, 1, 2, 3])):
        c["dev"]["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        got = []
        for bound in (0, 16):
            out = torch.full((5, 8, 64), 9.0, dtype=dtype, device=DEV)
            attend(c, multi=True, out=out, max_seq_len=bound)
            want = torch.full_like(out, 9.0)
            want[zero] = 0
            assert torch.equal(out, want), (cu, bound)
            got.append(pk.pk_get_device_error())
        assert got[0] == got[1] == (0 if cu == [0, 0, 0, 0] else N.DEVERR_SEQ_LEN)
