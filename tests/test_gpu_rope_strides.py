"""The token stride of a single token, which no address depends on."""
import numpy as np
import pytest
import torch

import paged_kv_cache_122_gb300 as pk
from fp8lib import DEV, bf16, to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("stride", [515, 3, 0])
def test_the_stride_of_a_single_token_does_not_matter(stride):
    rng = np.random.default_rng(1)
    freq = to_dev((10000.0 ** (-np.arange(0, 64, 2) / 64)).astype(np.float32))
    q, k, v = (bf16(rng, 1, h, 64)[0] for h in (8, 2, 2))
    odd = [x.as_strided(x.shape, (stride, 64, 1)) for x in (q, k, v)]
    bt, sl = torch.tensor([[1]], dtype=torch.int32, device=DEV), torch.tensor([3], dtype=torch.int32, device=DEV)
    got = []
    for a in ((q, k, v), odd):
        kc, vc = (torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        room = torch.zeros(1, 8, 64, dtype=torch.bfloat16, device=DEV)
        out = pk.rope_and_cache(*a, kc, vc, torch.tensor([5], device=DEV), torch.tensor([7], device=DEV), freq,
                                q_out=room.as_strided(room.shape, (stride, 64, 1)))
        c8 = pk.new_cache_fp8(2, 2, 16, 64, DEV)
        out8 = pk.rope_and_cache_fp8(*a, *c8, bt, sl, freq)
        got.append([out, kc, vc, out8, *(x.view(torch.uint8) for x in c8)])
    for x, y in zip(*got):
        assert torch.equal(x, y)
    assert torch.any(got[0][1] != 0) and pk.pk_get_device_error() == 0
