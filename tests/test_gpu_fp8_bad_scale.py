"""An append to a block whose older tokens' scale is not one the cache may hold.

The older rows stand for nothing any more: they become NaN, the block takes the
new rows' scale, and the call reports PK_DEVERR_SCALE.  No value that was never
written may come out of a later call.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_122_gb300 as pk
from fp8lib import DEV, bf16, cache, cache_bytes, cu_of, tables, to_cache, to_dev
from oracle import fp8_ref as R

pytestmark = pytest.mark.gpu

BAD = (0.0, -1.0, float("nan"), float("inf"), 2.0 ** 65, 2.0 ** -65)


@pytest.mark.parametrize("D,B,Hkv", [(64, 16, 2), (128, 8, 3), (128, 32, 1)])
@pytest.mark.parametrize("which", ["k", "v"])
def test_older_rows_become_nan_and_others_keep_their_values(D, B, Hkv, which):
    rng = np.random.default_rng(D + B)
    before, new = [5, B + 3, 2 * B], [1, 2, 3]
    lens = [b + n for b, n in zip(before, new)]
    bt, pool = tables(rng, lens, B)
    kb, ks = cache(rng, pool, Hkv, B, D)
    vb, vs = cache(rng, pool, Hkv, B, D)
    k, k64 = bf16(rng, sum(new), Hkv, D)
    v, v64 = bf16(rng, sum(new), Hkv, D)
    h = Hkv - 1
    for bad in BAD:
        s = dict(k=ks.copy(), v=vs.copy())
        s[which][bt[0, 0], h] = bad
        s[which][bt[1, 1], h] = bad
        s[which][bt[2, 2], h] = bad                             # no older token there: any scale will do
        t = dict(k=to_cache(kb), v=to_cache(vb), ks=to_dev(s["k"]), vs=to_dev(s["v"]))
        pk.rope_and_cache_fp8(None, k, v, t["k"], t["v"], t["ks"], t["vs"], to_dev(bt), to_dev(np.asarray(lens, np.int32)),
                              cu_q_lens=to_dev(cu_of(new)), max_q_len=3)
        assert pk.pk_get_device_error() == pk._native.DEVERR_SCALE
        want = R.append_fp8(k64, v64, kb, vb, s["k"], s["v"], bt, lens, cu_of(new))
        for name, x, scales in (("k", want[0], want[2]), ("v", want[1], want[3])):
            assert np.array_equal(t[name + "s"].cpu().numpy(), scales)
            assert np.array_equal(cache_bytes(t[name]), x)
        got = cache_bytes(t[which])
        assert np.all(got[bt[0, 0], h, :5] == 0x7F) and np.all(got[bt[1, 1], h, :3] == 0x7F)

        # What a later call gives: NaN for the lost rows, nothing else of them.
        rows = [torch.zeros(sum(lens), Hkv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        pk.gather_kv_fp8(t["k"], t["v"], t["ks"], t["vs"], to_dev(bt), to_dev(np.asarray(lens, np.int32)),
                         to_dev(cu_of(lens)[:-1].astype(np.int64)), *rows)
        x = rows[0 if which == "k" else 1]
        at = cu_of(lens)
        assert torch.all(torch.isnan(x[:5, h])) and torch.all(torch.isfinite(x[5:at[1]]))
        assert torch.all(torch.isnan(x[at[1] + B:at[1] + B + 3, h])) and torch.all(torch.isfinite(x[at[2]:]))
        q = torch.ones(3, 4 * Hkv, D, dtype=torch.bfloat16, device=DEV)
        out = pk.paged_attention_decode_fp8(q, t["k"], t["v"], t["ks"], t["vs"], to_dev(bt),
                                            to_dev(np.asarray(lens, np.int32)), D ** -0.5)
        assert torch.all(torch.isnan(out[:2, 4 * h:])) and torch.all(torch.isfinite(out[2]))
        assert torch.all(torch.isfinite(out[:2, :4 * h]))
        assert pk.pk_get_device_error() == 0
