"""The 8-bit decode kernel's bounded waits give up cleanly, and it plans again
where the lengths that it read ahead have changed.

As for the bf16 kernel (test_gpu_timeout.py, test_gpu_recheck.py), for one and
for two groups of softmax warps, whose give-up paths meet at named barriers.  No
fault is made: CTA 0's producers stop before a tile, so that nothing arrives on its
barriers, and the limit is a few milliseconds.
"""
import time

import numpy as np
import pytest
import torch

import paged_kv_cache_122_gb300 as pk
from fp8lib import DEV, attend, attention_case, check_attention

pytestmark = pytest.mark.gpu
N = pk._native

# (head dim, KV heads, heads per KV head): one group; one, head pairs; two; two, head pairs.
SHAPES = [(128, 8, 4), (64, 8, 4), (128, 8, 16), (64, 8, 8), (64, 3, 16)]


def _workspace(c):
    n, H, D = c["q"].shape
    cap = c["dev"]["bt"].shape[1] * c["kb"].shape[2]
    return pk.new_workspace(pk.pk_decode_fp8_workspace_bytes(n, H, c["kb"].shape[1], D, cap), DEV), cap


def _args(c, out):
    d = c["dev"]
    return out, c["q"], d["k"], d["v"], d["ks"], d["vs"], d["bt"], d["sl"], c["scale"]


@pytest.mark.parametrize("D,Hkv,G", SHAPES)
@pytest.mark.parametrize("lens,stall", [([3000] * 24, 1), ([3000] * 24, 5), ([300, 700, 129] * 40, 4), ([200] * 256, 4)])
def test_waits_run_out_and_the_next_call_is_correct(D, Hkv, G, lens, stall):
    c = attention_case(G + stall, lens, [1] * len(lens), G, Hkv, D, 16)
    ws, cap = _workspace(c)
    want = attend(c)
    out = torch.zeros_like(want)
    assert pk.pk_get_device_error() == 0
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    assert pk.pk_selftest_decode_fp8_wait_timeout(*_args(c, out), cap, ws, stall, 5000) == 0
    torch.cuda.synchronize()
    elapsed = time.perf_counter() - t0
    assert pk.pk_get_device_error() == N.DEVERR_TIMEOUT
    assert elapsed < 0.5                                        # a few limits of 5 ms, not of the 1 s of other calls
    for _ in range(2):
        assert torch.equal(attend(c, workspace=ws), want)
        assert pk.pk_get_device_error() == 0


def test_a_stall_beyond_the_range_is_none():
    c = attention_case(3, [700, 300], [1, 1], 4, 2, 128, 16)
    ws, cap = _workspace(c)
    out = torch.zeros(2, 8, 128, device=DEV)
    assert pk.pk_selftest_decode_fp8_wait_timeout(*_args(c, out), cap, ws, 1000, 5000) == 0
    check_attention(c, out, "no stall")
    assert torch.equal(out, attend(c)) and pk.pk_get_device_error() == 0


@pytest.mark.parametrize("D,Hkv,G", SHAPES)
@pytest.mark.parametrize("kind", ["zeros", "reversed", "out of range", "same"])
def test_stale_lengths_give_the_normal_result(D, Hkv, G, kind):
    rng = np.random.default_rng(G)
    lens = [int(x) for x in rng.integers(0, 3000, size=60)]
    c = attention_case(G, lens, [1] * 60, G, Hkv, D, 16)
    ws, cap = _workspace(c)
    stale = {"zeros": np.zeros(60), "reversed": lens[::-1], "out of range": rng.integers(-5, 2 * cap, size=60), "same": lens}[kind]
    want = attend(c)
    out = torch.full_like(want, float("nan"))
    stale = torch.tensor(np.asarray(stale, np.int32), device=DEV)
    assert pk.pk_selftest_decode_fp8_stale_lengths(*_args(c, out), cap, stale, ws) == 0
    assert torch.equal(out, want) and pk.pk_get_device_error() == 0
    if kind == "reversed":
        check_attention(c, out, kind)


@pytest.mark.parametrize("D,Hkv,G", [(128, 2, 4), (128, 1, 16)])
@pytest.mark.parametrize("stale", ["ones", "reversed"])
def test_lengths_written_by_the_previous_kernel(D, Hkv, G, stale):
    # The kernel before the call writes the lengths: an append whose cache rows are
    # the lengths' array (one KV head of 64 elements: 32 int32 a slot), held up behind
    # a long fill.  The decode grid is its programmatic dependent and may read the
    # lengths before they are written.
    lens = [900, 30, 2500, 129] * 10
    c = attention_case(7, lens, [1] * 40, G, Hkv, D, 16)
    ws, cap = _workspace(c)
    want = attend(c, workspace=ws)
    first = torch.tensor([1] * 40 if stale == "ones" else lens[::-1], dtype=torch.int32, device=DEV)
    cache = torch.zeros(1, 16, 1, 64, dtype=torch.bfloat16, device=DEV)
    other = torch.zeros_like(cache)
    view = cache.view(-1).view(torch.int32)[:40]
    rows = np.zeros(64, np.int32)
    rows[:40] = lens
    k = torch.from_numpy(rows.view(np.int16).copy()).view(torch.bfloat16).view(2, 1, 64).to(DEV)
    v, slots = torch.zeros_like(k), torch.arange(2, device=DEV)
    hold = torch.empty(1 << 30, dtype=torch.uint8, device=DEV)
    c["dev"]["sl"] = view
    for _ in range(3):
        view.copy_(first)
        torch.cuda.synchronize()
        hold.fill_(1)
        pk.reshape_and_cache(k, v, cache, other, slots)
        out = attend(c, workspace=ws)
        torch.cuda.synchronize()
        assert pk.pk_get_device_error() == 0
        assert torch.equal(out, want)
