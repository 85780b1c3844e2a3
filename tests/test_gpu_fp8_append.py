"""The append to the 8-bit cache (with rotation), the gather and the block
moves, against the float64 reference.

Scales are compared bit for bit (they follow from the inputs' exponents), and so
are values that are not rotated.  A rotated value is within half a step of
e4m3 of the exact one, which its 32-bit arithmetic (2^-21 of the pair's length,
as for the bf16 append) can move, plus that.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_122_gb300 as pk
from fp8lib import DEV, bf16, cache, cache_bytes, cu_of, tables, to_cache, to_dev
from oracle import fp8_ref as R

pytestmark = pytest.mark.gpu


def _freq(rot):
    return (10000.0 ** (-np.arange(0, rot, 2) / rot)).astype(np.float32)


def _case(seed, before, new, H, Hkv, D, B, rot, big=1.0):
    rng = np.random.default_rng(seed)
    lens = [b + n for b, n in zip(before, new)]
    bt, pool = tables(rng, lens, B)
    kb, ks = cache(rng, pool, Hkv, B, D)
    vb, vs = cache(rng, pool, Hkv, B, D)
    T = sum(new)
    q, q64 = bf16(rng, T, H, D)
    k, k64 = bf16(rng, T, Hkv, D, scale=big)
    v, v64 = bf16(rng, T, Hkv, D)
    k64[..., ::16] *= 4.0
    k = torch.from_numpy(k64).to(torch.bfloat16).to(DEV)
    return dict(lens=lens, bt=bt, kb=kb, vb=vb, ks=ks, vs=vs, q=q, q64=q64, k=k, k64=k64, v=v, v64=v64, cu=cu_of(new),
                f=_freq(rot) if rot else None, new=new)


def _run(c, q=True, **kw):
    t = dict(k=to_cache(c["kb"]), v=to_cache(c["vb"]), ks=to_dev(c["ks"]), vs=to_dev(c["vs"]))
    out = pk.rope_and_cache_fp8(c["q"] if q else None, c["k"], c["v"], t["k"], t["v"], t["ks"], t["vs"], to_dev(c["bt"]),
                                to_dev(np.asarray(c["lens"], np.int32)), None if c["f"] is None else to_dev(c["f"]), **kw)
    return out, t


def _compare(c, t, interleaved=False, factor=1.0, positions=None):
    k, v, ks, vs, exact = R.append_fp8(c["k64"], c["v64"], c["kb"], c["vb"], c["ks"], c["vs"], c["bt"], c["lens"], c["cu"],
                                       c["f"], interleaved, factor, positions)
    assert np.array_equal(t["ks"].cpu().numpy(), ks) and np.array_equal(t["vs"].cpu().numpy(), vs)
    assert np.array_equal(cache_bytes(t["v"]), v)
    got = cache_bytes(t["k"])
    if c["f"] is None:
        assert np.array_equal(got, k)
        return
    new = np.zeros(k.shape[:3], dtype=bool)
    length = np.sqrt(np.sum(c["k64"] ** 2, axis=-1)).max() * factor
    for block, row, y in exact["k"]:
        new[block, :, row] = True
        y = np.clip(y, -448, 448)
        step = R.e4m3_step(y) / 2 + 2.0 ** -21 * length / ks[block].astype(np.float64)[:, None]
        assert np.all(np.abs(R.e4m3_decode(got[block, :, row]) - y) <= step)
    assert np.array_equal(got[~new], k[~new])                   # older rows re-rounded alike, others as they were


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,B,Hkv,H,rot", [(128, 16, 8, 16, 128), (64, 8, 3, 6, 32), (128, 32, 2, 2, 48), (64, 32, 5, 5, 64),
                                           (128, 8, 1, 16, 0), (64, 16, 17, 17, 16)])
def test_chunks_of_every_length(D, B, Hkv, H, rot, interleaved):
    before = [0, 1, B - 1, B, B + 3, 5 * B, 77, 0, 9, 40]
    new = [1, B, 1, 2 * B + 1, 0, B - 1, 100, 3 * B, 2, 1]
    c = _case(D + B + Hkv, before, new, H, Hkv, D, B, rot)
    out, t = _run(c, cu_q_lens=to_dev(c["cu"]), max_q_len=max(new), interleaved=interleaved, factor=1.5)
    _compare(c, t, interleaved, 1.5)
    pos = np.concatenate([np.arange(b, b + n) for b, n in zip(before, new)])
    y = R.rope(c["q64"], pos, c["f"], interleaved, 1.5)
    length = np.sqrt(np.sum(c["q64"] ** 2, axis=-1, keepdims=True)) * 1.5
    assert np.all(np.abs(out.double().cpu().numpy() - y) <= 2.0 ** -8 * np.abs(y) + 2.0 ** -21 * length)
    assert pk.pk_get_device_error() == 0


def test_one_token_each_growing_and_keeping_scales():
    # Without cu_q_lens; key magnitudes far above and below what the blocks hold.
    for big in (1e-3, 1.0, 50.0, 1e5):
        c = _case(int(big * 7) + 1, [0, 15, 16, 17, 100, 31], [1] * 6, 8, 2, 128, 16, 128, big)
        _, t = _run(c)
        _compare(c, t)
        c = _case(int(big * 7) + 2, [5, 8, 130], [1] * 3, 8, 3, 64, 8, 0, big)
        _, t = _run(c, q=False)
        _compare(c, t)
    assert pk.pk_get_device_error() == 0


def test_unequal_batch_is_found_by_search():
    # One long chunk among many single tokens: more than twice as many cells
    # bounded by max_q_len as by the total, so sequences are found by search.
    rng = np.random.default_rng(3)
    new = [int(x) for x in rng.integers(0, 3, size=300)]
    new[137] = 700
    before = [int(x) for x in rng.integers(0, 40, size=300)]
    c = _case(4, before, new, 2, 1, 64, 16, 64)
    _, t = _run(c, cu_q_lens=to_dev(c["cu"]), max_q_len=700)
    _compare(c, t)
    assert pk.pk_get_device_error() == 0


def test_given_positions_turn_the_angles_alone():
    new = [5, 20, 1]
    c = _case(9, [3, 16, 0], new, 4, 2, 128, 16, 128)
    pos = np.random.default_rng(1).integers(0, 1 << 20, size=sum(new))
    out, t = _run(c, cu_q_lens=to_dev(c["cu"]), max_q_len=20, positions=to_dev(pos))
    _compare(c, t, positions=pos)
    y = R.rope(c["q64"], pos, c["f"])
    assert np.abs(out.double().cpu().numpy() - y).max() <= 2.0 ** -8 * np.abs(y).max() + 1e-3


def test_not_finite_and_extreme_values():
    c = _case(10, [0, 3], [4, 2], 2, 2, 64, 16, 0)
    k = c["k64"].copy()
    k[0, 0, :4] = [np.nan, np.inf, -np.inf, 1.0]
    k[1, 1, 5] = 3e38
    k[4, 0] = 0.0                                               # zeros beside older rows: the scale stays
    c["k64"], c["k"] = k, torch.from_numpy(k).to(torch.bfloat16).to(DEV)
    c["k64"] = c["k"].double().cpu().numpy()
    _, t = _run(c, cu_q_lens=to_dev(c["cu"]), max_q_len=4)
    _compare(c, t)
    z = _case(11, [0], [3], 2, 2, 64, 16, 0)
    z["k64"] = np.zeros_like(z["k64"])
    z["k"] = torch.zeros_like(z["k"])
    _, t = _run(z, cu_q_lens=to_dev(z["cu"]), max_q_len=3)
    assert np.all(t["ks"].cpu().numpy()[z["bt"][0, 0]] == 2.0 ** -64)        # nothing to hold yet
    _compare(z, t)
    assert pk.pk_get_device_error() == 0


def test_prefill_in_chunks_equals_token_by_token_scales():
    # The scale of a block only grows to what its largest token needs, however
    # the tokens arrive; values that are rounded once are the same too.
    B, L = 16, 64
    c = _case(12, [0], [L], 2, 2, 128, B, 0)
    _, whole = _run(c, cu_q_lens=to_dev(c["cu"]), max_q_len=L)
    t = dict(k=to_cache(c["kb"]), v=to_cache(c["vb"]), ks=to_dev(c["ks"]), vs=to_dev(c["vs"]))
    for i in range(L):
        pk.rope_and_cache_fp8(None, c["k"][i:i + 1], c["v"][i:i + 1], t["k"], t["v"], t["ks"], t["vs"], to_dev(c["bt"]),
                              torch.tensor([i + 1], dtype=torch.int32, device=DEV))
    blocks = c["bt"][0, :L // B]
    assert torch.equal(t["ks"][blocks], whole["ks"][blocks]) and torch.equal(t["vs"][blocks], whole["vs"][blocks])
    # Re-rounding moves only values below 2^-6 of the scale, by half of 2^-9 a time.
    a, b = (R.e4m3_decode(cache_bytes(x["k"])[blocks]) for x in (t, whole))
    assert np.all(np.abs(a - b)[np.abs(b) >= 2.0 ** -5] == 0) and np.abs(a - b).max() <= 2.0 ** -9


def test_bad_metadata_is_reported_and_nothing_of_it_written():
    new = [2, 3, 1, 4]
    c = _case(13, [5, 6, 7, 8], new, 4, 2, 64, 16, 64)
    good, t0 = _run(c, cu_q_lens=to_dev(c["cu"]), max_q_len=4)

    def call(**kw):
        a = dict(cu_q_lens=to_dev(kw.get("cu", c["cu"])), max_q_len=kw.get("mq", 4))
        t = dict(k=to_cache(c["kb"]), v=to_cache(c["vb"]), ks=to_dev(c["ks"]), vs=to_dev(c["vs"]))
        out = torch.full_like(c["q"], 9.0)
        pk.rope_and_cache_fp8(c["q"], c["k"], c["v"], t["k"], t["v"], t["ks"], t["vs"], to_dev(kw.get("bt", c["bt"])),
                              to_dev(np.asarray(kw.get("lens", c["lens"]), np.int32)), to_dev(c["f"]), q_out=out, **a)
        return out, t, pk.pk_get_device_error()
    N = pk._native
    for lens in ([7, 9, 8, -1], [7, 9, 8, 10 ** 6], [7, 9, 8, 3], [7, 9, 8, 2 ** 31 - 1]):
        out, t, err = call(lens=lens)
        assert err == N.DEVERR_SEQ_LEN
        assert torch.equal(out[:6], good[:6]) and torch.all(out[6:] == 9.0)
        blocks = to_dev(c["bt"][3, :1].astype(np.int64))
        assert torch.equal(t["k"].view(torch.uint8)[blocks], to_cache(c["kb"]).view(torch.uint8)[blocks])
    out, t, err = call(mq=3)
    assert err == N.DEVERR_SEQ_LEN and torch.all(out[6:] == 9.0) and torch.equal(out[:6], good[:6])
    for cu in ([0, 2, 5, 6, 99], [0, 2, 5, 4, 10], [-3, 2, 5, 6, 10]):
        _, _, err = call(cu=np.asarray(cu, np.int32))
        assert err == N.DEVERR_SEQ_LEN
    for bad in (-1, c["kb"].shape[0], 2 ** 31 - 1):
        bt = c["bt"].copy()
        bt[1, 0] = bad
        out, t, err = call(bt=bt)
        assert err == N.DEVERR_BLOCK_ID and torch.equal(out, good)
        assert torch.equal(t["ks"][to_dev(c["bt"][0, :1].astype(np.int64))], t0["ks"][to_dev(c["bt"][0, :1].astype(np.int64))])


def test_rows_that_run_backwards_are_reported_where_sequences_are_searched():
    from paged_kv_cache_122_gb300 import _native as N
    new = [600] + [1] * 30
    c = _case(33, [5, 5, 400] + [5] * 28, new, 4, 2, 128, 16, 64)
    cu = c["cu"].copy()
    cu[2] = 300                                                 # sequence 1 has -300 rows, sequence 2 302 of its 401
    _run(c, cu_q_lens=to_dev(cu), max_q_len=600)
    assert pk.pk_get_device_error() == N.DEVERR_SEQ_LEN
    _, t = _run(c, cu_q_lens=to_dev(c["cu"]), max_q_len=600)
    assert pk.pk_get_device_error() == 0
    _compare(c, t)


def test_scale_outside_the_range_is_reported():
    c = _case(14, [5], [1], 2, 2, 64, 16, 0)
    b = int(c["bt"][0, 0])
    for bad in (0.0, -1.0, float("nan"), float("inf"), 2.0 ** 65):
        c["ks"][b, 1] = bad
        _, t = _run(c)
        assert pk.pk_get_device_error() == pk._native.DEVERR_SCALE
        assert t["ks"][b, 1].item() == R.needed_scale(R.largest_square(c["k64"], 0, False, 1.0)[1])


@pytest.mark.parametrize("D,B,Hkv", [(64, 8, 3), (128, 16, 8), (64, 32, 1), (128, 32, 5)])
def test_gather_gives_the_values(D, B, Hkv):
    rng = np.random.default_rng(D + B)
    lens = [0, 1, B, B + 1, 300, 33, 1000]
    bt, pool = tables(rng, lens, B, pad=10 ** 6)
    kb, ks = cache(rng, pool, Hkv, B, D)
    vb, vs = cache(rng, pool, Hkv, B, D)
    total = sum(lens)
    cu = cu_of(lens)[:-1].astype(np.int64)
    ok, ov = (torch.full((total + 4, Hkv, D), 5.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pk.gather_kv_fp8(to_cache(kb), to_cache(vb), to_dev(ks), to_dev(vs), to_dev(bt), to_dev(np.asarray(lens, np.int32)),
                     to_dev(cu), ok, ov)
    want = [np.concatenate([R.rows_fp8(b, s, bt[i], n) for i, n in enumerate(lens)]) for b, s in ((kb, ks), (vb, vs))]
    assert np.array_equal(ok[:total].double().cpu().numpy(), want[0])        # exact: e4m3 times a power of two
    assert np.array_equal(ov[:total].double().cpu().numpy(), want[1])
    assert torch.all(ok[total:] == 5.0) and torch.all(ov[total:] == 5.0)
    assert pk.pk_get_device_error() == 0


def test_gather_reports_and_skips():
    rng = np.random.default_rng(2)
    lens, B = [20, 20], 16
    bt, pool = tables(rng, lens, B)
    kb, ks = cache(rng, pool, 2, B, 64)
    N = pk._native

    def go(bt=bt, ks=ks, lens=lens, cu=(0, 20), msl=None):
        ok, ov = (torch.full((40, 2, 64), 5.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        pk.gather_kv_fp8(to_cache(kb), to_cache(kb), to_dev(ks), to_dev(ks), to_dev(bt), to_dev(np.asarray(lens, np.int32)),
                         to_dev(np.asarray(cu, np.int64)), ok, ov, max_seq_len=msl)
        return ok, pk.pk_get_device_error()
    good, err = go()
    assert err == 0
    bad = bt.copy()
    bad[0, 1] = pool
    ok, err = go(bt=bad)
    assert err == N.DEVERR_BLOCK_ID and torch.equal(ok[:16], good[:16]) and torch.all(ok[16:20] == 5.0)
    s = ks.copy()
    s[bt[1, 0]] = np.nan
    ok, err = go(ks=s)
    assert err == N.DEVERR_SCALE and torch.all(ok[20:36] == 5.0) and torch.equal(ok[36:], good[36:])
    for cu in ((0, 21), (-1, 20), (0, 2 ** 62)):
        ok, err = go(cu=cu)
        assert err == N.DEVERR_SEQ_LEN
    ok, err = go(lens=[20, 10 ** 6], msl=20)
    assert err == N.DEVERR_SEQ_LEN and torch.equal(ok, good)


@pytest.mark.parametrize("D,B,Hkv", [(64, 8, 1), (128, 16, 8), (128, 32, 40)])
def test_copy_and_swap_blocks(D, B, Hkv):
    rng = np.random.default_rng(Hkv)
    P = 12
    kb, ks = cache(rng, P, Hkv, B, D)
    vb, vs = cache(rng, P, Hkv, B, D)
    pairs = np.array([[0, 7], [0, 8], [3, 9], [11, 2]], dtype=np.int64)
    t = [to_cache(kb), to_cache(vb), to_dev(ks), to_dev(vs)]
    pk.copy_blocks_fp8(*t, to_dev(pairs))
    for x, was in zip(t, (kb, vb, ks, vs)):
        was = was.copy()
        was[pairs[:, 1]] = was[pairs[:, 0]]
        assert np.array_equal(cache_bytes(x) if x.dtype == torch.float8_e4m3fn else x.cpu().numpy(), was)
    host = [torch.empty((6,) + tuple(x.shape[1:]), dtype=torch.uint8 if x.dtype == torch.float8_e4m3fn else x.dtype,
                        pin_memory=True) for x in t]
    host = [h.zero_().view(x.dtype) for h, x in zip(host, t)]
    out = np.array([[0, 5], [8, 1], [2, 2]], dtype=np.int64)
    pk.swap_blocks_fp8(host, t, to_dev(out))
    back = [torch.zeros_like(x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x).view(x.dtype) for x in t]
    pk.swap_blocks_fp8(back, host, to_dev(out[:, ::-1].copy()))
    torch.cuda.synchronize()
    for x, y in zip(t, back):
        x, y = (z.view(torch.uint8) if z.dtype == torch.float8_e4m3fn else z for z in (x, y))
        assert torch.equal(x[[0, 8, 2]], y[[0, 8, 2]]) and torch.all(y[[1, 3, 4]] == 0)
    assert pk.pk_get_device_error() == 0
    pk.copy_blocks_fp8(*t, to_dev(np.array([[0, P], [-1, 3], [1, 4]], dtype=np.int64)))
    assert pk.pk_get_device_error() == pk._native.DEVERR_PAIR
    assert torch.equal(t[0].view(torch.uint8)[1], t[0].view(torch.uint8)[4])
