"""Attention over the 8-bit paged cache against the float64 attention of the
values that the cache stands for (bounds: fp8_ref.attention_bound)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_122_gb300 as pk
from fp8lib import DEV, attend, attention_case, cache, check_attention, to_cache, to_dev
from oracle import fp8_ref as R

pytestmark = pytest.mark.gpu

LENS = [1, 2, 15, 127, 128, 129, 255, 256, 257, 700, 0, 1500]


@pytest.mark.parametrize("G", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("D,Hkv,B", [(128, 2, 16), (64, 2, 8), (64, 3, 32), (128, 3, 8), (64, 4, 16), (128, 1, 32)])
def test_decode_matches(G, D, Hkv, B):
    c = attention_case(G * 10 + Hkv, LENS, [1] * len(LENS), G, Hkv, D, B)
    out = attend(c)
    check_attention(c, out, f"G={G} D={D} Hkv={Hkv} B={B}")
    assert torch.all(out[LENS.index(0)] == 0)
    bf = attend(c, torch.bfloat16)
    check_attention(c, bf, "bf16")
    assert torch.equal(bf, out.to(torch.bfloat16))
    assert torch.equal(attend(c), out)                          # run to run
    assert pk.pk_get_device_error() == 0


@pytest.mark.parametrize("G,qmax", [(8, 2), (4, 3), (2, 8), (1, 16), (16, 1), (1, 5), (4, 4)])
@pytest.mark.parametrize("D,Hkv,B", [(128, 2, 16), (64, 2, 32), (64, 3, 8)])
def test_multi_query_matches(G, qmax, D, Hkv, B):
    rng = np.random.default_rng(qmax)
    qlens = [min(n, int(rng.integers(0, qmax + 1))) for n in LENS]
    qlens[-1] = qmax
    c = attention_case(G + qmax, LENS, qlens, G, Hkv, D, B)
    check_attention(c, attend(c, multi=True), f"G={G} q={qmax}")
    check_attention(c, attend(c, torch.bfloat16, multi=True), "bf16")
    assert pk.pk_get_device_error() == 0


def test_one_query_a_sequence_is_the_decode_call():
    c = attention_case(1, LENS, [1] * len(LENS), 8, 2, 128, 16)
    c["cu"] = np.arange(len(LENS) + 1, dtype=np.int32)
    live = [i for i, n in enumerate(LENS) if n]
    a, b = attend(c), attend(c, multi=True)
    assert torch.equal(a[live], b[live])
    assert pk.pk_get_device_error() == pk._native.DEVERR_SEQ_LEN    # the empty sequence has a query here


def test_long_contexts_and_many_sequences():
    c = attention_case(2, [20000, 9001, 31000], [1] * 3, 8, 2, 128, 16)
    check_attention(c, attend(c), "long")
    c = attention_case(3, [40000], [1], 16, 1, 64, 8)
    check_attention(c, attend(c), "one sequence over every CTA")
    rng = np.random.default_rng(4)
    for n in (256, 257, 1300, 2100):                            # both sides of the lengths kept in shared memory
        lens = [int(x) for x in rng.integers(0, 40, size=n)]
        c = attention_case(n, lens, [1] * n, 2 if n < 2000 else 16, 1, 64, 8)
        check_attention(c, attend(c), f"{n} sequences")
    assert pk.pk_get_device_error() == 0


def test_scores_of_any_size_and_any_finite_scale():
    for qscale, scale in ((60.0, None), (1e-4, None), (2.0, -0.1), (2.0, 0.0), (1e4, 1e-5)):
        c = attention_case(5, [5, 300, 1000], [1] * 3, 8, 2, 128, 16, qscale=qscale)
        if scale is not None:
            c["scale"] = scale
        check_attention(c, attend(c), f"q x {qscale}, scale {scale}")
    c = attention_case(6, [300, 129], [1] * 2, 4, 2, 128, 16)
    c["q"].zero_()
    c["q64"] = np.zeros_like(c["q64"])
    check_attention(c, attend(c), "zero queries")


def test_a_peak_over_a_long_flat_tail():
    # One token far above thousands that share what is left: their sum is a
    # fifth of the result, each of them 2^-16 of the peak.
    L = 13000
    c = attention_case(7, [L], [1], 1, 1, 64, 16, qscale=0.0)
    kb = np.zeros_like(c["kb"])
    c["q64"] = np.zeros((1, 1, 64))
    c["q64"][0, 0, 0] = 1.0
    c["q"] = torch.from_numpy(c["q64"]).to(torch.bfloat16).to(DEV)
    peak = 6000
    block, row = c["bt"][0, peak // 16], peak % 16
    kb[block, 0, row, 0] = R.e4m3_encode(np.array(88.0))[()]
    c["ks"][:] = 1.0
    c["scale"] = 0.125                                          # the peak's score: 11 = ln 2^15.9
    c["kb"] = kb
    c["dev"]["k"], c["dev"]["ks"] = to_cache(kb), to_dev(c["ks"])
    check_attention(c, attend(c), "flat tail")


def test_scales_of_any_size():
    # Value scales that differ by 2^90 within a sequence, and scales that are
    # no powers of two.
    c = attention_case(8, [600, 40, 129], [1] * 3, 4, 2, 128, 16)
    rng = np.random.default_rng(8)
    for vs in (np.exp2(rng.integers(-60, 30, size=c["vs"].shape)), rng.uniform(0.003, 0.02, size=c["vs"].shape)):
        c["vs"] = vs.astype(np.float32)
        c["ks"] = rng.uniform(0.004, 0.01, size=c["ks"].shape).astype(np.float32)
        c["dev"]["vs"], c["dev"]["ks"] = to_dev(c["vs"]), to_dev(c["ks"])
        check_attention(c, attend(c), "scales")
    assert pk.pk_get_device_error() == 0


@pytest.mark.parametrize("D,Hkv,G", [(128, 2, 8), (64, 2, 4), (64, 3, 2), (128, 1, 16)])
def test_masked_places_may_hold_anything(D, Hkv, G):
    # NaN bytes in every row behind a sequence's last token, in every block no
    # table names, and bad ids behind the tables' last entries.
    lens = [1, 17, 130, 300, 128]
    c = attention_case(9, lens, [1] * 5, G, Hkv, D, 16, pad=2 ** 31 - 1)
    used = np.zeros(c["kb"].shape[:3], dtype=bool)
    for s, n in enumerate(lens):
        for j in range(n):
            used[c["bt"][s, j // 16], :, j % 16] = True
    for name in ("kb", "vb"):
        c[name] = c[name].copy()
        c[name][~used] = 0x7F
    for name in ("ks", "vs"):
        c[name] = c[name].copy()
        c[name][~used.any(axis=(1, 2))] = np.nan                # scales of blocks that no table names
    c["dev"].update(k=to_cache(c["kb"]), v=to_cache(c["vb"]), ks=to_dev(c["ks"]), vs=to_dev(c["vs"]))
    clean = {n: np.where(np.isnan(c[n]), 1.0, c[n]) for n in ("ks", "vs")}
    kb, vb = (np.where(used[..., None], c[n], 0) for n in ("kb", "vb"))
    for _ in range(3):                                          # stale shared memory of the call before
        check_attention(c, attend(c), "masked", kb, vb, clean["ks"], clean["vs"])
    assert pk.pk_get_device_error() == 0


def test_nan_of_an_attended_token_shows():
    c = attention_case(10, [40, 300, 1000], [1] * 3, 4, 2, 128, 16)
    good = attend(c)
    for where in ("k", "v"):
        c["dev"][where].view(torch.uint8)[int(c["bt"][1, 3]), 1, 5, 7] = 0x7F
        out = attend(c)
        assert torch.equal(out[[0, 2]], good[[0, 2]]) and torch.equal(out[1, :4], good[1, :4])
        hit = out[1, 4:] if where == "k" else out[1, 4:, 7]
        assert torch.all(torch.isnan(hit))
        c["dev"][where].view(torch.uint8)[int(c["bt"][1, 3]), 1, 5, 7] = 0
    c["q"][2, 3, 9] = float("inf")
    out = attend(c)
    assert torch.all(torch.isnan(out[2, 3])) and torch.all(torch.isfinite(out[:2]))


@pytest.mark.parametrize("D,Hkv,G", [(128, 2, 8), (64, 2, 4), (64, 2, 8)])
def test_bad_blocks_and_scales_are_hidden_and_reported(D, Hkv, G):
    lens = [40, 300, 700]
    c = attention_case(11, lens, [1] * 3, G, Hkv, D, 16)
    N = pk._native

    def without(block_of, heads):
        """The attention of the other tokens, by zero weights in the reference."""
        q64, out = c["q64"], np.zeros((3, G * Hkv, D))
        for s, n in enumerate(lens):
            K, V = R.rows_fp8(c["kb"], c["ks"], c["bt"][s], n), R.rows_fp8(c["vb"], c["vs"], c["bt"][s], n)
            for h in range(G * Hkv):
                keep = np.ones(n, bool)
                if s == 1 and h // G in heads:
                    keep[block_of * 16:(block_of + 1) * 16] = False
                z = c["scale"] * K[keep, h // G] @ q64[s, h]
                p = np.exp(z - z.max())
                out[s, h] = p @ V[keep, h // G] / p.sum()
        return out
    bt = c["bt"].copy()
    for bad in (-1, c["pool"], 2 ** 31 - 1):
        bt[1, 9] = bad
        c["dev"]["bt"] = to_dev(bt)
        out = attend(c)
        assert pk.pk_get_device_error() == N.DEVERR_BLOCK_ID
        assert np.abs(out.double().cpu().numpy() - without(9, range(Hkv))).max() < 0.02
    c["dev"]["bt"] = to_dev(c["bt"])
    for name in ("ks", "vs"):
        for bad in (0.0, -1.0, float("nan"), 2.0 ** 65):
            t = c["dev"][name].clone()
            t[int(c["bt"][1, 2]), 1] = bad
            keep, c["dev"][name] = c["dev"][name], t
            out = attend(c)
            c["dev"][name] = keep
            assert pk.pk_get_device_error() == N.DEVERR_SCALE
            assert np.abs(out.double().cpu().numpy() - without(2, [1])).max() < 0.02
    all_bad = torch.full_like(c["dev"]["ks"], float("nan"))
    keep, c["dev"]["ks"] = c["dev"]["ks"], all_bad
    assert torch.all(attend(c) == 0)                            # nothing left to attend
    c["dev"]["ks"] = keep
    assert pk.pk_get_device_error() == N.DEVERR_SCALE


def test_bad_lengths_and_query_rows():
    c = attention_case(12, [40, 300, 129], [1] * 3, 4, 2, 128, 16)
    good = attend(c)
    N = pk._native
    c["dev"]["sl"] = torch.tensor([40, -7, 10 ** 6], dtype=torch.int32, device=DEV)
    out = attend(c)
    assert pk.pk_get_device_error() & N.DEVERR_SEQ_LEN
    assert torch.equal(out[0], good[0]) and torch.all(out[1] == 0)
    m = attention_case(13, [40, 300, 129], [2, 1, 2], 4, 2, 128, 16)
    good = attend(m, multi=True)
    for cu in ([0, 2, 3, 99], [0, 2, 1, 5], [-4, 2, 3, 5], [0, 2, 5, 5]):
        out = torch.full_like(good, 9.0)
        m["dev"]["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        attend(m, multi=True, out=out)
        assert pk.pk_get_device_error() == N.DEVERR_SEQ_LEN
        if cu[:2] == [0, 2]:
            assert torch.equal(out[:2], good[:2])


def test_empty_batches_and_tiny_bounds():
    c = attention_case(14, [0, 0, 0], [1] * 3, 4, 2, 64, 16)
    assert torch.all(attend(c) == 0)
    out = torch.full((3, 8, 64), 5.0, device=DEV)
    attend(c, out=out, max_seq_len=0)
    assert torch.all(out == 0)
    c = attention_case(15, [1], [1], 1, 1, 64, 8)
    check_attention(c, attend(c, max_seq_len=1), "one token")
    empty = torch.empty(0, 8, 64, dtype=torch.bfloat16, device=DEV)
    d = c["dev"]
    got = pk.paged_attention_decode_fp8(empty[:, :1], d["k"], d["v"], d["ks"], d["vs"], d["bt"][:0], d["sl"][:0], 0.1)
    assert got.shape == (0, 1, 64)
    # A bound below a length: the first max_seq_len tokens, reported.
    c = attention_case(16, [500, 20], [1] * 2, 4, 2, 64, 16)
    out = attend(c, max_seq_len=256)
    assert pk.pk_get_device_error() == pk._native.DEVERR_SEQ_LEN
    c["lens"] = np.array([256, 20], np.int32)
    check_attention(c, out, "bounded")


def test_rows_around_the_output_and_offsets_beyond_32_bits():
    # A pool of more than 4 GiB in each cache; the sequences use its last blocks.
    P, Hkv, B, D = 300000, 8, 16, 128
    k = torch.zeros(P, Hkv, B, D, dtype=torch.uint8, device=DEV)
    v = torch.zeros_like(k)
    ks, vs = (torch.ones(P, Hkv, device=DEV) for _ in range(2))
    lens = [300, 77]
    c = attention_case(17, lens, [1, 1], 4, Hkv, D, B)
    shift = P - c["pool"]
    k[shift:], v[shift:] = to_dev(c["kb"]), to_dev(c["vb"])
    ks[shift:], vs[shift:] = to_dev(c["ks"]), to_dev(c["vs"])
    bt = np.where(c["bt"] >= 0, c["bt"] + shift, -1).astype(np.int32)
    c["dev"].update(k=k.view(torch.float8_e4m3fn), v=v.view(torch.float8_e4m3fn), ks=ks, vs=vs, bt=to_dev(bt))
    room = torch.full((6, 4 * Hkv, D), 3.0, device=DEV)
    out = attend(c, out=room[2:4])
    check_attention(c, out, "far blocks")
    assert torch.all(room[:2] == 3.0) and torch.all(room[4:] == 3.0)
    new = torch.ones(2, Hkv, D, dtype=torch.bfloat16, device=DEV)
    pk.rope_and_cache_fp8(None, new, new, c["dev"]["k"], c["dev"]["v"], ks, vs, c["dev"]["bt"], c["dev"]["sl"])
    assert torch.all(ks[to_dev(bt[0, :1].astype(np.int64))] == to_dev(c["ks"][c["bt"][0, :1]]))
    rows = torch.empty(sum(lens), Hkv, D, dtype=torch.bfloat16, device=DEV)
    rv = torch.empty_like(rows)
    pk.gather_kv_fp8(c["dev"]["k"], c["dev"]["v"], ks, vs, c["dev"]["bt"], c["dev"]["sl"],
                     torch.tensor([0, 300], device=DEV), rows, rv)
    assert torch.all(rows[299] == 1.0) and torch.all(rv[376] == 1.0)
    want = R.rows_fp8(c["kb"], c["ks"], c["bt"][0], 288)
    assert np.array_equal(rows[:288].double().cpu().numpy(), want)
    assert pk.pk_get_device_error() == 0


def test_refusals():
    c = attention_case(18, [300], [1], 4, 2, 128, 16)
    d = c["dev"]
    f = pk.paged_attention_decode_fp8
    args = (d["k"], d["v"], d["ks"], d["vs"], d["bt"], d["sl"], 0.1)
    with pytest.raises(ValueError):
        f(c["q"].expand(2, -1, -1).contiguous(), *args)
    with pytest.raises(ValueError, match="scales"):
        f(c["q"], d["k"], d["v"], d["ks"][:, :1].contiguous(), *args[3:])
    with pytest.raises(TypeError):
        f(c["q"], d["k"], d["v"], d["ks"].double(), *args[3:])
    with pytest.raises(ValueError, match="contiguous"):
        f(c["q"].expand(1, 8, 128)[:, :, ::2], *args)
    with pytest.raises(TypeError):
        f(c["q"], *args, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        f(c["q"], *args, out=torch.empty(2, 8, 128, device=DEV))
    with pytest.raises(ValueError, match="small"):
        f(c["q"], *args, workspace=torch.empty(100, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        f(c["q"], *args, workspace=torch.empty(1 << 25, dtype=torch.uint8))
    with pytest.raises(pk.PagedKVError, match="SHAPE"):
        f(c["q"], *args, max_seq_len=10 ** 6)
    with pytest.raises(pk.PagedKVError, match="UNSUPPORTED"):
        pk.paged_attention_multi_query_fp8(c["q"], d["cu"], 5, *args)
    assert pk.pk_get_device_error() == 0
